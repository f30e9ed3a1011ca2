"""Rotation of heads and appends with it, CPU side: frequencies, refusals before
any CUDA call, the header from strict C99, the NVTX ranges."""
import copy
import ctypes
import math
import os
import pickle
import re
import shutil
import subprocess
import sys

import pytest
import torch

import rotary_ref as ref
from paged_kv_cache_255_gb300 import build
from paged_kv_cache_255_gb300 import pagedattn as pa

from test_tracing import recorder  # noqa: F401  (fixture)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("scaling", [None, "linear", "ntk", "yarn", "banded"])
@pytest.mark.parametrize("rot_dim,base,factor,original", [(128, 1e4, 8.0, 4096), (64, 5e5, 32.0, 8192),
                                                          (16, 1e4, 2.0, 64), (96, 1.5, 1.0, 1)])
def test_frequencies(pa_lib, scaling, rot_dim, base, factor, original):
    R = pa.Rotary(rot_dim, base=base, scaling=scaling, factor=factor, original_context=original)
    want = ref.frequencies(rot_dim, base, scaling, factor, original)
    # powers and products of a few roundings in 64 bits, cut to whole units of 2^-64 turns
    for got, theta in zip(R._struct.turns, want):
        assert abs(got / 2 ** 64 * 2 * math.pi - theta) <= 1e-12 * theta + 2 * math.pi * 2 ** -64
    assert R.rot_dim == rot_dim and not R.interleaved
    assert list(R._struct.turns)[rot_dim // 2:] == [0] * (64 - rot_dim // 2)


def test_copies_do_not_share_memory(pa_lib):
    R = pa.Rotary(64, interleaved=True, scaling="yarn", factor=4.0, original_context=4096)
    for C in (copy.copy(R), copy.deepcopy(R), pickle.loads(pickle.dumps(R))):
        assert bytes(C._struct) == bytes(R._struct) and (C.rot_dim, C.interleaved) == (64, True)
        assert C._addr == ctypes.addressof(C._struct) != R._addr


def test_frequencies_of_more_than_a_turn_and_negative(pa_lib):
    f = [2 * math.pi * x for x in (0.25, 1.25, -0.25, -1.0, 3.0, 0.0, 1000.5, -1e-30)]
    R = pa.Rotary(16, frequencies=f)
    got = [t / 2 ** 64 for t in R._struct.turns[:8]]
    for g, w in zip(got, (0.25, 0.25, 0.75, 0.0, 0.0, 0.0, 0.5, 0.0)):
        assert min(abs(g - w), 1 - abs(g - w)) < 1e-12
    assert R.amplitude == 1.0


@pytest.mark.parametrize("kw,status", [
    (dict(rot_dim=0), pa.PA_ERR_UNSUPPORTED), (dict(rot_dim=24), pa.PA_ERR_UNSUPPORTED),
    (dict(rot_dim=144), pa.PA_ERR_UNSUPPORTED), (dict(rot_dim=-16), pa.PA_ERR_UNSUPPORTED),
    (dict(base=1.0), pa.PA_ERR_INVALID_ARG), (dict(base=float("nan")), pa.PA_ERR_INVALID_ARG),
    (dict(base=float("inf")), pa.PA_ERR_INVALID_ARG),
    (dict(scaling="linear", factor=0.5), pa.PA_ERR_INVALID_ARG),
    (dict(scaling="ntk", factor=float("inf")), pa.PA_ERR_INVALID_ARG),
    (dict(scaling="yarn", factor=2.0), pa.PA_ERR_INVALID_ARG),                     # no original context
    (dict(scaling="banded", factor=2.0, original_context=64, low=4.0, high=4.0), pa.PA_ERR_INVALID_ARG),
    (dict(scaling="yarn", factor=2.0, original_context=64, low=0.0), pa.PA_ERR_INVALID_ARG),
    (dict(amplitude=float("nan")), pa.PA_ERR_INVALID_ARG),
    (dict(rot_dim=16, frequencies=[float("nan")] * 8), pa.PA_ERR_INVALID_ARG),
    (dict(rot_dim=16, frequencies=[1e7] * 8), pa.PA_ERR_INVALID_ARG),
    (dict(rot_dim=8, frequencies=[1.0] * 4), pa.PA_ERR_UNSUPPORTED),
])
def test_rotations_that_are_refused(pa_lib, kw, status):
    with pytest.raises(pa.PagedAttnError) as e:
        pa.Rotary(**kw)
    assert e.value.status == status


def test_rotations_the_binding_refuses(pa_lib):
    for kw in (dict(scaling="other"), dict(rot_dim=16, frequencies=[1.0] * 7), dict(amplitude=0.0)):
        with pytest.raises(ValueError):
            pa.Rotary(**kw)


def rotary(**kw):
    r = pa._RotaryStruct(rot_dim=128, interleaved=0, amplitude=1.0)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


OK = rotary()
BAD_DIM, BAD_AMPLITUDE = rotary(rot_dim=24), rotary(amplitude=float("inf"))

SHARED = [
    (dict(D=64), pa.PA_ERR_UNSUPPORTED),
    (dict(T=-1), pa.PA_ERR_INVALID_ARG),
    (dict(Hq=-1), pa.PA_ERR_INVALID_ARG),
    (dict(Hq=1 << 20), pa.PA_ERR_UNSUPPORTED),
    (dict(T=1 << 31), pa.PA_ERR_UNSUPPORTED),
    (dict(q=None), pa.PA_ERR_INVALID_ARG),
    (dict(q=24), pa.PA_ERR_INVALID_ARG),
    (dict(qts=-1024), pa.PA_ERR_INVALID_ARG),
    (dict(qts=1025), pa.PA_ERR_INVALID_ARG),
    (dict(qhs=132), pa.PA_ERR_INVALID_ARG),
    (dict(qo=None), pa.PA_ERR_INVALID_ARG),
    (dict(qohs=120), pa.PA_ERR_INVALID_ARG),            # output heads overlap
    (dict(qots=2040), pa.PA_ERR_INVALID_ARG),           # output tokens overlap
    (dict(qots=0), pa.PA_ERR_INVALID_ARG),
    (dict(qots=128, qohs=376), pa.PA_ERR_INVALID_ARG),  # heads outermost, and overlapping
    (dict(k=None), pa.PA_ERR_INVALID_ARG),
    (dict(khs=4), pa.PA_ERR_INVALID_ARG),
    (dict(pos=None), pa.PA_ERR_INVALID_ARG),
    (dict(rot=BAD_DIM), pa.PA_ERR_UNSUPPORTED),
    (dict(rot=BAD_AMPLITUDE), pa.PA_ERR_INVALID_ARG),
    (dict(qw=8), pa.PA_ERR_INVALID_ARG),
    (dict(kw=40), pa.PA_ERR_INVALID_ARG),
    (dict(eps=-1e-6), pa.PA_ERR_INVALID_ARG),
    (dict(eps=float("nan")), pa.PA_ERR_INVALID_ARG),
    (dict(T=0, q=None, k=None, v=None, qo=None, pos=None, sm=None), pa.PA_OK),
]


def arguments(over):
    a = dict(q=16, qts=2048, qhs=128, qo=16, qots=2048, qohs=128, Hq=16, k=16, kts=1024, khs=128, ko=16, kots=1024,
             kohs=128, v=16, vts=1024, vhs=128, Hkv=8, D=128, kc=16, vc=16, sm=16, bs=16, NB=10, layout=0, pos=16, T=4,
             rot=OK, qw=None, kw=None, eps=1e-6)
    a.update(over)
    a["rot"] = None if a["rot"] is None else ctypes.addressof(a["rot"])
    return a


@pytest.mark.parametrize("over,want", SHARED + [
    (dict(Hkv=-1), pa.PA_ERR_INVALID_ARG),
    (dict(ko=None), pa.PA_ERR_INVALID_ARG),
    (dict(kohs=0), pa.PA_ERR_INVALID_ARG),
    (dict(Hq=0, Hkv=0, q=None, qo=None, k=None), pa.PA_OK),
])
def test_rotate_host_checks(pa_lib, over, want):
    a = arguments(over)
    order = "q qts qhs qo qots qohs Hq k kts khs ko kots kohs Hkv D pos T rot qw kw eps".split()
    assert pa_lib.pa_rotate(*(a[n] for n in order), None) == want


@pytest.mark.parametrize("over,want", SHARED + [
    (dict(Hkv=0), pa.PA_ERR_INVALID_ARG),
    (dict(v=None), pa.PA_ERR_INVALID_ARG),
    (dict(v=8), pa.PA_ERR_INVALID_ARG),
    (dict(vts=1020), pa.PA_ERR_INVALID_ARG),
    (dict(kc=24), pa.PA_ERR_INVALID_ARG),
    (dict(vc=None), pa.PA_ERR_INVALID_ARG),
    (dict(sm=None), pa.PA_ERR_INVALID_ARG),
    (dict(bs=24), pa.PA_ERR_UNSUPPORTED),
    (dict(layout=2), pa.PA_ERR_INVALID_ARG),
    (dict(NB=-1), pa.PA_ERR_INVALID_ARG),
])
def test_append_host_checks(pa_lib, over, want):
    a = arguments(over)
    order = ("q qts qhs qo qots qohs Hq k kts khs v vts vhs Hkv D kc vc sm bs NB layout pos T rot qw kw eps").split()
    assert pa_lib.pa_append_kvcache(*(a[n] for n in order), None) == want


def test_binding_refuses(pa_lib):
    x = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    pos = torch.zeros(2, dtype=torch.int32)
    R = pa.Rotary(128)
    with pytest.raises(ValueError):
        pa.rotate(x, x, pos, R)
    with pytest.raises(ValueError):
        pa.rotate(None, None, pos, R)
    with pytest.raises(ValueError):
        pa.append_kvcache(None, x, x, x.view(1, 2, 4, 128), x.view(1, 2, 4, 128), pos.long(), pos, R)


C_PROGRAM = """
#include <stdio.h>
#include "pagedattn/rotary.h"
int main(void)
{
    pa_status_t (*init)(pa_rotary_t *, int, int, double, pa_rotary_scaling_t, double, double, double, double,
                        double) = pa_rotary_init;
    pa_status_t (*given)(pa_rotary_t *, int, int, const double *, double) = pa_rotary_init_frequencies;
    pa_status_t (*rotate)(const void *, int64_t, int64_t, void *, int64_t, int64_t, int, const void *, int64_t,
                          int64_t, void *, int64_t, int64_t, int, int, const int32_t *, int64_t,
                          const pa_rotary_t *, const void *, const void *, float, void *) = pa_rotate;
    pa_status_t (*append)(const void *, int64_t, int64_t, void *, int64_t, int64_t, int, const void *, int64_t,
                          int64_t, const void *, int64_t, int64_t, int, int, void *, void *, const int64_t *, int,
                          int64_t, pa_layout_t, const int32_t *, int64_t, const pa_rotary_t *, const void *,
                          const void *, float, void *) = pa_append_kvcache;
    pa_rotary_t r;
    double f[8] = {0};
    int bad = 0;
    bad += init(&r, 128, 0, 10000.0, PA_ROTARY_YARN, 4.0, 4096.0, 1.0, 32.0, 0.0) != PA_OK;
    bad += r.rot_dim != 128 || r.amplitude < 1.13f || r.amplitude > 1.14f;
    bad += given(&r, 16, 1, f, 1.0) != PA_OK || given(&r, 16, 2, f, 1.0) != PA_ERR_INVALID_ARG;
    bad += given(NULL, 16, 1, f, 1.0) != PA_ERR_INVALID_ARG;
    bad += init(NULL, 128, 0, 10000.0, PA_ROTARY_PLAIN, 1.0, 0.0, 0.0, 0.0, 0.0) != PA_ERR_INVALID_ARG;
    bad += rotate(NULL, 0, 0, NULL, 0, 0, 4, NULL, 0, 0, NULL, 0, 0, 2, 128, NULL, 0, &r, NULL, NULL, 0.f, NULL) != PA_OK;
    bad += append(NULL, 0, 0, NULL, 0, 0, 4, NULL, 0, 0, NULL, 0, 0, 2, 64, NULL, NULL, NULL, 16, 10,
                  PA_LAYOUT_HEAD_MAJOR, NULL, 0, &r, NULL, NULL, 0.f, NULL) != PA_ERR_UNSUPPORTED;
    printf("ok %d\\n", bad);
    return bad;
}
"""


def test_header_from_c99(pa_lib, tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not found")
    with open(os.path.join(ROOT, "include", "pagedattn", "rotary.h")) as fh:
        declared = set(re.findall(r"PA_API\s+[\w\s\*]+?\b(pa_\w+)\s*\(", fh.read()))
    assert set(re.findall(r"=\s*(pa_\w+);", C_PROGRAM)) == declared
    for n in declared:
        assert hasattr(pa_lib, n) and n in pa.SIGNATURES, n
    src, exe = tmp_path / "rotary.c", tmp_path / "rotary"
    src.write_text(C_PROGRAM)
    lib_dir = os.path.dirname(build.LIB_PATH)
    subprocess.run([gcc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I",
                    os.path.join(ROOT, "include"), str(src), "-o", str(exe), "-L", lib_dir,
                    "-lpagedattn", "-Wl,-rpath," + lib_dir], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120,
                       env=dict(os.environ, CUDA_VISIBLE_DEVICES=""))
    assert r.returncode == 0 and r.stdout.strip() == "ok 0", r.stdout + r.stderr


def test_ranges(recorder, tmp_path):  # noqa: F811
    log = tmp_path / "events.txt"
    script = (f"import sys\nsys.path.insert(0, {ROOT!r})\n"
              "from paged_kv_cache_255_gb300 import pagedattn as pa\nL = pa.lib()\n"
              "print(L.pa_rotate(*[None, 0, 0] * 2, 4, *[None, 0, 0] * 2, 2, 128, None, 0, None, None, None, 0.0, None),"
              "L.pa_append_kvcache(*[None, 0, 0] * 2, 4, *[None, 0, 0] * 2, 2, 64, None, None, None, 16, 10, 0, None, 0,"
              "None, None, None, 0.0, None))")
    env = dict(os.environ, NVTX_INJECTION64_PATH=recorder, NVTX_RECORD_PATH=str(log), CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, "-c", script], env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "0 2", r.stdout + r.stderr
    events = [ln.split(" ", 2) for ln in log.read_text().splitlines()]
    ours = [e for e in events if len(e) > 1 and e[1] == "libpagedattn"][1:]
    assert ours == [e for n in ("pa_rotate", "pa_append_kvcache")
                    for e in (["push", "libpagedattn", n], ["pop", "libpagedattn"])]
