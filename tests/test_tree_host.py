"""Decode over trees and keeping accepted tokens, CPU side: refusals before any CUDA call,
the header from strict C99, the NVTX ranges, the model that the GPU is compared with."""
import ctypes
import os
import re
import shutil
import subprocess
import sys

import numpy as np
import pytest
import torch

import tree_ref as ref
from paged_kv_cache_255_gb300 import build
from paged_kv_cache_255_gb300 import pagedattn as pa

from test_tracing import recorder  # noqa: F401  (fixture)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("over,want", [
    (dict(D=64), pa.PA_ERR_UNSUPPORTED),
    (dict(bs=24), pa.PA_ERR_UNSUPPORTED),
    (dict(bs=512), pa.PA_ERR_UNSUPPORTED),
    (dict(Hq=12, Hkv=8), pa.PA_ERR_INVALID_ARG),
    (dict(Hq=34, Hkv=2), pa.PA_ERR_UNSUPPORTED),        # group of 17
    (dict(S=-1), pa.PA_ERR_INVALID_ARG),
    (dict(T=-1), pa.PA_ERR_INVALID_ARG),
    (dict(W=0), pa.PA_ERR_INVALID_ARG),
    (dict(W=17), pa.PA_ERR_UNSUPPORTED),
    (dict(T=1 << 27), pa.PA_ERR_UNSUPPORTED),           # 2^31 rows
    (dict(mb=1 << 27), pa.PA_ERR_UNSUPPORTED),          # tokens past 32 bits
    (dict(q=None), pa.PA_ERR_INVALID_ARG),
    (dict(cl=None), pa.PA_ERR_INVALID_ARG),
    (dict(sl=None), pa.PA_ERR_INVALID_ARG),
    (dict(mask=None), pa.PA_ERR_INVALID_ARG),
    (dict(mask=20), pa.PA_ERR_INVALID_ARG),
    (dict(out=24), pa.PA_ERR_INVALID_ARG),
    (dict(v=8), pa.PA_ERR_INVALID_ARG),
    (dict(layout=5), pa.PA_ERR_INVALID_ARG),
    (dict(scale=float("inf")), pa.PA_ERR_INVALID_ARG),
    (dict(mb=0), pa.PA_ERR_INVALID_ARG),
    (dict(NB=0), pa.PA_ERR_INVALID_ARG),
    (dict(NB=1 << 27), pa.PA_ERR_UNSUPPORTED),
    (dict(S=40, mb=1 << 26), pa.PA_ERR_UNSUPPORTED),    # 40 x 8 units of 2^23 key tiles
    (dict(T=1 << 17, S=1, mb=1 << 22), pa.PA_ERR_UNSUPPORTED),  # 8 x 1024 units of 2^19
    (dict(S=0, q=None, sl=None), pa.PA_OK),
    (dict(T=0, q=None, mask=None), pa.PA_OK),
])
def test_tree_host_checks(pa_lib, over, want):
    a = dict(q=16, k=16, v=16, bt=16, mb=4, cl=16, sl=16, mask=16, W=1, scale=0.1, out=16, S=2, T=9, Hq=16, Hkv=8, D=128,
             bs=16, NB=10, layout=0, ws=16, wsb=1 << 28)
    a.update(over)
    assert pa_lib.pa_decode_tree(*a.values(), None) == want


def test_workspace_size_rejects(pa_lib):
    for args in ((12, 8, 128), (16, 8, 64), (34, 2, 128), (0, 1, 128), (16, 0, 128), (-4, -2, 128)):
        assert pa_lib.pa_decode_tree_workspace_size(*args) == 0


_keep = (ctypes.c_void_p * 2)(16, 32)
_bad = (ctypes.c_void_p * 2)(16, 24)
POOLS, MISALIGNED = (ctypes.addressof(x) for x in (_keep, _bad))


@pytest.mark.parametrize("over,want", [
    (dict(D=64), pa.PA_ERR_UNSUPPORTED),
    (dict(bs=8), pa.PA_ERR_UNSUPPORTED),
    (dict(NB=1 << 31), pa.PA_ERR_UNSUPPORTED),
    (dict(Hkv=65536), pa.PA_ERR_UNSUPPORTED),
    (dict(NB=0), pa.PA_ERR_INVALID_ARG),
    (dict(nc=-1), pa.PA_ERR_INVALID_ARG),
    (dict(caches=None), pa.PA_ERR_INVALID_ARG),
    (dict(caches=MISALIGNED), pa.PA_ERR_INVALID_ARG),
    (dict(m=0), pa.PA_ERR_INVALID_ARG),
    (dict(m=1025), pa.PA_ERR_UNSUPPORTED),
    (dict(S=-1), pa.PA_ERR_INVALID_ARG),
    (dict(S=65536), pa.PA_ERR_UNSUPPORTED),
    (dict(mb=0), pa.PA_ERR_INVALID_ARG),
    (dict(mb=1 << 27), pa.PA_ERR_UNSUPPORTED),
    (dict(bt=None), pa.PA_ERR_INVALID_ARG),
    (dict(cl=None), pa.PA_ERR_INVALID_ARG),
    (dict(sl=None), pa.PA_ERR_INVALID_ARG),
    (dict(kept=None), pa.PA_ERR_INVALID_ARG),
    (dict(layout=2), pa.PA_ERR_INVALID_ARG),
    (dict(S=0, bt=None, kept=None), pa.PA_OK),
])
def test_keep_host_checks(pa_lib, over, want):
    a = dict(caches=POOLS, nc=2, bt=16, mb=4, cl=16, sl=16, kept=16, m=5, S=2, rc=None, Hkv=8, D=128, bs=16, NB=10, layout=0)
    a.update(over)
    assert pa_lib.pa_keep_tokens(*a.values(), None) == want


def test_binding_refuses_cpu_tensors(pa_lib):
    q = torch.zeros(2, 16, 128, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        pa.decode_tree(q, q, q, i.view(2, 1), i, i, i.long().view(2, 1), 0.1)
    with pytest.raises(ValueError):
        pa.decode_tree_workspace_size(12, 8, device="cuda:0") if torch.cuda.is_available() else pa.CachePools([q])


def test_masks_of_a_tree():
    # 0 - 1 - 2, 0 - 3 - 4
    assert ref.ancestors([-1, 0, 1, 0, 3]) == [0b1, 0b11, 0b111, 0b1001, 0b11001]
    w = ref.words([1 << 64 | 3, 1 << 63], 2)
    assert w.tolist() == [[3, 1], [-1 << 63, 0]]


@pytest.mark.parametrize("hm", [False, True])
def test_the_model_keeps_the_path(hm):
    rng = np.random.default_rng(0)
    bs, NB, Hkv = 16, 12, 2
    pool = rng.integers(0, 1 << 16, size=(NB, Hkv, bs, 4) if hm else (NB, bs, Hkv, 4), dtype=np.uint16)
    tables = np.array([[3, 7, 1, 9, 0], [2, 4, 0, 0, 0]], np.int32)
    lens, starts = np.array([50, 20], np.int32), np.array([0, 30, 33], np.int32)
    refs = np.zeros(NB, np.int32)
    refs[[3, 7, 1, 9, 2, 4]] = 1
    view = pool.transpose(0, 2, 1, 3) if hm else pool
    rows = lambda s, L: view[tables[s, np.arange(L) // bs], np.arange(L) % bs].copy()     # noqa: E731
    before = rows(0, 50), rows(1, 20)
    kept = np.array([[0, 4, 5, 29, -1], [1, 0, -1, -1, -1]], np.int32)
    assert ref.keep([pool], tables, lens, starts, kept, refs, bs, hm) == {5}
    assert lens.tolist() == [24, 18] and tables.tolist() == [[3, 7, 0, 0, 0], [2, 4, 0, 0, 0]]
    assert refs[[3, 7, 2, 4]].tolist() == [1] * 4 and refs[[1, 9]].tolist() == [0, 0]
    assert np.array_equal(rows(0, 24), before[0][list(range(20)) + [20, 24, 25, 49]])
    assert np.array_equal(rows(1, 18), before[1][list(range(17)) + [18]])


C_PROGRAM = """
#include <stdio.h>
#include "pagedattn/decode_tree.h"
int main(void)
{
    size_t (*size)(int, int, int) = pa_decode_tree_workspace_size;
    pa_status_t (*tree)(const void *, const void *, const void *, const int32_t *, int, const int32_t *,
                        const int32_t *, const uint64_t *, int, float, void *, int, int, int, int, int, int, int64_t,
                        pa_layout_t, void *, size_t, void *) = pa_decode_tree;
    pa_status_t (*keep)(void *const *, int, int32_t *, int, int32_t *, const int32_t *, const int32_t *, int, int,
                        int32_t *, int, int, int, int64_t, pa_layout_t, void *) = pa_keep_tokens;
    int bad = 0;
    bad += size(12, 8, 128) != 0;
    bad += tree(NULL, NULL, NULL, NULL, 4, NULL, NULL, NULL, 1, 0.1f, NULL, 0, 0, 16, 8, 128, 16, 10,
                PA_LAYOUT_HEAD_MAJOR, NULL, 0, NULL) != PA_OK;
    bad += keep(NULL, 0, NULL, 4, NULL, NULL, NULL, PA_KEEP_MAX_TOKENS + 1, 2, NULL, 8, 128, 16, 10,
                PA_LAYOUT_TOKEN_MAJOR, NULL) != PA_ERR_UNSUPPORTED;
    bad += PA_TREE_MAX_WORDS != 16;
    printf("ok %d\\n", bad);
    return bad;
}
"""


def test_header_from_c99(pa_lib, tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not found")
    with open(os.path.join(ROOT, "include", "pagedattn", "decode_tree.h")) as fh:
        declared = set(re.findall(r"PA_API\s+[\w\s\*]+?\b(pa_\w+)\s*\(", fh.read()))
    assert set(re.findall(r"=\s*(pa_\w+);", C_PROGRAM)) == declared
    for n in declared:
        assert hasattr(pa_lib, n) and n in pa.SIGNATURES, n
    src, exe = tmp_path / "tree.c", tmp_path / "tree"
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
              "print(L.pa_decode_tree(16, 16, 16, 16, 4, 16, 16, 16, 1, 0.1, 16, 2, 9, 16, 8, 64, 16, 10, 0, 16, 99, None),"
              "L.pa_keep_tokens(None, 0, 16, 4, 16, 16, 16, 5, 0, None, 8, 128, 16, 10, 0, None))")
    env = dict(os.environ, NVTX_INJECTION64_PATH=recorder, NVTX_RECORD_PATH=str(log), CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, "-c", script], env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "2 0", r.stdout + r.stderr
    events = [ln.split(" ", 2) for ln in log.read_text().splitlines()]
    ours = [e for e in events if len(e) > 1 and e[1] == "libpagedattn"][1:]
    assert ours == [e for n in ("pa_decode_tree", "pa_keep_tokens")
                    for e in (["push", "libpagedattn", n], ["pop", "libpagedattn"])]
