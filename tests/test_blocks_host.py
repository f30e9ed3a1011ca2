"""Block operations, CPU side: the model the GPU tests compare with keeps its
own invariants, the C entry points refuse bad arguments before any CUDA call,
the header compiles as strict C99, and each call opens its NVTX range."""
import ctypes
import glob
import os
import re
import shutil
import subprocess
import sys

import numpy as np
import pytest
import torch

import blocks_ref as ref
from paged_kv_cache_255_gb300 import build
from paged_kv_cache_255_gb300 import pagedattn as pa

from test_tracing import recorder  # noqa: F401  (fixture)

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


# -- the model --------------------------------------------------------------------

def _tokens(pool, tables, lens, row, bs, head_major):
    n, nb = ref.owned(tables, lens, row, bs)
    x = pool[tables[row, :nb]]
    x = x.transpose(0, 2, 1, 3) if head_major else x
    return x.reshape(-1, *x.shape[2:])[:n]


@pytest.mark.parametrize("head_major", [False, True])
@pytest.mark.parametrize("seed", range(4))
def test_model_keeps_tokens_and_counts(seed, head_major):
    rng = np.random.default_rng(seed)
    bs, NB, Hkv, D = 16, 80, 2, 4
    tables, lens, refs = ref.draw(rng, 5, 6, bs, NB, shared=2, spare=6)
    shape = (NB, Hkv, bs, D) if head_major else (NB, bs, Hkv, D)
    pool = rng.integers(0, 1 << 16, size=shape, dtype=np.uint16)
    want = [_tokens(pool, tables, lens, r, bs, head_major).copy() for r in range(5)]
    parents, children = [0, 3, 3, 0], [5, 6, 7, 8]
    assert ref.fork([pool], tables, lens, refs, parents, children, bs, head_major) == set()
    assert np.array_equal(refs, ref.counts(tables, lens, NB, bs))
    for p, c in zip(parents, children):
        assert np.array_equal(_tokens(pool, tables, lens, c, bs, head_major), want[p])
        if lens[p] % bs:    # the partly filled block is the child's own
            assert refs[tables[c, lens[p] // bs]] == 1
    assert ref.free(tables, lens, refs, [3, 5, -1], bs) == set()
    assert np.array_equal(refs, ref.counts(tables, lens, NB, bs))
    codes, remap, n = ref.compact([pool], tables, lens, refs, bs)
    assert codes == set() and np.array_equal(refs, ref.counts(tables, lens, NB, bs))
    assert sorted(np.nonzero(refs)[0]) == list(range(1, n + 1))
    assert sorted(remap[remap > 0]) == list(range(1, n + 1))
    for r, src in ((0, 0), (1, 1), (2, 2), (4, 4), (6, 3), (7, 3), (8, 0)):
        assert np.array_equal(_tokens(pool, tables, lens, r, bs, head_major), want[src])


# -- refusals ------------------------------------------------------------------------

_keep = (ctypes.c_void_p * 2)(16, 32)
_bad = (ctypes.c_void_p * 2)(16, 24)
_null = (ctypes.c_void_p * 2)(16, None)
POOLS, MISALIGNED, WITH_NULL = (ctypes.addressof(x) for x in (_keep, _bad, _null))

POOL_CASES = [
    (dict(D=64), pa.PA_ERR_UNSUPPORTED),
    (dict(bs=8), pa.PA_ERR_UNSUPPORTED),
    (dict(bs=48), pa.PA_ERR_UNSUPPORTED),
    (dict(bs=512), pa.PA_ERR_UNSUPPORTED),
    (dict(NB=1 << 31), pa.PA_ERR_UNSUPPORTED),
    (dict(Hkv=65536), pa.PA_ERR_UNSUPPORTED),
    (dict(Hkv=0), pa.PA_ERR_INVALID_ARG),
    (dict(NB=0), pa.PA_ERR_INVALID_ARG),
    (dict(NB=-1), pa.PA_ERR_INVALID_ARG),
    (dict(nc=-1), pa.PA_ERR_INVALID_ARG),
    (dict(caches=None), pa.PA_ERR_INVALID_ARG),
    (dict(caches=MISALIGNED), pa.PA_ERR_INVALID_ARG),
    (dict(caches=WITH_NULL), pa.PA_ERR_INVALID_ARG),
]
WS_CASES = [(dict(ws=None), pa.PA_ERR_WORKSPACE), (dict(ws=24), pa.PA_ERR_WORKSPACE),
            (dict(wsb=16), pa.PA_ERR_WORKSPACE)]


@pytest.mark.parametrize("over,want", POOL_CASES + [
    (dict(n=-1), pa.PA_ERR_INVALID_ARG),
    (dict(pairs=None), pa.PA_ERR_INVALID_ARG),
    (dict(pairs=20), pa.PA_ERR_INVALID_ARG),            # not 8-byte aligned
    (dict(n=0, pairs=None), pa.PA_OK),
    (dict(nc=0, caches=None), pa.PA_OK),
])
def test_copy_host_checks(pa_lib, over, want):
    a = dict(caches=POOLS, nc=2, pairs=16, n=3, Hkv=8, D=128, bs=16, NB=10)
    a.update(over)
    assert pa_lib.pa_copy_blocks(a["caches"], a["nc"], a["pairs"], a["n"], a["Hkv"], a["D"],
                                 a["bs"], a["NB"], None) == want


@pytest.mark.parametrize("over,want", POOL_CASES + WS_CASES + [
    (dict(n=-1), pa.PA_ERR_INVALID_ARG),
    (dict(n=5), pa.PA_ERR_INVALID_ARG),                 # more forks than rows
    (dict(R=-1, n=0), pa.PA_ERR_INVALID_ARG),
    (dict(mb=-1), pa.PA_ERR_INVALID_ARG),
    (dict(mb=0), pa.PA_ERR_INVALID_ARG),
    (dict(layout=2), pa.PA_ERR_INVALID_ARG),
    (dict(bt=None), pa.PA_ERR_INVALID_ARG),
    (dict(cl=None), pa.PA_ERR_INVALID_ARG),
    (dict(refs=None), pa.PA_ERR_INVALID_ARG),
    (dict(par=None), pa.PA_ERR_INVALID_ARG),
    (dict(ch=None), pa.PA_ERR_INVALID_ARG),
    (dict(n=0, bt=None, par=None, ws=None), pa.PA_OK),
])
def test_fork_host_checks(pa_lib, over, want):
    a = dict(caches=POOLS, nc=2, bt=16, mb=4, cl=16, R=4, refs=16, par=16, ch=16, n=2, Hkv=8, D=128,
             bs=16, NB=10, layout=0, ws=16, wsb=1 << 20)
    a.update(over)
    assert pa_lib.pa_fork_blocks(a["caches"], a["nc"], a["bt"], a["mb"], a["cl"], a["R"], a["refs"],
                                 a["par"], a["ch"], a["n"], a["Hkv"], a["D"], a["bs"], a["NB"],
                                 a["layout"], a["ws"], a["wsb"], None) == want


@pytest.mark.parametrize("over,want", [
    (dict(bs=20), pa.PA_ERR_UNSUPPORTED),
    (dict(NB=1 << 31), pa.PA_ERR_UNSUPPORTED),
    (dict(NB=0), pa.PA_ERR_INVALID_ARG),
    (dict(n=-1), pa.PA_ERR_INVALID_ARG),
    (dict(R=-1), pa.PA_ERR_INVALID_ARG),
    (dict(mb=0), pa.PA_ERR_INVALID_ARG),
    (dict(bt=None), pa.PA_ERR_INVALID_ARG),
    (dict(cl=None), pa.PA_ERR_INVALID_ARG),
    (dict(refs=None), pa.PA_ERR_INVALID_ARG),
    (dict(rows=None), pa.PA_ERR_INVALID_ARG),
    (dict(n=0, rows=None, bt=None), pa.PA_OK),
])
def test_free_host_checks(pa_lib, over, want):
    a = dict(bt=16, mb=4, cl=16, R=4, refs=16, rows=16, n=2, bs=16, NB=10)
    a.update(over)
    assert pa_lib.pa_free_blocks(a["bt"], a["mb"], a["cl"], a["R"], a["refs"], a["rows"], a["n"],
                                 a["bs"], a["NB"], None) == want


@pytest.mark.parametrize("over,want", POOL_CASES + WS_CASES + [
    (dict(R=-1), pa.PA_ERR_INVALID_ARG),
    (dict(mb=-1), pa.PA_ERR_INVALID_ARG),
    (dict(mb=0), pa.PA_ERR_INVALID_ARG),
    (dict(bt=None), pa.PA_ERR_INVALID_ARG),
    (dict(cl=None), pa.PA_ERR_INVALID_ARG),
    (dict(refs=None), pa.PA_ERR_INVALID_ARG),
    (dict(remap=None), pa.PA_ERR_INVALID_ARG),
    (dict(live=None), pa.PA_ERR_INVALID_ARG),
])
def test_compact_host_checks(pa_lib, over, want):
    a = dict(caches=POOLS, nc=2, bt=16, mb=4, cl=16, R=4, refs=16, remap=16, live=16, Hkv=8, D=128,
             bs=16, NB=10, ws=16, wsb=1 << 20)
    a.update(over)
    if a["wsb"] == 16:
        a["NB"] = 1 << 20
    assert pa_lib.pa_compact_blocks(a["caches"], a["nc"], a["bt"], a["mb"], a["cl"], a["R"],
                                    a["refs"], a["remap"], a["live"], a["Hkv"], a["D"], a["bs"],
                                    a["NB"], a["ws"], a["wsb"], None) == want


def test_workspace_size(pa_lib):
    assert pa_lib.pa_blocks_workspace_size(-1, 10) == 0
    assert pa_lib.pa_blocks_workspace_size(4, 0) == 0
    assert pa_lib.pa_blocks_workspace_size(4, 1 << 31) == 0
    # a record, a claim and a block per fork; a move per two blocks
    assert pa_lib.pa_blocks_workspace_size(100, 2) >= 100 * 24
    assert pa_lib.pa_blocks_workspace_size(0, 1 << 20) >= (1 << 19) * 8


def test_binding_refuses_cpu_tensors(pa_lib):
    c = torch.zeros(4, 16, 8, 128, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        pa.CachePools([c, c.clone()])
    with pytest.raises(ValueError):
        pa.CachePools([])
    with pytest.raises(ValueError):
        pa.free_blocks(i.view(4, 1), i, i, i, 16)


# -- header and ranges ----------------------------------------------------------------

def _declared():
    with open(os.path.join(ROOT, "include", "pagedattn", "blocks.h")) as fh:
        return set(re.findall(r"PA_API\s+[\w\s\*]+?\b(pa_\w+)\s*\(", fh.read()))


def test_every_header_entry_point_is_exported_and_bound(pa_lib):
    assert glob.glob(os.path.join(ROOT, "include", "pagedattn", "*.h"))
    assert {"pa_copy_blocks", "pa_fork_blocks", "pa_free_blocks", "pa_compact_blocks"} <= _declared()
    for n in _declared():
        assert hasattr(pa_lib, n) and n in pa.SIGNATURES, n


C_PROGRAM = """
#include <stdio.h>
#include "pagedattn/blocks.h"
int main(void)
{
    pa_status_t (*copy)(void *const *, int, const int32_t *, int64_t, int, int, int, int64_t,
                        void *) = pa_copy_blocks;
    size_t (*size)(int, int64_t) = pa_blocks_workspace_size;
    pa_status_t (*fork)(void *const *, int, int32_t *, int, int32_t *, int, int32_t *,
                        const int32_t *, const int32_t *, int, int, int, int, int64_t, pa_layout_t,
                        void *, size_t, void *) = pa_fork_blocks;
    pa_status_t (*release)(int32_t *, int, int32_t *, int, int32_t *, const int32_t *, int, int,
                           int64_t, void *) = pa_free_blocks;
    pa_status_t (*compact)(void *const *, int, int32_t *, int, const int32_t *, int, int32_t *,
                           int32_t *, int32_t *, int, int, int, int64_t, void *, size_t, void *) =
        pa_compact_blocks;
    int bad = 0;
    bad += copy(NULL, 0, NULL, 0, 8, 128, 16, 10, NULL) != PA_OK;
    bad += size(4, 0) != 0;
    bad += fork(NULL, 0, NULL, 4, NULL, 4, NULL, NULL, NULL, 0, 8, 128, 16, 10,
                PA_LAYOUT_TOKEN_MAJOR, NULL, 0, NULL) != PA_OK;
    bad += release(NULL, 4, NULL, 4, NULL, NULL, 0, 16, 10, NULL) != PA_OK;
    bad += compact(NULL, 0, NULL, 4, NULL, 0, NULL, NULL, NULL, 8, 128, 16, 10, NULL, 0, NULL) !=
           PA_ERR_INVALID_ARG;
    printf("ok %d\\n", bad);
    return bad;
}
"""


def test_header_from_c99(pa_lib, tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not found")
    assert set(re.findall(r"=\s*(pa_\w+);", C_PROGRAM)) == _declared()
    src, exe = tmp_path / "blocks.c", tmp_path / "blocks"
    src.write_text(C_PROGRAM)
    lib_dir = os.path.dirname(build.LIB_PATH)
    subprocess.run([gcc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I",
                    os.path.join(ROOT, "include"), str(src), "-o", str(exe), "-L", lib_dir,
                    "-lpagedattn", "-Wl,-rpath," + lib_dir], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120,
                       env=dict(os.environ, CUDA_VISIBLE_DEVICES=""))
    assert r.returncode == 0 and r.stdout.strip() == "ok 0", r.stdout + r.stderr


CALLS = [
    ("pa_copy_blocks", "L.pa_copy_blocks(None, 0, None, 0, 8, 128, 16, 10, None)"),
    ("pa_fork_blocks", "L.pa_fork_blocks(None, 0, None, 4, None, 4, None, None, None, 0, 8, 128, 16, 10, 1, "
                       "None, 0, None)"),
    ("pa_free_blocks", "L.pa_free_blocks(None, 4, None, 4, None, None, 0, 16, 10, None)"),
    ("pa_compact_blocks", "L.pa_compact_blocks(None, 0, None, 4, None, 0, 16, 16, 16, 8, 64, 16, 10, 16, 99, None)"),
]


def test_ranges(recorder, tmp_path):  # noqa: F811
    log = tmp_path / "events.txt"
    script = (f"import sys\nsys.path.insert(0, {ROOT!r})\n"
              "from paged_kv_cache_255_gb300 import pagedattn as pa\nL = pa.lib()\n"
              f"print([{', '.join(c for _, c in CALLS)}])")
    env = dict(os.environ, NVTX_INJECTION64_PATH=recorder, NVTX_RECORD_PATH=str(log),
               CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, "-c", script], env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "[0, 0, 0, 2]", r.stdout + r.stderr
    events = [ln.split(" ", 2) for ln in log.read_text().splitlines()]
    ours = [e for e in events if len(e) > 1 and e[1] == "libpagedattn"][1:]
    want = []
    for name, _ in CALLS:
        want += [["push", "libpagedattn", name], ["pop", "libpagedattn"]]
    assert ours == want
