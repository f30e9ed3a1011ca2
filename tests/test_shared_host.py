"""Decode over shared prefixes, CPU side: refusals before any CUDA call, the
header from strict C99, the NVTX range."""
import os
import re
import shutil
import subprocess
import sys

import pytest
import torch

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
    (dict(G=-1), pa.PA_ERR_INVALID_ARG),
    (dict(G=4097), pa.PA_ERR_UNSUPPORTED),
    (dict(S=65536), pa.PA_ERR_UNSUPPORTED),
    (dict(Hq=65536, Hkv=65536), pa.PA_ERR_UNSUPPORTED),
    (dict(q=None), pa.PA_ERR_INVALID_ARG),
    (dict(cl=None), pa.PA_ERR_INVALID_ARG),
    (dict(gs=None), pa.PA_ERR_INVALID_ARG),
    (dict(pb=None), pa.PA_ERR_INVALID_ARG),
    (dict(out=24), pa.PA_ERR_INVALID_ARG),
    (dict(v=8), pa.PA_ERR_INVALID_ARG),
    (dict(layout=5), pa.PA_ERR_INVALID_ARG),
    (dict(scale=float("inf")), pa.PA_ERR_INVALID_ARG),
    (dict(mb=0), pa.PA_ERR_INVALID_ARG),
    (dict(NB=0), pa.PA_ERR_INVALID_ARG),
    (dict(NB=1 << 27), pa.PA_ERR_UNSUPPORTED),
    (dict(S=0, q=None, gs=None), pa.PA_OK),
    (dict(G=0, gs=None, pb=None), pa.PA_OK),
])
def test_host_checks(pa_lib, over, want):
    a = dict(q=16, k=16, v=16, bt=16, mb=4, cl=16, gs=16, pb=16, G=2, scale=0.1, out=16, S=2, Hq=16, Hkv=8,
             D=128, bs=16, NB=10, layout=0, ws=16, wsb=1 << 28)
    a.update(over)
    assert pa_lib.pa_decode_shared(a["q"], a["k"], a["v"], a["bt"], a["mb"], a["cl"], a["gs"], a["pb"], a["G"],
                                   a["scale"], a["out"], a["S"], a["Hq"], a["Hkv"], a["D"], a["bs"], a["NB"],
                                   a["layout"], a["ws"], a["wsb"], None) == want


def test_workspace_size_rejects(pa_lib):
    for args in ((-1, 1, 16, 8, 128), (4, -1, 16, 8, 128), (4, 4097, 16, 8, 128), (4, 1, 12, 8, 128),
                 (4, 1, 16, 8, 64), (4, 1, 34, 2, 128), (65536, 1, 16, 8, 128), (4, 1, 65536, 65536, 128)):
        assert pa_lib.pa_decode_shared_workspace_size(*args) == 0


def test_binding_refuses_cpu_tensors(pa_lib):
    q = torch.zeros(2, 16, 128, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        pa.decode_shared(q, q, q, i.view(2, 1), i, i, i[:1], 0.1)


C_PROGRAM = """
#include <stdio.h>
#include "pagedattn/decode_shared.h"
int main(void)
{
    size_t (*size)(int, int, int, int, int) = pa_decode_shared_workspace_size;
    pa_status_t (*shared)(const void *, const void *, const void *, const int32_t *, int,
                          const int32_t *, const int32_t *, const int32_t *, int, float, void *,
                          int, int, int, int, int, int64_t, pa_layout_t, void *, size_t, void *) =
        pa_decode_shared;
    int bad = 0;
    bad += size(4, 1, 12, 8, 128) != 0;
    bad += shared(NULL, NULL, NULL, NULL, 4, NULL, NULL, NULL, 1, 0.1f, NULL, 0, 16, 8, 128, 16, 10,
                  PA_LAYOUT_HEAD_MAJOR, NULL, 0, NULL) != PA_OK;
    printf("ok %d\\n", bad);
    return bad;
}
"""


def test_header_from_c99(pa_lib, tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not found")
    with open(os.path.join(ROOT, "include", "pagedattn", "decode_shared.h")) as fh:
        declared = set(re.findall(r"PA_API\s+[\w\s\*]+?\b(pa_\w+)\s*\(", fh.read()))
    assert set(re.findall(r"=\s*(pa_\w+);", C_PROGRAM)) == declared | {"pa_decode_shared"}
    for n in declared:
        assert hasattr(pa_lib, n) and n in pa.SIGNATURES, n
    src, exe = tmp_path / "shared.c", tmp_path / "shared"
    src.write_text(C_PROGRAM)
    lib_dir = os.path.dirname(build.LIB_PATH)
    subprocess.run([gcc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I",
                    os.path.join(ROOT, "include"), str(src), "-o", str(exe), "-L", lib_dir,
                    "-lpagedattn", "-Wl,-rpath," + lib_dir], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120,
                       env=dict(os.environ, CUDA_VISIBLE_DEVICES=""))
    assert r.returncode == 0 and r.stdout.strip() == "ok 0", r.stdout + r.stderr


def test_range(recorder, tmp_path):  # noqa: F811
    log = tmp_path / "events.txt"
    script = (f"import sys\nsys.path.insert(0, {ROOT!r})\n"
              "from paged_kv_cache_255_gb300 import pagedattn as pa\n"
              "print(pa.lib().pa_decode_shared(16, 16, 16, 16, 4, 16, 16, 16, 2, 0.1, 16, 2, 16, 8, 64, 16, 10, "
              "0, 16, 99, None))")
    env = dict(os.environ, NVTX_INJECTION64_PATH=recorder, NVTX_RECORD_PATH=str(log), CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, "-c", script], env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "2", r.stdout + r.stderr
    events = [ln.split(" ", 2) for ln in log.read_text().splitlines()]
    ours = [e for e in events if len(e) > 1 and e[1] == "libpagedattn"][1:]
    assert ours == [["push", "libpagedattn", "pa_decode_shared"], ["pop", "libpagedattn"]]
