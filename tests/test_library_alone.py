"""The library needs the driver and the C and C++ libraries alone: a program can load it on a
machine without the toolkit or torch."""
import re
import shutil
import subprocess

import pytest

from paged_kv_cache_255_gb300 import build


def test_the_cuda_runtime_is_inside(pa_lib):
    readelf = shutil.which("readelf")
    if readelf is None:
        pytest.skip("readelf not found")
    r = subprocess.run([readelf, "-d", build.LIB_PATH], capture_output=True, text=True, check=True)
    needed = set(re.findall(r"\(NEEDED\).*\[(.+)\]", r.stdout))
    assert needed and not [n for n in needed if "cuda" in n.lower()], needed
    assert not re.search(r"\((RUNPATH|RPATH)\)", r.stdout), r.stdout        # no path of the building machine
