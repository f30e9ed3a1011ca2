"""How a rotation's heads are shared among warps, on the CPU: compiled from its header and gone
through with sizes of every kind. Each slice has heads, all heads are in one, and items are
counted in 32 bits."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cstdio>
#include <random>
#include "rotary_split.h"
static long bad = 0, sliced = 0;
static void look(int64_t tokens, int rows, int sms)
{
    const pa::RotarySplit s = pa::rotary_split(tokens, rows, sms);
    sliced += s.slices > 1;
    bad += s.quads < 1 || s.slices < 1 || tokens * s.slices > INT32_MAX;
    bad += s.slices > 1 && tokens * s.slices >= 3 * 32 * sms;
    bad += (int64_t)s.slices * s.quads * 4 < rows;                  // heads that no slice has
    bad += (int64_t)(s.slices - 1) * s.quads * 4 >= rows;           // a slice without heads
}
int main()
{
    for (int rows = 1; rows <= 200; ++rows)
        for (int64_t tokens = 1; tokens <= 6000; ++tokens) look(tokens, rows, 152);
    std::mt19937_64 rng(2);
    for (int k = 0; k < 3000000; ++k) {
        const int64_t tokens = 1 + rng() % ((uint64_t)1 << rng() % 32);
        const int rows = 1 + (int)(rng() % ((uint64_t)1 << rng() % 22));
        look(tokens > INT32_MAX ? INT32_MAX : tokens, rows, 1 + (int)(rng() % 300));
    }
    look(INT32_MAX, 3 << 20, 1);
    look(INT32_MAX, 1, 152);
    std::printf("sliced %d bad %ld\n", sliced > 0, bad);
    return bad != 0;
}
"""


def test_every_slice_has_heads(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not found")
    src, exe = tmp_path / "split.cpp", tmp_path / "split"
    src.write_text(PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-I",
                    os.path.join(ROOT, "paged_kv_cache_255_gb300", "csrc"), str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "sliced 1 bad 0", r.stdout + r.stderr
