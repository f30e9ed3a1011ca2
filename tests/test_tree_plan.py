"""The counts of decode over trees, on the CPU: how it reads starts and lengths and what it
counts in 32 bits are compiled from their header and gone through with arrays of every kind."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run(tmp_path, program):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not found")
    src, exe = tmp_path / "plan.cpp", tmp_path / "plan"
    src.write_text(program)
    subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-I",
                    os.path.join(ROOT, "paged_kv_cache_255_gb300", "csrc"), str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    return r.returncode, r.stdout.strip(), r.stdout + r.stderr


COUNTS = r"""
#include <cstdio>
#include <random>
#include <vector>
#include "tree_plan.h"
int main()
{
    std::mt19937_64 rng(3);
    long taken = 0, bad = 0, fallen_past = 0;
    auto log_up_to = [&](int64_t most) {        // 0 .. most, over its logarithm
        const int64_t top = (int64_t)1 << rng() % 32;
        return (int64_t)(rng() % (uint64_t)((most < top ? most : top) + 1));
    };
    for (int k = 0; k < 200000; ++k) {
        const int G = 1 << rng() % 5, Hkv = 1 + (int)log_up_to(64), S = 1 + (int)log_up_to(300);
        const int T = (int)log_up_to(INT32_MAX / (G * Hkv));
        const int64_t max_len = 16 + log_up_to(INT32_MAX - 127 - 16);
        if (!pa::tree_places_fit(T, G, S, max_len, Hkv)) continue;
        ++taken;
        // starts: ascending, any numbers, or all rows over and over; lengths: the longest, any numbers
        const int kind = (int)(rng() % 3);
        std::vector<int> start(S + 1);
        int64_t at = 0;
        for (int s = 0; s <= S; ++s) {
            if (kind == 0) at += log_up_to(T), start[s] = (int)(at < INT32_MAX ? at : INT32_MAX);
            else start[s] = kind == 1 ? (int)rng() : (s % 2 ? T : 0);
        }
        bool falls = false;
        int64_t sum = 0;
        for (int s = 0; s < S; ++s) {
            const int len = rng() % 2 ? INT32_MAX : (int)rng();
            const pa::TreeSeq q = pa::tree_seq(start[s], start[s + 1], len, T, max_len, G);
            falls |= q.n < 0;
            bad += q.q0 < 0 || q.q0 > T || q.n > T - q.q0 || q.L < 0 || q.L > max_len || q.nt < 1;
            bad += q.n <= 0 ? q.pairs != 0 : (int64_t)q.pairs * 256 < (int64_t)q.n * G;
            const int64_t places = (int64_t)q.pairs * Hkv * (q.nt + pa::kTreeUnitPlaces);
            bad += places != pa::tree_seq_places(q, Hkv);
            sum += places;
        }
        // what the kernel counts in 32 bits without counting again
        bad += !falls && sum > INT32_MAX;
        fallen_past += falls && sum > INT32_MAX;
    }
    std::printf("taken %d bad %ld past %d\n", taken > 1000, bad, fallen_past > 0);
    return bad != 0;
}
"""


def test_places_fit_unless_the_starts_fall(tmp_path):
    rc, out, log = run(tmp_path, COUNTS)
    assert rc == 0 and out == "taken 1 bad 0 past 1", log


LANES = r"""
#include <cstdio>
#include "tree_plan.h"
int main()
{
    long bad = 0, side = 0;
    for (int workers = 1; workers <= 255; ++workers)
        for (int pairs = 1; pairs <= 600; ++pairs) {
            const int lanes = pa::tree_lanes(pairs, pairs, workers);
            side += lanes > 1;
            bad += lanes != 1 && lanes != pairs;                // a unit of each sequence and head to a lane
            const int busy = workers / lanes * lanes;
            bad += busy < 1 || (workers - busy) * 8 > workers;  // CTAs that no share is for
            bad += pairs > 1 && pa::tree_lanes(pairs, pairs - 1, workers) != 1;
        }
    bad += pa::tree_lanes(0, INT_MAX, 152) != 1;                // no units at all
    const int good[] = {2, 3, 8, 17, 76, 152};
    for (int pairs : good) bad += pa::tree_lanes(pairs, pairs, 152) != pairs;
    std::printf("side %d bad %ld\n", side > 0, bad);
    return bad != 0;
}
"""


def test_lanes_leave_few_ctas_without_a_share(tmp_path):
    rc, out, log = run(tmp_path, LANES)
    assert rc == 0 and out == "side 1 bad 0", log
