"""Lists of kept tokens, on the CPU: the rule by which keep_kernel takes an entry is compiled
from its header and gone through with every list of a small draft and long random ones. What
stands behind a list's end may be anything: no entry that the rule takes, before or behind
the end, leads to a place outside the draft, and up to the end the rule is the path's."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <climits>
#include <cstdio>
#include <random>
#include <vector>
#include "keep_path.h"
static long outside = 0, wrong = 0, taken = 0;
static void look(const std::vector<int> &list, int n)
{
    const int m = (int)list.size();
    // the path and how it ends, one entry after the other
    int count = 0;
    while (count < m && list[count] >= 0 && list[count] < n && (count == 0 || list[count] > list[count - 1])) ++count;
    const bool bad_end = count < m && list[count] != -1;
    int first = m;
    bool first_bad = false;
    for (int i = 0; i < m; ++i) {       // as the kernel's threads: each its entry and the one before
        bool bad;
        const bool ok = pa::path_continues(list[i], i ? list[i - 1] : INT_MIN, i, n, bad);
        if (!ok && first == m) {
            first = i;
            first_bad = bad;
        }
        if (!ok) continue;
        ++taken;
        // the token of place i and of node list[i], from the draft's first: both inside it
        outside += i >= n || list[i] < 0 || list[i] >= n;
    }
    wrong += first != count || first_bad != bad_end;
}
int main()
{
    // every list of up to 5 of these entries
    const int kinds[] = {-1, 0, 1, 2, 3, -7, INT_MAX, INT_MIN};
    for (int n = 1; n <= 4; ++n)
        for (int m = 1; m <= 5; ++m) {
            std::vector<int> at(m, 0), list(m);
            for (bool more = true; more;) {
                for (int i = 0; i < m; ++i) list[i] = kinds[at[i]];
                look(list, n);
                more = false;
                for (int i = 0; i < m && !more; ++i) {
                    at[i] = (at[i] + 1) % 8;
                    more = at[i] != 0;
                }
            }
        }
    // long lists with what earlier drafts left behind the end
    std::mt19937 rng(5);
    for (int k = 0; k < 3000; ++k) {
        const int n = 1 + rng() % 40, m = 1 + rng() % 1024;
        std::vector<int> list(m);
        for (int i = 0; i < m; ++i) list[i] = k % 2 ? (int)(rng() % (n + 2)) - 1 : i % (n + 1) - 1;
        look(list, n);
    }
    std::printf("taken %d outside %ld wrong %ld\n", taken > 0, outside, wrong);
    return outside != 0 || wrong != 0;
}
"""


def test_no_entry_leads_out_of_the_draft(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not found")
    src, exe = tmp_path / "path.cpp", tmp_path / "path"
    src.write_text(PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-I",
                    os.path.join(ROOT, "paged_kv_cache_255_gb300", "csrc"), str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == "taken 1 outside 0 wrong 0", r.stdout + r.stderr
