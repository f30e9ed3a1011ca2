"""Records of decode over shared prefixes, on the CPU: the checks that the combine
makes are compiled from its header and gone through with every record of a
small launch. Whatever a record holds, an accepted one leads only to slots of
the workspace, and every record that the kernels write is accepted."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <climits>
#include <cstdio>
#include "shared_records.h"
struct R { int x, y, z; };
static bool inside(int64_t slot, int workers) { return slot >= 0 && slot < 2 * workers; }
int main()
{
    const int odd[] = {INT_MIN, INT_MIN + 1, -1000, 1000, INT_MAX - 1, INT_MAX};
    long accepted = 0, bad = 0;
    for (int workers = 1; workers <= 5; ++workers) {
        int v[32], n = 0;
        for (int i = -5; i <= 2 * workers + 4; ++i) v[n++] = i;
        for (int o : odd) v[n++] = o;
        for (int i = 0; i < n; ++i)
            for (int j = 0; j < n; ++j)
                for (int k = 0; k < n; ++k) {
                    const R r{v[i], v[j], v[k]};
                    for (int done = 0; done < 2; ++done) {
                        if (!pa::unit_record_ok(r, workers, done != 0)) continue;
                        ++accepted;
                        if (r.x == pa::kRecordWhole || (done && r.x == pa::kRecordDone)) continue;
                        for (int at = 0; at <= r.y - r.z; ++at)
                            bad += !inside(pa::record_slot(r.x, at, 2), workers);
                    }
                    if (pa::prefix_record_ok(r, workers)) {
                        ++accepted;
                        for (int at = 0; at < r.y; ++at)
                            bad += !inside(pa::record_slot(r.x, at, r.z), workers);
                    }
                }
        // what the kernels write: a unit that begins as a share's first or later piece and ends
        // in the same share or a later one; a prefix unit over `parts` shares of a lane
        for (int w = 0; w < workers; ++w) {
            bad += !pa::unit_record_ok(R{pa::kRecordWhole, w, w}, workers, false);
            bad += !pa::unit_record_ok(R{pa::kRecordWhole, w, w}, workers, true);
            bad += !pa::unit_record_ok(R{pa::kRecordDone, w, w}, workers, true);
            bad += pa::unit_record_ok(R{pa::kRecordDone, w, w}, workers, false);
            for (int piece = 0; piece < 2; ++piece) {
                for (int last = w; last < workers; ++last)
                    bad += !pa::unit_record_ok(R{2 * w + piece, last, w}, workers, false);
                for (int lanes = 1; lanes <= workers; ++lanes)
                    for (int parts = 1; w + (parts - 1) * lanes < workers; ++parts)
                        bad += !pa::prefix_record_ok(R{2 * w + piece, parts, 2 * lanes}, workers);
            }
        }
        bad += !pa::prefix_record_ok(R{0, 0, 0}, workers);
    }
    std::printf("accepted %d bad %ld\n", accepted > 0, bad);
    return bad != 0;
}
"""


def test_no_record_leads_out_of_the_workspace(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not found")
    src, exe = tmp_path / "records.cpp", tmp_path / "records"
    src.write_text(PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-I",
                    os.path.join(ROOT, "paged_kv_cache_255_gb300", "csrc"), str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == "accepted 1 bad 0", r.stdout + r.stderr
