"""The order in which workgroups take tiles (tile.h), run on the host: every tile is
taken by one workgroup, however many more there are, and has a place of its own
(no GPU needed)."""
import os
import subprocess

import pytest

from test_lib_host_sanitized import HIPCC

PROGRAM = r"""
#include <stdio.h>
#include <vector>
#include "tile.h"
using namespace vs::tile;
int main() {
    const int64_t totals[] = {1, 2, 7, 8, 9, 15, 16, 17, 63, 64, 65, 100, 1216, 5000, 19200, 19203};
    for (int64_t total : totals)
        for (int64_t more = 0; more <= 40; ++more) {
            std::vector<int> taken(total, 0);
            for (int64_t id = 0; id < (total + more + 7) / 8 * 8; ++id) {
                int64_t at = -1;
                if (!xcd_tile(id, total, at)) continue;
                if (at < 0 || at >= total) return printf("%ld: %ld\n", (long)total, (long)at), 1;
                ++taken[at];
            }
            for (int64_t t = 0; t < total; ++t)
                if (taken[t] != 1)
                    return printf("%ld + %ld: tile %ld %d times\n", (long)total, (long)more, (long)t,
                                  taken[t]), 1;
        }
    for (int64_t rows : {1, 2, 5, 64, 300})
        for (int64_t cols : {1, 7, 8, 9, 16, 31}) {
            std::vector<int> taken(rows * cols, 0);
            for (int64_t t = 0; t < rows * cols; ++t) {
                const Place p = place(t, rows, cols);
                if (p.row < 0 || p.row >= rows || p.col < 0 || p.col >= cols) return printf("place\n"), 1;
                ++taken[p.row * cols + p.col];
            }
            for (int n : taken)
                if (n != 1) return printf("%ld x %ld\n", (long)rows, (long)cols), 1;
        }
    printf("taken once\n");
    return 0;
}
"""


@pytest.mark.timeout(300)
def test_every_tile_is_taken_once(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc is not installed")
    from farthest_vector_search_amd import build as b
    src, exe = tmp_path / "order.hip", str(tmp_path / "order")
    src.write_text(PROGRAM)
    r = subprocess.run([HIPCC, *b.FLAGS, "-O1", str(src), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout == "taken once\n", r.stdout
