"""The size query of the matrices' gradient over the whole range of its arguments: the
host side of units.hip alone, built to trap on undefined behaviour and linked without
the HIP runtime (no GPU needed)."""
import os
import shutil
import subprocess

import pytest

from test_lib_host_sanitized import HIPCC

PROGRAM = r"""
#include <stdint.h>
#include <stdio.h>
extern "C" {  // kernels are registered with nobody, and none is launched
void **__hipRegisterFatBinary(const void *) { return nullptr; }
void __hipRegisterFunction(void **, const void *, char *, const char *, unsigned, void *, void *, void *, void *, int *) {}
void __hipRegisterVar(void **, void *, char *, char *, int, size_t, int, int) {}
void __hipUnregisterFatBinary(void **) {}
}
namespace vs { size_t unit_mats_workspace(int64_t m, int64_t G, int32_t cols, int32_t d); }
int main() {
    const int64_t rows[] = {0, 1, 127, 1024, 4096, 70000, 2147483647}, units[] = {1, 2, 64, 511, 512, 100000, 2147483646};
    const int32_t sizes[] = {1, 2, 63, 64, 65, 512, 4097, 1 << 20};
    long some = 0;
    for (int64_t m : rows)
        for (int64_t G : units)
            for (int32_t c : sizes)
                for (int32_t d : sizes) {
                    const size_t n = vs::unit_mats_workspace(m, G, c, d), one = (size_t)G * c * d * 4;
                    if (!n) continue;
                    ++some;
                    // 2 .. 32 arrays of matrices, of fewer than 512 tiles of 128 x 128
                    if ((double)G * c * d > 512.0 * 128 * 128 || n % one || n / one < 2 || n / one > 32 || m / G < 256)
                        return printf("%ld %ld %d %d: %zu\n", (long)m, (long)G, c, d, n), 1;
                }
    printf("sizes hold %d\n", some > 100);
    return 0;
}
"""


@pytest.mark.timeout(300)
def test_workspace_of_every_size(tmp_path):
    if not os.path.exists(HIPCC) or not shutil.which("g++"):
        pytest.skip("hipcc or g++ is not installed")
    from farthest_vector_search_amd import build as b
    src, obj, exe = tmp_path / "sizes.cpp", str(tmp_path / "units.o"), str(tmp_path / "sizes")
    src.write_text(PROGRAM)
    for cmd in ([HIPCC, *(f for f in b.FLAGS if f != "-O3"), "-O1", "--offload-host-only", "-Xarch_host",
                 "-fsanitize=undefined", "-Xarch_host", "-fsanitize-trap=undefined",
                 "-c", os.path.join(b.CSRC, "units.hip"), "-o", obj],
                ["g++", "-O1", str(src), obj, "-Wl,--unresolved-symbols=ignore-all", "-o", exe]):
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout == "sizes hold 1\n", (r.returncode, r.stdout, r.stderr)
