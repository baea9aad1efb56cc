"""The host code of the units' products, the row norm and the 8-bit tables under
AddressSanitizer and UndefinedBehaviorSanitizer (no GPU): api.hip is rebuilt with
the sanitizers on its host side, linked with the library's other objects, and the
refusals of test_row_products_host.py run against that build in a child process."""
import os
import subprocess
import sys

import pytest

from test_lib_host_sanitized import HIPCC, ROOT, _asan_runtime


@pytest.mark.timeout(900)
def test_row_products_clean_under_sanitizers(tmp_path):
    asan = _asan_runtime()
    if asan is None or not os.path.exists(HIPCC):
        pytest.skip("hipcc or clang's AddressSanitizer runtime is not installed")
    from farthest_vector_search_amd import build as b
    objs = [os.path.join(b.BUILD, os.path.splitext(s)[0] + ".o") for s in b.SOURCES if s != "api.hip"]
    if not all(os.path.exists(o) for o in objs):
        b.build(verbose=False)
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-omit-frame-pointer"]
    api_o, lib = str(tmp_path / "api.o"), str(tmp_path / "libvs_san.so")
    flags = [f for f in b.FLAGS if f != "-O3"] + ["-O1", "-g"]
    for cmd in ([HIPCC, *flags, *san, "-c", os.path.join(b.CSRC, "api.hip"), "-o", api_o],
                [HIPCC, f"--offload-arch={b.ARCH}", "-shared", "-fPIC", *san, "-o", lib, api_o,
                 *objs]):
        r = subprocess.run(cmd, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]
    child = (
        "import sys\n"
        f"sys.path[:0] = [{ROOT!r}, {os.path.join(ROOT, 'tests')!r}]\n"
        "import farthest_vector_search_amd as vs\n"
        f"vs.LIB_PATH = {lib!r}\n"
        "import pytest\n"
        "sys.exit(pytest.main(['-q', '-x', '-m', 'not gpu', '-p', 'no:cacheprovider',\n"
        f"    {os.path.join(ROOT, 'tests', 'test_row_products_host.py')!r}]))\n")
    env = dict(os.environ, LD_PRELOAD=asan,
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=1:halt_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([sys.executable, "-c", child], capture_output=True, text=True, env=env,
                       cwd=ROOT, timeout=600)
    assert r.returncode == 0, (r.stdout[-3000:], r.stderr[-3000:])
    assert " passed" in r.stdout
