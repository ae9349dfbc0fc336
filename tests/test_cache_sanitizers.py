"""The host layer of the key/value cache under AddressSanitizer and UndefinedBehaviorSanitizer, on the
CPU: `sanitize/cache_driver.cpp` calls every entry point with caches and descriptors drawn from
lists of usual and extreme values; the stub launchers abort where a bad one gets through."""
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "bit_floating_point_amd", "csrc")
CLANG = "/opt/rocm/llvm/bin/clang++"


@pytest.mark.skipif(not os.path.exists(CLANG), reason="ROCm clang++ not installed")
def test_cache_host_under_sanitizers(tmp_path):
    exe = str(tmp_path / "cache_san")
    # the 4-bit launchers that fp4_api.cpp names are never reached
    r = subprocess.run([CLANG, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                        "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", os.path.join(CSRC, "fp4_api.cpp"),
                        os.path.join(CSRC, "cache_api.cpp"), os.path.join(HERE, "sanitize", "cache_driver.cpp"), "-o", exe,
                        "-Wl,--unresolved-symbols=ignore-all", "-rtlib=compiler-rt", "-unwindlib=libgcc"],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=dict(os.environ, UBSAN_OPTIONS="print_stacktrace=1"))
    assert r.returncode == 0 and "Sanitizer" not in r.stderr and "runtime error" not in r.stderr, r.stdout[-1000:] + r.stderr[-3000:]
    print(r.stdout)
