"""What the host decides for a cache of few bits, drafted tokens and a loss's gradient, and the
searches that the cache's kernels make with a caller's offsets and tables, built
for the CPU under AddressSanitizer and UndefinedBehaviorSanitizer:
tests/sanitize/lm_cache_driver.cpp, one check per test."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SAN = ["-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer",
       "-g", "-O1"]


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("g++ not available")
    exe = tmp_path_factory.mktemp("lm_cache") / "driver"
    src = os.path.join(ROOT, "byte_level_bpe_pretokenize_amd", "csrc_lm")
    # (the header of the layouts includes the HIP runtime's; no HIP call is made)
    subprocess.run(["g++", "-std=c++17", *SAN, "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include",
                    "-I", os.path.join(ROOT, "include"), "-I", src,
                    os.path.join(ROOT, "tests", "sanitize", "lm_cache_driver.cpp"),
                    os.path.join(src, "lm_layout.cpp"), "-o", str(exe)], check=True)
    return str(exe)


@pytest.mark.parametrize("check", ["shape", "refusals", "limit", "request", "slot", "gradient", "regions"])
def test_layout(driver, check):
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=1:verify_asan_link_order=0",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([driver, check], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert "passed" in r.stdout
