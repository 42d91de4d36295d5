"""The C ABI layer of the operators around a selective state space
(mamba_ssd_chunked_fwd_amd/csrc/ssd_selective_api.cpp) and the plan by which they cut packed
sequences (ssd_selective_plan.h) under AddressSanitizer and UndefinedBehaviorSanitizer, as
test_sanitize_host.py does for the SSD's: built with g++ against stand-in launchers
(tests/sanitize/selective_abi_driver.cpp).  No GPU."""
import os
import subprocess

from test_sanitize_host import ROOT, SAN, pytestmark  # noqa: F401


def test_selective_abi_layer_under_sanitizers(tmp_path):
    exe, csrc = str(tmp_path / "driver"), os.path.join(ROOT, "mamba_ssd_chunked_fwd_amd", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=address,undefined",
                    "-fno-sanitize-recover=undefined", "-fno-omit-frame-pointer", "-g",
                    "-I", os.path.join(ROOT, "include"), "-I", csrc,
                    os.path.join(SAN, "selective_abi_driver.cpp"),
                    os.path.join(csrc, "ssd_selective_api.cpp"), "-o", exe], check=True)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "all checks passed" in r.stdout
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr
