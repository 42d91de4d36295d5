"""How a selective scan cuts packed sequences of unequal lengths
(mamba_ssd_chunked_fwd_amd/csrc/ssd_selective_plan.h), in plain C++ under AddressSanitizer and
UndefinedBehaviorSanitizer (tests/sanitize/selective_plan_driver.cpp): every token in one run,
one long sequence cut alike however many short ones lie beside it, and no sequence whole that
would outlast the rest.  No GPU."""
import os
import subprocess

from test_sanitize_host import ROOT, SAN, pytestmark  # noqa: F401


def test_unequal_sequences_under_sanitizers(tmp_path):
    exe, csrc = str(tmp_path / "driver"), os.path.join(ROOT, "mamba_ssd_chunked_fwd_amd", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=address,undefined",
                    "-fno-sanitize-recover=undefined", "-fno-omit-frame-pointer", "-g",
                    "-I", os.path.join(ROOT, "include"), "-I", csrc,
                    os.path.join(SAN, "selective_plan_driver.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "all checks passed" in r.stdout
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr
