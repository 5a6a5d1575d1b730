"""The appended codes' short cut around a division on the CPU
(csrc/append_quick.h): wherever it is taken it gives the division's code, with
the reciprocal as far off as the hardware's may be."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_short_cut_gives_the_divisions_codes(tmp_path):
    exe = str(tmp_path / "driver")
    r = subprocess.run(["g++", "-std=c++17", "-O2", "-ffp-contract=off", "-Wall", "-Werror",
                        "-I", os.path.join(ROOT, "bit_affine_quantized_amd", "csrc"),
                        os.path.join(ROOT, "tests", "sanitize", "append_quick_driver.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr
