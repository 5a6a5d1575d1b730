"""How attention's lengths are cut into chunks (csrc/kv_chunks.h), on the CPU:
the chunks cover every length and stay within the room that the launch and the
workspace have for them, up to the most slots that a call accepts."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_chunks_cover_the_lengths_and_fit_their_room(tmp_path):
    exe = str(tmp_path / "driver")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-Wall", "-Werror", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                        "-I", os.path.join(ROOT, "bit_affine_quantized_amd", "csrc"),
                        os.path.join(ROOT, "tests", "sanitize", "kv_chunks_driver.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
