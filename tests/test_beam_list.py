"""The selection scan's list of hits on the CPU (csrc/beam_list.h): in every
order of the threads' atomics, only places that were written are read back.
An entry read from a place that no thread wrote would be used as an index."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("beam_list") / "driver")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-Wall", "-Werror", "-fsanitize=address,undefined",
                        "-I", os.path.join(ROOT, "bit_affine_quantized_amd", "csrc"),
                        os.path.join(ROOT, "tests", "sanitize", "beam_list_driver.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return exe


@pytest.mark.parametrize("threads", [
    # a last chunk of 3616 logits, 25 runs of eight of every 64 above the bound, by wave: 400, 400, 400, 232
    [(25, 16), (39, 0)] * 3 + [(4, 16), (21, 8), (39, 0)],
    # equal logits, 50257 of them: the last chunk's 1105, 16 a thread, the last one's a single one
    [(64, 16), (5, 16), (1, 1), (186, 0)],
    [(256, 16)], [(256, 4)], [(64, 16), (192, 0)], [(256, 5)], [(255, 4), (1, 5)], [(20, 64), (236, 0)], [(256, 64)], [(255, 0), (1, 7)], [(256, 0)]])
def test_no_unwritten_place_is_read(driver, threads):
    assert sum(c for c, _ in threads) == 256
    r = subprocess.run([driver, *[str(x) for pair in threads for x in pair]], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
