"""The split of attn_decode over CTAs, compiled for the host and checked there."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_every_tile_once_and_no_index_past_the_arrays(tmp_path):
    exe = str(tmp_path / "split_check")
    build = subprocess.run(["g++", "-std=c++17", "-O1", "-w", "-fsanitize=address,undefined",
                            "-I", os.path.join(ROOT, "scaled_dot_product_saving_b200", "csrc"),
                            os.path.join(ROOT, "tests", "c", "split_check.cpp"), "-o", exe],
                           capture_output=True, text=True)
    assert build.returncode == 0, build.stderr
    run = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stdout + run.stderr
    assert "split_check ok" in run.stdout
