"""The products' tiles, without a GPU: each row of each column tile has one
block. A row that two blocks store is wrong where the residual is the output
itself: the second reads what the first has stored."""
import os
import shutil
import subprocess

import pytest

from combine_topk_ids_dest_amd import build as hip_build

HERE = os.path.dirname(os.path.abspath(__file__))


def test_every_row_and_column_tile_has_one_block(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("g++ is not installed")
    exe = str(tmp_path / "tiles_cover")
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Wextra", "-Werror",
                    "-I", hip_build.CSRC, os.path.join(HERE, "tiles_cover.cpp"), "-o", exe],
                   check=True, capture_output=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout[:600] + " ... " + r.stdout[-200:]
