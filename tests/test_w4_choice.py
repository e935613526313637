"""Which tiles the products with 4-bit weights take, without a GPU: the choice goes by
the rows that there are."""
import os
import shutil
import subprocess

import pytest

from combine_topk_ids_dest_amd import build as hip_build

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def choice(tmp_path_factory):
    """choice(lines): (kernel, tiles in use) of each."""
    if shutil.which("g++") is None:
        pytest.skip("g++ is not installed")
    exe = str(tmp_path_factory.mktemp("w4") / "w4_choice")
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Wextra", "-Werror",
                    "-I", hip_build.CSRC, os.path.join(HERE, "w4_choice.cpp"), "-o", exe],
                   check=True, capture_output=True)

    def ask(*lines):
        out = subprocess.run([exe], input="\n".join(lines), capture_output=True, text=True,
                             check=True).stdout.split("\n")
        return [(w.split()[0], set(w.split()[1:])) for w in out if w]

    return ask


def experts(counts, rows, H, N, gated, group):
    return f"experts {rows} {H} {N} {int(gated)} {group} " + " ".join(map(str, counts))


def test_few_rows_of_most_experts_count_beside_a_big_tile(choice):
    """One expert of 20 rows and 31 of one: few-row tiles for all 118 us, a 32-row
    tile with the others behind it 153 (7168 -> 2 x 2048, E4M3)."""
    one = [20] + [1] * 31
    assert choice(experts(one, 256, 7168, 2048, True, 16)) == [("big", {"few"})]
    assert choice(experts(one, 256, 7168, 2048, True, 32)) == [("big", {"few"})]
    # alone it is the other way round with eight of them
    assert choice(experts([20] * 8, 256, 7168, 2048, True, 16)) == [("big", {"32"})]

