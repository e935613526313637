"""Which tiles the products with 4-bit weights take, without a GPU: the cases of the
GPU tests reach every kind, and the choice goes by the rows that there are."""
import os
import shutil
import subprocess

import pytest

from combine_topk_ids_dest_amd import build as hip_build
from w4_cases import EXPERTS, H, TOKENS, WIDE_N

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


@pytest.mark.parametrize("group", [16, 32])
@pytest.mark.parametrize("gated", [False, True])
def test_the_cases_take_every_kind_of_tile(choice, gated, group):
    got = choice(*(f"dense {T} {H} {WIDE_N[gated]} {int(gated)} {group}" for T in TOKENS))
    for (T, want), (_, tiles) in zip(TOKENS.items(), got):
        assert want in tiles, (T, tiles)
    for name, (counts, rows, N, Ng, kernel, want) in EXPERTS.items():
        for columns in (H, 544, 16 * group):
            (k, tiles), = choice(experts(counts, rows, columns, Ng if gated else N, gated, group))
            assert k == kernel and want <= tiles, (name, columns, k, tiles)


def test_few_rows_of_most_experts_count_beside_a_big_tile(choice):
    """One expert of 20 rows and 31 of one: few-row tiles for all 118 us, a 32-row
    tile with the others behind it 153 (7168 -> 2 x 2048, E4M3)."""
    one = [20] + [1] * 31
    assert choice(experts(one, 256, 7168, 2048, True, 16)) == [("big", {"few"})]
    assert choice(experts(one, 256, 7168, 2048, True, 32)) == [("big", {"few"})]
    # alone it is the other way round with eight of them
    assert choice(experts([20] * 8, 256, 7168, 2048, True, 16)) == [("big", {"32"})]


@pytest.mark.parametrize("rows", [24, 32])
def test_the_room_for_rows_does_not_choose_their_tiles(choice, rows):
    """32 experts of 24 or 32 rows take 32-row tiles with room for 32 rows as with
    more (128 and 281 us), and few-row tiles where they have few rows."""
    for H, N, gated in ((7168, 2048, True), (2048, 7168, False)):
        for group in (16, 32):
            room = [choice(experts([rows] * 32, c, H, N, gated, group)) for c in (32, 33, 256)]
            assert all(r[0][1] == {"32"} for r in room), room
            sparse = [choice(experts([1, 2, 0, 16] * 8, c, H, N, gated, group))
                      for c in (16, 32, 33, 256)]
            assert all(r[0][1] == {"few"} for r in sparse), sparse
    # where all full experts' few-row tiles take less, that kernel alone
    assert choice(experts([32] * 8, 32, 512, 1024, False, 32)) == [("few", {"few"})]
