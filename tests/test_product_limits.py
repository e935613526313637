"""The products' limit on rows, without a GPU: sums like rows + 255 are formed
in 32 bits, so the last 255 numbers below 2^31 are refused. (No call here passes
every check.)"""
import pytest

from combine_topk_ids_dest_amd import binding as B

FAKE = 0x7F0000000000
TOP = 2 ** 31 - 1 - 255


def _matmul(T, x=FAKE):
    return B.load().moe_ep_matmul(x, 8, FAKE, 8, None, T, 8, 8, 0, None, 0, FAKE, 8, 0, None)


def _experts(rows, x=FAKE):
    return B.load().moe_ep_expert_matmul(x, rows * 8, FAKE, 64, None, 0, FAKE, 1, rows, 8, 8, 0,
                                         FAKE, rows * 8, 0, None)


def _experts_fp8(rows, x=FAKE):
    return B.load().moe_ep_expert_matmul_fp8(x, rows * 128, FAKE, rows * 4, FAKE, 16 * 128, FAKE, 1,
                                             None, 0, FAKE, 1, rows, 128, 16, 0, FAKE, rows * 16, 0,
                                             None, 0, None)


@pytest.mark.parametrize("call", [_matmul, _experts, _experts_fp8])
def test_rows_near_two_to_the_31_are_refused(call):
    for rows in (TOP + 1, TOP + 128, 2 ** 31 - 16, 2 ** 31 - 1):
        # misaligned as well, so that no call is launched: sizes are checked first
        assert call(rows, FAKE + 2) == B.EINVAL, rows
    assert call(TOP, FAKE + 2) == B.EALIGN
