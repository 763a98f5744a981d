"""When the gated delta rule walks long sequences in segments (seen from the
workspace, which holds the segments' states): where few rows leave the card idle
and the sequence is long enough, and not where the whole walk was measured to
take less time (256 CUs; the times are the forward kernels')."""
import pytest

from nonlinear_rnn_solve_pararnn_amd import api

F32, BF16 = 0, 1


def in_segments(backward, dtype, L, H, dk, dv):
    ws = api.load_library().pararnn_delta_workspace_bytes
    rows = 2048 // H + 1
    one, many = ws(backward, dtype, 1, L, H, H, dk, dv), ws(backward, dtype, rows, L, H, H, dk, dv)
    assert one > 0 and many > 0
    return one > 1.01 * many / rows + 4096


@pytest.mark.parametrize("backward", (0, 1))
@pytest.mark.parametrize("dtype,L,H,dk,dv", [(F32, 32771, 8, 64, 128), (BF16, 4096, 16, 128, 128), (F32, 4096, 8, 128, 128),
                                             (BF16, 8192, 4, 64, 64), (F32, 8192, 2, 256, 256), (BF16, 32768, 2, 256, 256)])
def test_few_rows_and_a_long_axis(backward, dtype, L, H, dk, dv):
    assert in_segments(backward, dtype, L, H, dk, dv)


@pytest.mark.parametrize("backward,dtype,L,groups,dk,dv", [
    (0, BF16, 1024, 80, 256, 256),   # 286 us in segments, 140 whole
    (1, BF16, 1024, 80, 256, 256),   # 463, 236
    (0, BF16, 2048, 48, 256, 256),   # 325, 256
    (1, BF16, 2048, 16, 256, 256),   # 463, 335
    (0, F32, 1024, 80, 256, 256),    # 369, 224
    (1, F32, 2048, 96, 256, 256),    # 1145, 865
    (0, F32, 1024, 96, 128, 128),    # 193, 149
    (1, F32, 1024, 80, 128, 128),    # 277, 220
    (0, F32, 1024, 96, 128, 64),     # 233, 163
    (1, F32, 2048, 96, 128, 64),     # 606, 525
    (0, BF16, 1024, 96, 128, 128),   # 110, 93
    (1, BF16, 1024, 96, 128, 128),   # 171, 151
])
def test_whole_where_that_is_faster(backward, dtype, L, groups, dk, dv):
    assert not in_segments(backward, dtype, L, groups // ((dv + 63) // 64 * (backward + 1)), dk, dv)


@pytest.mark.parametrize("backward", (0, 1))
def test_short_sequences_and_full_cards_are_walked_whole(backward):
    for dtype in (F32, BF16):
        assert not in_segments(backward, dtype, 512, 2, 64, 64) and not in_segments(backward, dtype, 8192, 128, 128, 128)
