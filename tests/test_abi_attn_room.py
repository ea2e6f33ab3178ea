"""Which calls of the paged attention take a workspace, so that the device may cut their tiles: every one whose table is
longer than its rows, however many rows the call has room for.  No GPU needed."""
import pytest

osc = pytest.importorskip("w4a4_outlier_split_amd", reason="libosc.so not built")


@pytest.mark.parametrize("R", [1, 2, 64])
@pytest.mark.parametrize("HQ,HKV", [(32, 8), (8, 1), (64, 8)])
def test_room_for_many_rows_over_a_long_table(R, HQ, HKV):
    need = {osc.osc_attn_workspace(S, R, HQ, HKV, 128, 64, 640) for S in (R + 1, 300, 2000, 8192, 20000)}
    assert len(need) == 1 and need.pop() > 0


def test_less_room_never_needs_more_than_the_fewest_rows_of_either_kernel():
    for R in (1, 3):
        for MB in (1, 8, 30, 40, 130, 640):
            for HQ, HKV in ((32, 8), (8, 1), (16, 16)):
                ws = lambda S: osc.osc_attn_workspace(S, R, HQ, HKV, 64, 16, MB)
                assert max(ws(S) for S in range(1, 2600, 7)) <= max(ws(R), ws(R + 1), ws(2600))
