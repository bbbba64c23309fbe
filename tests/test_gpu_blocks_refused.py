"""pkv_kv_blocks_update: what becomes of a request whose growth is refused, with a
window and without."""
import pytest
import torch

from paged_kv_cache_41_gb300 import pkv

from test_gpu_blocks import Step

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("refusal", ["pool", "rows"])
def test_blocks_behind_the_window_go_though_the_growth_is_refused(refusal):
    # 10 blocks each, of which a decode over 160 rows sees the sinks' and the last
    # three; nothing is free but what lies behind the two windows
    s = Step([160, 160], 100, spare=0)
    first = s.plain.tables[0][:]
    add, rows, bit = ([0, 16 * 30], 1000, pkv.DEVERR_POOL) if refusal == "pool" else ([0, 33], 32, pkv.DEVERR_LENGTH)
    got, err = s.update("lens", add, rows, window=48, sinks=16)
    assert err == bit
    assert got[0].tolist() == [160, 160] and (got[2] == -1).all() and (got[3] == -1).all()
    assert s.count.item() == 12
    for r in range(2):
        assert all((s.plain.tables[r][j] < 0) == (1 <= j < 7) for j in range(10))
        assert s.plain.tables[r][10:] == [-1] * 90
    # the same growth afterwards, of a size that what went has room for
    assert s.plain.tables[0][0] == first[0]
    got, err = s.update("lens", [0, 16 * 12], 1000, window=48, sinks=16)
    assert err == 0 and got[0].tolist() == [160, 352] and s.count.item() == 0


def test_without_a_window_a_refused_growth_changes_nothing():
    s = Step([160, 160], 100, spare=3)
    before = [x.clone() for x in (s.tables, s.free, s.count)]
    got, err = s.update("lens", [0, 16 * 30], 1000)
    assert err == pkv.DEVERR_POOL and got[0].tolist() == [160, 160]
    for x, y in zip(before, (s.tables, s.free, s.count)):
        assert torch.equal(x, y)


def test_lengths_that_make_no_sense_keep_the_whole_table():
    s = Step([160, 160], 100, spare=3)
    before = s.tables.clone()
    got, err = s.update("lens", [-161, 10**6], 1000, window=48, sinks=16)
    assert err == pkv.DEVERR_LENGTH and got[0].tolist() == [160, 160]
    assert torch.equal(before, s.tables) and got[1].tolist() == [0, 0, 0]
