"""pkv_draft_tree_attention over many short sequences, several to a CTA, that
hold values no other sequence may see, and over bad tables."""
import numpy as np
import pytest
import torch

from paged_kv_cache_41_gb300 import pkv

import serving_util as su
from test_gpu_draft import Draft

pytestmark = pytest.mark.gpu


def same(a, b):
    """Bit for bit, a NaN like any other."""
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(torch.nan_to_num(a.float(), nan=0.0),
                                                                       torch.nan_to_num(b.float(), nan=0.0))


@pytest.mark.parametrize("dtype", ["bf16", "f32", "mxfp8"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("b,hq,n,ctx", [
    (64, 32, 5, (65, 124)),    # one warp of a group has rows, the other group's clear the drafted ones' V
    (200, 32, 5, (0, 60)),     # one stage a piece
    (64, 64, 20, (40, 230)),   # two row tiles: a group clears for both
    (96, 32, 3, (120, 140)),   # drafted rows in two stages
])
def test_non_finite_rows_of_many_short_sequences(dtype, d, b, hq, n, ctx):
    rng = np.random.default_rng(b + n)
    dr = Draft(rng.integers(ctx[0], ctx[1] + 1, b), [n] * b, dtype=dtype, hq=hq, hkv=8, d=d, seed=b + d)
    # in most sequences one drafted row holds values that are not finite, in
    # every kv head; every other row sees it
    words = []
    for r in range(b):
        j = int(rng.integers(0, n))
        own = [(1 | 1 << i) & ~(1 << j) | ((i + r) % 2) << j for i in range(n)]
        words.append(own)
        if r % 8 == 7:
            continue
        slot = int(dr.cache.slots(r, [dr.ctx[r] + j])[0])
        if dtype == "mxfp8":
            dr.cache.v.elements.view(-1, 8, d)[slot, :, 3:d - 5:3] = 0x7F
            dr.cache.v.elements.view(-1, 8, d)[slot, :, d - 2] = 0xFF
        else:
            v = dr.cache.v.view(-1, 8, d)
            v[slot, :, 3:d - 5:3] = float("inf") if r % 3 else float("nan")
            v[slot, :, d - 2] = -float("inf")
    dr.words = words
    dr.masks = su.as_int64(sum(words, [])).cuda()
    out, lse = dr.call()
    assert pkv.get_device_error() == 0
    dr.check(out, lse)
    for _ in range(20):  # the warps' order differs from call to call
        o, l = dr.call()
        assert same(o, out) and torch.equal(l, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "mxfp8"])
@pytest.mark.parametrize("bad", [-2, -3, -2**31, 2**31 - 2])
@pytest.mark.parametrize("place", [0, 3, 12])
def test_any_bad_block_sets_the_error(dtype, bad, place):
    # in the first block, in one of the context, and in the drafted rows' own
    dr = Draft([190, 30], [14, 5], dtype=dtype, hq=8, hkv=2, d=128, seed=13)
    dr.cache.tables[0, place] = bad
    dr.call()
    assert pkv.get_device_error() == pkv.DEVERR_BLOCK
    # a table that is right where rows are, and anything behind them
    dr = Draft([190, 30], [14, 5], dtype=dtype, hq=8, hkv=2, d=128, width=20, seed=13)
    dr.cache.tables[0, 13:] = bad
    dr.cache.tables[1, 3:] = bad
    dr.run()
