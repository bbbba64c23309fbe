"""Rows that pkv_kv_compact does not move: K, V and their weights alike."""
import numpy as np
import pytest

from paged_kv_cache_41_gb300 import pkv

from test_gpu_evict import Compact

pytestmark = pytest.mark.gpu


def moved(c, bad):
    """Per kv head, which kept rows of sequence 0 are not held by the bad block,
    and whether one is that would have to move (one in its place is not looked
    at)."""
    p, n = c.cache.p, int(c.keep_lens[0])
    out, held = [], False
    for h in range(c.cache.hkv):
        k = c.keep[0, h if c.keep.shape[1] > 1 else 0, :n] + c.base[0]
        to = c.base[0] + np.arange(n)
        out.append((k // p != bad) & (to // p != bad))
        held |= bool((~out[-1] & (k != to)).any())
    return out, held


@pytest.mark.parametrize("dtype", ["bf16", "f32", "mxfp8"])
@pytest.mark.parametrize("pattern", ["last", "random", "ends"])
@pytest.mark.parametrize("bad", [0, 1, 9])
@pytest.mark.parametrize("per_head,base", [(True, None), (False, [5, 0])])
def test_a_bad_block_holds_rows_and_weights(dtype, pattern, bad, per_head, base):
    c = Compact([200, 60], [70, 20], seed=8, pattern=pattern, dtype=dtype, per_head=per_head, base=base)
    before = c.cache.rows64(0, 200)
    w0 = c.w.cpu().numpy().copy()
    good = int(c.cache.tables_np[0, bad])
    c.cache.tables[0, bad] = -5
    c.call()
    rows_ok, held = moved(c, bad)
    assert pkv.get_device_error() == (pkv.DEVERR_BLOCK if held else 0)
    c.cache.tables[0, bad] = good
    after = c.cache.rows64(0, 200)
    w = c.w.cpu().numpy()
    b0, n = int(c.base[0]), int(c.keep_lens[0])
    for h, ok in enumerate(rows_ok):
        ks = c.keep[0, h if per_head else 0, :n]
        ref = w0[0, h].copy()
        rows = [x[:, h].copy() for x in before]
        to, frm = b0 + np.flatnonzero(ok), b0 + ks[ok]
        ref[to] = w0[0, h, frm]
        for x, y in zip(rows, before):
            x[to] = y[frm, h]
        ref[b0 + n:200] = 0
        assert np.array_equal(w[0, h], ref)
        for x, y in zip(rows, after):
            assert np.array_equal(x, y[:, h])
