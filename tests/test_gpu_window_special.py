"""pkv_paged_attention_decode_window: infinities of V in rows that are seen, the two
bf16 terms that a weight is held in, and the smallest K scale."""
import numpy as np
import pytest
import torch

from paged_kv_cache_41_gb300 import pkv

import serving_util as su
from test_gpu_window import Window

pytestmark = pytest.mark.gpu

# Over bf16 and MXFP8 pools a weight p of [2^e, 2^(e+1)) goes into the product as hi +
# lo, two bf16 terms: hi is cut off, lo is what that leaves of p (1 + 2^-23), at most
# a hair above 2^(e-7) (and then rounded back to it), else rounded by half a step of
# the binade below, 2^(e-16): 2^-16 of p, and the 2^-23 itself.
P_TERMS = 2.0 ** -16 + 2.0 ** -23
P_BITS = {"bf16": P_TERMS, "mxfp8": P_TERMS, "f32": 0.0}


class Exact(Window):
    def check(self, out, lse):
        c = self.c
        out, lse, q = (x.double().cpu().numpy() for x in (out, lse, self.q))
        g = self.hq // c.hkv
        for r, n in enumerate(self.lens):
            for h in range(self.hq):
                o, l, _, absv, mag = su.attend64(q[r:r + 1, h], self.k64[r][:, h // g], self.v64[r][:, h // g],
                                                 self.seen[r][None], self.scale)
                su.check_attention(c.dtype, c.d, out[r:r + 1, h], lse[r:r + 1, h], o, l, absv, mag, max(n, 1),
                                   f"sequence {r} ({n} rows) head {h}", p_bits=P_BITS[c.dtype])

    def reread(self):
        self.k64, self.v64 = zip(*(self.c.rows64(r, n) for r, n in enumerate(self.lens)))


# one CTA a segment, one cluster, several clusters; under fp32 one CTA, parts, the balanced split
SHAPES = [([1, 2, 40, 300], 33), ([5, 300, 1, 17] * 100, 120), ([700, 3], 600), ([9000, 1], 8000)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,d", [(2, 2, 64), (4, 2, 128), (8, 2, 128), (8, 1, 64), (8, 1, 128)])
@pytest.mark.parametrize("lens,window", SHAPES)
def test_infinities_of_seen_rows_come_through(dtype, hq, hkv, d, lens, window):
    # whatever the parts that a weight is held in, the largest of a head (exactly 1)
    # and those that bf16 holds exactly among them
    w = Exact(lens, window, 4, dtype=dtype, hq=hq, hkv=hkv, d=d, seed=hq + d)
    w.q *= 0.25  # no weight near the smallest numbers
    v = w.c.v.view(-1, hkv, d)
    for r, n in enumerate(lens[:8]):
        rows = np.nonzero(w.seen[r])[0]
        s = (w.k64[r][rows, 0] @ w.q[r, 0].double().cpu().numpy()).argmax()
        for i, (t, x) in enumerate([(rows[0], float("inf")), (rows[-1], -float("inf")), (rows[s], float("inf")),
                                    (rows[len(rows) // 2], float("nan"))]):
            v[int(w.c.slots(r, [t])[0]), :, 10 * i:10 * i + 3] = x
    w.reread()
    out, lse = w.call()
    assert pkv.get_device_error() == 0
    w.check(out, lse)
    for r in range(min(8, len(lens))):
        assert (out[r, :, :3] == float("inf")).all() and (out[r, :, 10:13] == -float("inf")).all()
        assert (out[r, :, 20:23] == float("inf")).all() and out[r, :, 30:33].isnan().all()


@pytest.mark.parametrize("same", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_infinities_where_every_weight_is_one(same, d):
    # keys of zero: every weight is 1 and so is held by the first term alone
    w = Exact([50, 1, 3], 40, 2, dtype="bf16", hq=4, hkv=1, d=d, seed=1)
    live = ~w.c.k.isnan()
    w.c.k[live] = 0.0
    v = w.c.v.view(-1, 1, d)
    for r, n in enumerate(w.lens):
        v[int(w.c.slots(r, [n - 1])[0]), 0, 7] = float("inf")
        if same:
            v[int(w.c.slots(r, [0])[0]), 0, 7] = float("inf")
    w.reread()
    out, lse = w.call()
    assert pkv.get_device_error() == 0
    w.check(out, lse)
    assert (out[:, :, 7] == float("inf")).all()


@pytest.mark.parametrize("dtype", ["bf16", "mxfp8"])
@pytest.mark.parametrize("hq,hkv,d", [(2, 2, 64), (4, 2, 128), (8, 2, 128), (16, 2, 128)])
@pytest.mark.parametrize("lens,window", [([2, 3, 64, 129, 700], 150), ([4000, 6001], 3000)])
def test_weights_are_held_in_two_terms(dtype, hq, hkv, d, lens, window):
    Exact(lens, window, 3, dtype=dtype, hq=hq, hkv=hkv, d=d, seed=hq + d).run()


@pytest.mark.parametrize("dtype", ["bf16", "mxfp8", "f32"])
@pytest.mark.parametrize("hq", [2, 4, 8, 16])
def test_few_keys_of_opposite_values(dtype, hq):
    # two keys of nearly the same weight and values of opposite sign: what is
    # left of the outputs is the weights' difference
    w = Exact([2, 2, 2], 2, 0, dtype=dtype, hq=hq, hkv=2, d=128, seed=hq)
    for r in range(3):
        a, b = (int(w.c.slots(r, [i])[0]) for i in range(2))
        if dtype == "mxfp8":
            w.c.v.elements.view(-1, 2, 128)[b] = w.c.v.elements.view(-1, 2, 128)[a] ^ 0x80
            ba, bb = a // 16, b // 16
            w.c.v.scales[bb, :, b % 16] = w.c.v.scales[ba, :, a % 16]
        else:
            w.c.v.view(-1, 2, 128)[b] = -w.c.v.view(-1, 2, 128)[a]
    w.reread()
    w.run()


@pytest.mark.parametrize("hq,d", [(1, 64), (2, 64), (4, 128), (8, 128)])
@pytest.mark.parametrize("lens,window", [([3, 50, 200], 70), ([3000, 1], 2500)])
def test_keys_of_the_smallest_scale(hq, d, lens, window):
    # K scales of 2^-127 against queries of about 2^112: scores of ordinary size
    w = Exact(lens, window, 2, dtype="mxfp8", hq=hq, hkv=1, d=d, seed=d)
    w.c.k.scales.zero_()
    w.q.copy_((w.q.float() * 2.0 ** 112).to(w.q.dtype))
    w.scale = 6.0
    w.reread()
    out, lse = w.call()
    assert pkv.get_device_error() == 0
    w.check(out, lse)
    assert (lse[1].exp() / min(lens[1], window + 2) - 1).abs().max() > 1e-3 or lens[1] < 3  # not all of score 0
