"""pkv_draft_tree_attention on the tensor cores holds its weights to more than
bf16: against the plain 64-bit form, and against the decode."""
import numpy as np
import pytest
import torch

from paged_kv_cache_41_gb300 import pkv

import serving_util as su
from test_gpu_draft import Draft

pytestmark = pytest.mark.gpu

# A weight p goes into the product as hi + lo, two bf16 terms: hi is p cut off
# (2^-7 p at most below it), lo is p (1 + 2^-20) - hi rounded (half a step,
# 2^-8 of at most (2^-7 + 2^-20) p), and the 2^-20 itself.
P_BITS = 2.0 ** -15 + 2.0 ** -28 + 2.0 ** -20


def check(dr, out, lse, p_bits=P_BITS):
    c = dr.cache
    o64, l64, q = [x.double().cpu().numpy() for x in (out, lse, dr.q)]
    g = dr.hq // c.hkv
    for r, (ctx, n) in enumerate(zip(dr.ctx, dr.n)):
        if n == 0:
            continue
        a, b = dr.ptr_np[r], dr.ptr_np[r + 1]
        k, v = c.rows64(r, ctx + n)
        seen = np.ones((n, ctx + n), bool)
        seen[:, ctx:] = [[(w >> j) & 1 for j in range(n)] for w in dr.words[r]]
        for h in range(dr.hq):
            o, l, _, absv, mag = su.attend64(q[a:b, h], k[:, h // g], v[:, h // g], seen, dr.scale)
            su.check_attention(c.dtype, c.d, o64[a:b, h], l64[a:b, h], o, l, absv, mag, ctx + n,
                               f"sequence {r} head {h}", p_bits=p_bits)


@pytest.mark.parametrize("dtype", ["bf16", "mxfp8"])
@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (16, 2, 128), (4, 2, 64)])
@pytest.mark.parametrize("ctx,n", [([300], [4]), ([0, 3, 9, 40], [1, 2, 7, 20]), ([63, 64, 65, 127, 128], [1] * 5),
                                   ([700, 129, 5], [64, 33, 64]), ([6001], [13])])
def test_weights_are_held_in_two_terms(dtype, hq, hkv, d, ctx, n):
    dr = Draft(ctx, n, dtype=dtype, hq=hq, hkv=hkv, d=d, seed=d + sum(n))
    out, lse = dr.call()
    assert pkv.get_device_error() == 0
    check(dr, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "mxfp8"])
def test_few_keys_of_opposite_values(dtype):
    # two keys of nearly the same weight and values of opposite sign: what is
    # left of the outputs is the weights' difference
    dr = Draft([2, 2, 1], [1, 3, 1], 0, dtype=dtype, hq=8, hkv=2, d=128, seed=30)
    c = dr.cache
    for r in range(3):
        s = [torch.from_numpy(c.slots(r, [i])).cuda() for i in range(2)]
        if dtype == "bf16":
            v = c.v.view(-1, 2, 128)
            v[s[1]] = -v[s[0]]
        else:
            c.v.elements.view(-1, 2, 128)[s[1]] = c.v.elements.view(-1, 2, 128)[s[0]] ^ 0x80
            p = c.v.shape[1]
            at = [(int(x) // p, int(x) % p) for x in s]
            c.v.scales[at[1][0], :, at[1][1]] = c.v.scales[at[0][0], :, at[0][1]]
    # sequence 2 has one row of context: its second row, drafted, is hidden
    out, lse = dr.call()
    assert pkv.get_device_error() == 0
    check(dr, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "mxfp8"])
@pytest.mark.parametrize("hq", [2, 8, 16])
def test_chain_of_one_agrees_with_the_decode(dtype, hq):
    dr = Draft([1000, 31, 8, 0, 127, 128, 2500], [1] * 7, "chain", dtype=dtype, hq=hq, hkv=2, d=128, seed=31)
    out, lse = dr.call()
    want_lse = torch.empty_like(lse)
    want = pkv.paged_attention_decode(dr.q, dr.cache.k, dr.cache.v, dr.cache.tables, dr.ctx_t + 1, dr.scale,
                                      lse=want_lse)
    assert pkv.get_device_error() == 0
    # each by its own bound: the decode holds weights in fp32 on the CUDA
    # cores and in two rounded bf16 terms (2^-16) for eight heads a kv head
    check(dr, out, lse)
    check(dr, want, want_lse, p_bits=2.0 ** -16 if hq == 16 else 0.0)
    # and of each other: both are the rounded value of something within its
    # bound of the same number, so they differ by half a step of each and the
    # two errors under it
    q, g = dr.q.double().cpu().numpy(), hq // 2
    a64, b64 = out.double().cpu().numpy(), want.double().cpu().numpy()
    for r, ctx in enumerate(dr.ctx):
        k, v = dr.cache.rows64(r, ctx + 1)
        for h in range(hq):
            o, l, _, absv, mag = su.attend64(q[r:r + 1, h], k[:, h // g], v[:, h // g],
                                             np.ones((1, ctx + 1), bool), dr.scale)
            e = su.score_error(128, mag, ctx + 1)
            rel = 2 * e[0] + ((ctx + 1) / 16 + 64) * su.U32 + P_BITS
            bound = 2 * (rel * absv + su.HALF["bf16"] * (np.abs(o) + rel * absv))
            su.check(a64[r:r + 1, h], b64[r:r + 1, h], bound, f"sequence {r} head {h}")
            apart = abs(float(lse[r, h]) - float(want_lse[r, h]))
            assert apart <= 2 * (e[0] + 2 * su.U32 * abs(l[0]) + 2.0 ** -22)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("ctx", [2, 40, 200, 1500])
def test_infinities_of_the_context_come_through(dtype, ctx):
    # context rows are seen by every drafted one: an infinite value of V makes
    # that output infinite, whatever the parts its weight is held in (the
    # largest weight of a row, exactly 1, among them)
    dr = Draft([ctx], [7], dtype=dtype, hq=8, hkv=2, d=128, seed=32)
    dr.q *= 0.25  # no weight near the smallest numbers
    v = dr.cache.v.view(-1, 2, 128)
    for i, (t, x) in enumerate([(0, float("inf")), (ctx - 1, -float("inf")), (ctx // 2, float("nan"))]):
        v[int(dr.cache.slots(0, [t])[0]), :, 10 * i:10 * i + 3] = x
    out, lse = dr.call()
    assert pkv.get_device_error() == 0
    check(dr, out, lse, p_bits=0.0 if dtype == "f32" else P_BITS)
    assert (out[:, :, :3] == float("inf")).all() and (out[:, :, 10:13] == -float("inf")).all()
    # the largest weight: one row of context alone
    one = Draft([1], [1], 0, dtype=dtype, hq=8, hkv=2, d=128, seed=33)
    one.cache.v.view(-1, 2, 128)[int(one.cache.slots(0, [0])[0]), :, 5] = -float("inf")
    out, lse = one.call()
    assert (out[:, :, 5] == -float("inf")).all()
    check(one, out, lse, p_bits=0.0 if dtype == "f32" else P_BITS)
