"""Caches, drafts and plain 64-bit forms for the tests of the draft-tree
attention and of the eviction operators.

The plain forms work on each sequence's rows read back from the pool through
its block table, in binary64 numpy, and share nothing with the kernels.
"""
import math

import numpy as np
import torch

from paged_kv_cache_41_gb300 import pkv

U32 = 2.0 ** -24                # half a step of fp32, relative
HALF = {"f32": U32, "bf16": 2.0 ** -8, "mxfp8": 2.0 ** -8}  # of the output type
IO = {"f32": torch.float32, "bf16": torch.bfloat16, "mxfp8": torch.bfloat16}


class Cache:
    """A paged K/V cache whose rows 0 .. lens[r] - 1 of every sequence are N(0, 1)
    and whose other bytes are NaN; block ids are dealt out in a seeded order."""

    def __init__(self, lens, *, dtype="bf16", hkv=2, d=64, p=16, seed=0, extra_blocks=3, width=None,
                 first_block=0):
        self.dtype, self.hkv, self.d, self.p = dtype, hkv, d, p
        self.lens = [int(t) for t in lens]
        need = [-(-t // p) for t in self.lens]
        used = sum(need) + extra_blocks
        nb = first_block + used
        rng = np.random.default_rng(seed)
        order = first_block + rng.permutation(used).astype(np.int32)
        self.max_blocks = width or max(need + [1])
        tables = np.full((len(lens), self.max_blocks), -1, np.int32)
        at = 0
        for r, n in enumerate(need):
            tables[r, :n] = order[at:at + n]
            at += n
        self.tables_np = tables
        self.tables = torch.from_numpy(tables).cuda()
        if dtype == "mxfp8":
            self.k = pkv.MxPool(nb, p, hkv, d, fill=0x7F)  # NaN codes
            self.v = pkv.MxPool(nb, p, hkv, d, fill=0x7F)
        else:
            self.k = torch.full((nb, p, hkv, d), float("nan"), dtype=IO[dtype], device="cuda")
            self.v = torch.full_like(self.k, float("nan"))
        self.gen = torch.Generator(device="cuda")
        self.gen.manual_seed(seed)
        total = sum(self.lens)
        if total:
            self.append(self.randn(total, hkv, d), self.randn(total, hkv, d),
                        np.concatenate([self.slots(r, np.arange(t)) for r, t in enumerate(self.lens)]))

    def randn(self, *shape):
        return torch.randn(shape, generator=self.gen, device="cuda").to(IO[self.dtype])

    def slots(self, r, pos):
        pos = np.asarray(pos, np.int64)
        return self.tables_np[r, pos // self.p].astype(np.int64) * self.p + pos % self.p

    def append(self, k, v, slots):
        pkv.kv_append(self.k, self.v, k, v, torch.from_numpy(np.asarray(slots, np.int64)).cuda())

    def rows64(self, r, n, pool=None):
        """Rows 0 .. n - 1 of sequence r of K and V, [n, Hkv, D] binary64."""
        out = []
        for x in (self.k, self.v):
            s = torch.from_numpy(self.slots(r, np.arange(n))).cuda()
            if self.dtype == "mxfp8":
                codes = x.elements.view(torch.float8_e4m3fn).view(-1, self.hkv, self.d)[s].double()
                sc = x.scales.transpose(1, 2).reshape(-1, self.hkv, self.d // 32)[s].double()
                y = codes * torch.exp2(sc - 127).repeat_interleave(32, dim=2)
            else:
                y = x.view(-1, self.hkv, self.d)[s].double()
            out.append(y.cpu().numpy())
        return out

    def raw(self):
        """Host copies of both pools' bytes."""
        if self.dtype == "mxfp8":
            return [x.buf.cpu().numpy().copy() for x in (self.k, self.v)]
        bits = torch.int16 if self.dtype == "bf16" else torch.int32
        return [x.view(bits).cpu().numpy().copy() for x in (self.k, self.v)]


def tree_masks(n, rng, width=4):
    """Bit masks of a random tree of n nodes (each node and its ancestors)."""
    words = []
    for i in range(n):
        parent = -1 if i == 0 else int(rng.integers(max(0, i - width), i))
        words.append((1 << i) | (words[parent] if parent >= 0 else 0))
    return words


def as_int64(words):
    return torch.tensor([w - (1 << 64) if w >> 63 else w for w in words], dtype=torch.int64)


def attend64(q, k, v, seen, scale):
    """One kv head in binary64: q [rows, D] against k, v [t, D], seen [rows, t].
    Returns out, lse, weights, and the two magnitudes the error bounds need:
    sum_t w |v| and the largest scale * sum_d |q k| over seen rows."""
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        s = np.where(seen, scale * (q @ k.T), -np.inf)
        top = s.max(axis=1, keepdims=True, initial=-np.inf)
        top = np.where(np.isneginf(top), 0.0, top)
        e = np.exp(s - top)
        total = e.sum(axis=1, keepdims=True)
        w = np.divide(e, total, out=np.zeros_like(e), where=total != 0)
        lse = np.where(total[:, 0] == 0, -np.inf, np.log(total[:, 0]) + top[:, 0])
        # a hidden row contributes nothing, whatever its bytes
        out = np.zeros((q.shape[0], v.shape[1]))
        absv = np.zeros_like(out)
        for i in range(q.shape[0]):
            on = seen[i]
            out[i] = w[i, on] @ v[on]
            absv[i] = w[i, on] @ np.abs(v[on])
        a = np.where(seen, scale * (np.abs(q) @ np.abs(k).T), 0.0)
    return out, lse, w, absv, a.max(axis=1, initial=0.0)


def score_error(d, a, t):
    """Bound on a weight's relative error, and on the LSE's absolute one, in
    fp32: the dot product's d + 2 roundings of terms adding up to a (fused,
    scaled by log2 e in q: two more), the exponential and logarithm
    approximations (2^-21 together) and the sum of t weights (pairs, tiles and
    pieces: at most t / 16 + 64 roundings in a row)."""
    return (d + 4) * U32 * a + 2.0 ** -21 + (t / 16 + 64) * U32


def check(got, want, bound, what):
    got = np.asarray(got, np.float64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    nan = np.isnan(want)
    inf = np.isinf(want)
    assert np.array_equal(np.isnan(got), nan), f"{what}: NaN in other places"
    assert np.array_equal(got[inf], want[inf]), f"{what}: infinities differ"
    ok = ~(nan | inf)
    err = np.abs(got[ok] - want[ok])
    bad = ~(err <= np.broadcast_to(bound, want.shape)[ok])
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside the bound, worst "
                           f"{(err / np.broadcast_to(bound, want.shape)[ok]).max():.3g} x")


def check_attention(dtype, d, got_out, got_lse, out, lse, absv, a, t, what, p_bits=None):
    """Compare one (rows, head) result with its binary64 form.  The bound of
    out: its own rounding, twice the weights' relative error (numerator and
    sum) and, where weights are rounded to bf16 for the tensor cores, half a
    bf16 step of each (p_bits = 2^-8), all times sum w |v|; the running sum of
    products adds one rounding per tile of 32 rows."""
    e = score_error(d, a, t)[:, None]
    rel = 2 * e + (t / 16 + 64) * U32 + (p_bits or 0.0)
    bound = rel * absv + HALF[dtype] * (np.abs(out) + rel * absv) + 1e-37
    check(got_out, out, bound, what + " out")
    if got_lse is not None:
        check(got_lse, lse, e[:, 0] + 2 * U32 * np.where(np.isfinite(lse), np.abs(lse), 0.0) + 2.0 ** -22,
              what + " lse")


def softmax_scale(d):
    return 1.0 / math.sqrt(d)
