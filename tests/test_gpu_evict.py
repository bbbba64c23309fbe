"""The eviction operators against plain forms: the weighing decode in 64 bits,
the selection and the compaction exactly."""
import numpy as np
import pytest
import torch

from paged_kv_cache_41_gb300 import pkv

import serving_util as su

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ weighing
class Weigh:
    def __init__(self, lens, *, dtype="bf16", hq=4, hkv=2, d=64, p=16, seed=0, slack=5, first_block=0):
        self.cache = su.Cache(lens, dtype=dtype, hkv=hkv, d=d, p=p, seed=seed, first_block=first_block)
        self.lens, self.hq = list(lens), hq
        self.q = self.cache.randn(len(lens), hq, d)
        self.lens_t = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.w = torch.rand(len(lens), hkv, max(self.lens) + slack, generator=self.cache.gen,
                            device="cuda")
        self.scale = su.softmax_scale(d)

    def call(self, **kw):
        c = self.cache
        lse = torch.empty(len(self.lens), self.hq, device="cuda")
        out = pkv.paged_attention_decode_weights(self.q, c.k, c.v, c.tables, self.lens_t, self.w,
                                                 self.scale, lse=lse, **kw)
        return out, lse

    def check(self, w0, out, lse, decay=1.0):
        c = self.cache
        g = self.hq // c.hkv
        # eight heads on the tensor cores: a weight as two bf16 terms
        p_bits = 2.0 ** -16 if g == 8 and c.dtype != "f32" else 0.0
        q = self.q.double().cpu().numpy()
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        w = self.w.double().cpu().numpy()
        w0 = w0.double().cpu().numpy()
        for r, t in enumerate(self.lens):
            assert np.array_equal(w[r, :, t:], w0[r, :, t:]), "entries past the length"
            k, v = c.rows64(r, t)
            seen = np.ones((g, t), bool)
            for h in range(c.hkv):
                mine = slice(h * g, (h + 1) * g)
                o, l, p, absv, mag = su.attend64(q[r, mine], k[:, h], v[:, h], seen, self.scale)
                su.check_attention(c.dtype, c.d, out[r, mine], lse[r, mine], o, l, absv, mag, t,
                                   f"sequence {r}", p_bits=p_bits)
                want = decay * w0[r, h, :t] + p.sum(0)
                # each weight: its score's and its LSE's error, the LSE's own
                # rounding; the sum and the update: a rounding each
                e = 2 * su.score_error(c.d, mag, t) + 4 * su.U32 * (np.abs(l) + 1) + 2.0 ** -21
                bound = (e[:, None] * p).sum(0) + (g + 2) * su.U32 * np.abs(want) + 1e-37
                su.check(w[r, h, :t], want, bound, f"sequence {r} kv head {h} weights")

    def run(self, decay=1.0, **kw):
        w0 = self.w.clone()
        out, lse = self.call(decay=decay, **kw)
        assert pkv.get_device_error() == 0
        self.check(w0, out, lse, decay)


LENS = [1, 0, 15, 16, 17, 31, 32, 33, 127, 128, 129, 500]


@pytest.mark.parametrize("dtype,g,d", [("bf16", g, d) for g in (1, 2, 4, 8) for d in (64, 128)]
                         + [("f32", g, d) for g in (1, 2, 4, 8) for d in (64, 128)]
                         + [("mxfp8", g, d) for g in (1, 2, 4) for d in (64, 128)] + [("mxfp8", 8, 128)])
def test_weigh_types_and_heads(dtype, g, d):
    Weigh(LENS, dtype=dtype, hq=2 * g, hkv=2, d=d, seed=g + d).run()


@pytest.mark.parametrize("p", [16, 32, 64, 96, 128, 256])
@pytest.mark.parametrize("g", [4, 8])
def test_weigh_block_sizes(p, g):
    Weigh([p - 1, p, p + 1, 3 * p + 7, 1], hq=2 * g, hkv=2, d=128, p=p, seed=p).run(decay=0.5)


@pytest.mark.parametrize("g", [4, 8])
def test_weigh_long_and_cut_segments(g):
    Weigh([20000, 3, 7777], hq=2 * g, hkv=2, d=128, seed=1).run()


def test_weigh_many_short():
    rng = np.random.default_rng(2)
    Weigh(rng.integers(0, 90, 700), hq=8, hkv=2, d=64, seed=2).run()


@pytest.mark.parametrize("decay", [0.0, 0.9, 1.0, -1.0])
def test_weigh_decay(decay):
    Weigh([100, 7], hq=8, hkv=2, d=128, seed=3).run(decay=decay)


def test_weigh_sums_over_steps():
    wg = Weigh([300, 40], dtype="f32", hq=4, hkv=2, d=64, seed=4)
    wg.w.zero_()
    for _ in range(4):
        wg.call()
        wg.q.copy_(wg.cache.randn(*wg.q.shape))
    # each step's weights of a head sum to one; the errors of 4 * 2 softmax
    # rows add, as does a rounding per row and step
    tot = wg.w.double().sum(-1).cpu().numpy()
    assert np.allclose(tot, 8.0, rtol=0, atol=8 * 2e-4)


@pytest.mark.parametrize("g", [2, 8])
def test_weigh_same_result_as_the_plain_decode(g):
    wg = Weigh([1000, 31, 0, 4000], hq=2 * g, hkv=2, d=128, seed=5)
    out, lse = wg.call()
    want_lse = torch.empty_like(lse)
    want = pkv.paged_attention_decode(wg.q, wg.cache.k, wg.cache.v, wg.cache.tables, wg.lens_t,
                                      wg.scale, lse=want_lse)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_weigh_rows_wider_than_the_view():
    wg = Weigh([60, 100], hq=4, hkv=2, d=64, seed=6)
    buf = torch.full((2, 2, 128), 3.0, device="cuda")
    buf[:, :, :101] = 0.25
    wg.w = buf[:, :, :101]
    w0 = wg.w.clone()
    out, lse = wg.call()
    wg.check(w0, out, lse)
    assert (buf[:, :, 101:] == 3.0).all()


def test_weigh_length_past_the_scores_and_the_table():
    wg = Weigh([60, 100, 20], hq=4, hkv=2, d=64, seed=7)
    w0 = wg.w.clone()
    full, _ = wg.call()
    done = wg.w
    wg.w = w0[:, :, :80].contiguous()
    out, _ = wg.call()
    assert pkv.get_device_error() == pkv.DEVERR_LENGTH
    assert torch.equal(out, full) and torch.equal(wg.w, done[:, :, :80])
    wg.w = w0.clone()
    wg.lens_t[2] = -3
    wg.call()
    assert pkv.get_device_error() == pkv.DEVERR_LENGTH
    assert torch.equal(wg.w[2], w0[2])


@pytest.mark.parametrize("g", [4, 8])
def test_weigh_bad_block(g):
    wg = Weigh([60, 100], hq=2 * g, hkv=2, d=128, seed=8)
    wg.cache.tables[0, 2] = wg.cache.k.shape[0]
    wg.call()
    assert pkv.get_device_error() == pkv.DEVERR_BLOCK


def test_weigh_pool_past_2_31_elements():
    Weigh([300, 77], hq=32, hkv=8, d=128, seed=9, first_block=2**31 // (16 * 8 * 128) + 5).run()


def test_weigh_graph_and_stream():
    wg = Weigh([700, 64], hq=8, hkv=2, d=128, seed=10)
    out, lse = torch.empty_like(wg.q), torch.empty(2, 8, device="cuda")
    ws = torch.empty(pkv.decode_weights_workspace_bytes(wg.cache.k, 2, 8, wg.cache.max_blocks),
                     dtype=torch.uint8, device="cuda")
    args = (wg.q, wg.cache.k, wg.cache.v, wg.cache.tables, wg.lens_t, wg.w, wg.scale)
    pkv.paged_attention_decode_weights(*args, out=out, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.paged_attention_decode_weights(*args, out=out, lse=lse, workspace=ws)
    w0 = wg.w.clone()
    ws.fill_(0xFF)
    wg.q.copy_(wg.cache.randn(*wg.q.shape))
    g.replay()
    torch.cuda.synchronize()
    wg.check(w0, out, lse)
    s = torch.cuda.Stream()
    w0 = wg.w.clone()
    torch.cuda.synchronize()
    pkv.paged_attention_decode_weights(*args, out=out, lse=lse, workspace=ws, stream=s)
    s.synchronize()
    wg.check(w0, out, lse)


# ----------------------------------------------------------------- selection
def select_plain(w, lens, budget, sinks, recent):
    b, hkv, n = w.shape
    keep = np.full((b, hkv, budget), -1, np.int32)
    for r in range(b):
        t = min(max(int(lens[r]), 0), n)
        for c in range(hkv):
            if t <= budget:
                kept = list(range(t))
            else:
                mid = list(range(sinks, t - recent))
                key = np.where(np.isnan(w[r, c]), -np.inf, w[r, c].astype(np.float64))
                nan = np.isnan(w[r, c])
                mid.sort(key=lambda i: (nan[i], -key[i], i))
                kept = sorted(list(range(sinks)) + list(range(t - recent, t))
                              + mid[:budget - sinks - recent])
            keep[r, c, :len(kept)] = kept
    return keep, np.minimum(np.clip(lens, 0, n), budget).astype(np.int32)


def run_select(w, lens, budget, sinks=0, recent=0, err=0, **kw):
    wt = torch.from_numpy(w).cuda() if isinstance(w, np.ndarray) else w
    keep, new = pkv.kv_evict_select(wt, torch.tensor(lens, dtype=torch.int32, device="cuda"), budget,
                                    num_sinks=sinks, num_recent=recent, **kw)
    assert pkv.get_device_error() == err
    want, want_new = select_plain(wt.cpu().numpy(), np.asarray(lens), budget, sinks, recent)
    assert np.array_equal(new.cpu().numpy(), want_new)
    got = keep.cpu().numpy()
    for r, c in np.argwhere((got != want).any(-1)):
        odd = sorted(set(got[r, c]) ^ set(want[r, c]))
        assert False, f"row {r} {c}: {[(int(i), wt[r, c, i].item()) for i in odd[:8]]}"


@pytest.mark.parametrize("n,budget,sinks,recent", [
    (1, 1, 0, 0), (5, 3, 1, 1), (64, 63, 4, 8), (1023, 100, 0, 10), (1024, 1000, 16, 0),
    (1025, 1, 0, 0), (1025, 512, 256, 256), (5000, 2048, 4, 128), (40001, 16384, 16, 1000),
    (70000, 65536, 0, 1), (131072, 5000, 3, 7), (131073, 70000, 2, 9), (8192, 1000, 4, 4),
    (8193, 8000, 0, 0), (16385, 300, 5, 5), (32769, 32768, 1, 1), (65537, 40000, 0, 100)])
def test_select_sizes(n, budget, sinks, recent):
    rng = np.random.default_rng(n)
    w = np.exp(2 * rng.standard_normal((3, 2, n))).astype(np.float32)
    run_select(w, [n, n // 2, max(0, budget - 1)], budget, sinks, recent)


@pytest.mark.parametrize("kind", ["equal", "two values", "zeros", "few", "signs", "special", "steps"])
@pytest.mark.parametrize("n", [300, 9000])
def test_select_ties_and_special_values(kind, n):
    rng = np.random.default_rng(5)
    shape = (2, 3, n)
    if kind == "equal":
        w = np.full(shape, 0.125)
    elif kind == "two values":
        w = rng.integers(0, 2, shape) * 1.0
    elif kind == "zeros":
        w = np.where(rng.random(shape) < 0.5, 0.0, -0.0)
    elif kind == "few":
        w = rng.integers(0, 7, shape) / 8.0
    elif kind == "signs":
        w = rng.standard_normal(shape)
    elif kind == "special":
        w = rng.choice([np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-42, -1e-42, 1.0, 3.4e38], shape)
    else:  # neighbours in the last bit
        w = (np.float32(1.0).view(np.int32) + rng.integers(0, 40, shape)).astype(np.int32).view(np.float32)
    w = np.ascontiguousarray(w, dtype=np.float32)
    for budget in (1, n // 3, n - 1):
        run_select(w, [n, n - 5], budget, min(2, budget // 2), min(5, budget // 2))


@pytest.mark.parametrize("n,budget,sinks,recent", [
    (196609, 9000, 4, 64), (393216, 200000, 0, 1000), (393217, 20000, 16, 64), (500001, 499999, 1, 1)])
def test_select_lengths_past_one_cta_and_past_a_cluster(n, budget, sinks, recent):
    rng = np.random.default_rng(n)
    w = np.exp(2 * rng.standard_normal((2, 2, n))).astype(np.float32)
    run_select(w, [n, n - 3], budget, sinks, recent)


@pytest.mark.parametrize("kind", ["equal", "special"])
def test_select_ties_past_a_cluster(kind):
    n = 400003
    rng = np.random.default_rng(15)
    w = (np.full((1, 2, n), 0.5) if kind == "equal" else
         rng.choice([np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-42, -1e-42, 1.0, 3.4e38], (1, 2, n)))
    for budget in (1, n // 3, n - 1):
        run_select(np.ascontiguousarray(w, dtype=np.float32), [n], budget, min(2, budget // 2), min(5, budget // 2))


def test_select_forced_rows_fill_the_budget():
    w = np.random.default_rng(6).random((2, 2, 400)).astype(np.float32)
    run_select(w, [400, 21], 20, 13, 7)
    run_select(w, [400, 21], 20, 20, 0)
    run_select(w, [400, 21], 20, 0, 20)


def test_select_lengths_zero_one_and_past_the_row():
    w = np.random.default_rng(7).random((5, 2, 50)).astype(np.float32)
    run_select(w, [0, 1, 2, 50, 3], 2)
    run_select(w, [0, 51, -1, 50, 3], 2, err=pkv.DEVERR_LENGTH)


def test_select_view_of_wider_rows_and_odd_stride():
    w = torch.rand(3, 2, 333, device="cuda")[:, :, :300]
    run_select(w, [300, 299, 7], 100, 3, 9)


def test_select_many_rows():
    w = np.random.default_rng(8).random((400, 4, 120)).astype(np.float32)
    run_select(w, np.random.default_rng(8).integers(0, 121, 400).tolist(), 50, 2, 10)


def test_select_graph_and_given_outputs():
    w = torch.rand(2, 2, 3000, device="cuda")
    lens = torch.tensor([3000, 1700], dtype=torch.int32, device="cuda")
    keep = torch.empty(2, 2, 700, dtype=torch.int32, device="cuda")
    new = torch.empty(2, dtype=torch.int32, device="cuda")
    pkv.kv_evict_select(w, lens, 700, num_sinks=3, num_recent=40, keep=keep, new_lens=new)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.kv_evict_select(w, lens, 700, num_sinks=3, num_recent=40, keep=keep, new_lens=new)
    w.copy_(torch.rand(2, 2, 3000, device="cuda"))
    keep.fill_(9)
    g.replay()
    torch.cuda.synchronize()
    want, _ = select_plain(w.cpu().numpy(), lens.cpu().numpy(), 700, 3, 40)
    assert np.array_equal(keep.cpu().numpy(), want)


# ---------------------------------------------------------------- compaction
def compact_plain(cache, raw, keep, keep_lens, base):
    """The moves on host copies of the pools' bytes (bf16 and fp32)."""
    out = []
    for x in raw:
        x = x.reshape(-1, cache.hkv, cache.d)
        y = x.copy()
        for r in range(len(cache.lens)):
            for h in range(cache.hkv):
                ks = keep[r, h if keep.shape[1] > 1 else 0, :keep_lens[r]]
                src = cache.slots(r, base[r] + ks)
                dst = cache.slots(r, base[r] + np.arange(len(ks)))
                y[dst, h] = x[src, h]
        out.append(y)
    return out


def compact_plain_mx(cache, raw, keep, keep_lens, base):
    out = []
    for x in raw:
        n = x.size // 33 * 32
        y = x.copy()
        e0, e1 = x[:n].reshape(-1, cache.hkv, cache.d), y[:n].reshape(-1, cache.hkv, cache.d)
        s0 = x[n:].reshape(-1, cache.hkv, cache.p, cache.d // 32)
        s1 = y[n:].reshape(-1, cache.hkv, cache.p, cache.d // 32)
        for r in range(len(cache.lens)):
            for h in range(cache.hkv):
                ks = keep[r, h if keep.shape[1] > 1 else 0, :keep_lens[r]]
                src = cache.slots(r, base[r] + ks)
                dst = cache.slots(r, base[r] + np.arange(len(ks)))
                e1[dst, h] = e0[src, h]
                s1[dst // cache.p, h, dst % cache.p] = s0[src // cache.p, h, src % cache.p]
        out.append(y)
    return out


class Compact:
    def __init__(self, lens, kept, *, per_head=True, base=None, dtype="bf16", hkv=2, d=64, p=16, seed=0,
                 weights=True, pad=3, pattern="random", first_block=0):
        self.cache = su.Cache(lens, dtype=dtype, hkv=hkv, d=d, p=p, seed=seed, first_block=first_block)
        rng = np.random.default_rng(seed + 1)
        b = len(lens)
        self.base = np.zeros(b, np.int32) if base is None else np.asarray(base, np.int32)
        self.has_base = base is not None
        self.keep_lens = np.asarray(kept, np.int32)
        self.keep = np.full((b, hkv if per_head else 1, max(kept) + pad), -7, np.int32)
        for r in range(b):
            room = lens[r] - self.base[r]
            for h in range(self.keep.shape[1]):
                n = kept[r]
                if pattern == "random":
                    ks = np.sort(rng.permutation(room)[:n])
                elif pattern == "last":
                    ks = np.arange(room - n, room)
                elif pattern == "first":
                    ks = np.arange(n)
                else:  # a few early rows, then the last ones
                    ks = np.concatenate([np.arange(n // 2), np.arange(room - (n - n // 2), room)])
                self.keep[r, h, :n] = ks
        self.w = torch.rand(b, hkv, max(lens) + 4, device="cuda") if weights else None

    def call(self, **kw):
        c = self.cache
        pkv.kv_compact(c.k, c.v, c.tables, torch.tensor(c.lens, dtype=torch.int32, device="cuda"),
                       torch.from_numpy(self.keep).cuda(), torch.from_numpy(self.keep_lens).cuda(),
                       base_lens=torch.from_numpy(self.base).cuda() if self.has_base else None,
                       weights=self.w, **kw)

    def run(self):
        c = self.cache
        raw = c.raw()
        w0 = self.w.cpu().numpy().copy() if self.w is not None else None
        self.call()
        assert pkv.get_device_error() == 0
        plain = compact_plain_mx if c.dtype == "mxfp8" else compact_plain
        want = plain(c, raw, self.keep, self.keep_lens, self.base)
        for got, ref in zip(c.raw(), want):
            assert np.array_equal(got.reshape(-1), ref.reshape(-1))
        if self.w is not None:
            ref = w0.copy()
            for r, t in enumerate(c.lens):
                for h in range(c.hkv):
                    n, b0 = self.keep_lens[r], self.base[r]
                    ks = self.keep[r, h if self.keep.shape[1] > 1 else 0, :n]
                    ref[r, h, b0:b0 + n] = w0[r, h, b0 + ks]
                    ref[r, h, b0 + n:t] = 0
            assert np.array_equal(self.w.cpu().numpy(), ref)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "mxfp8"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("per_head", [True, False])
def test_compact_types(dtype, d, per_head):
    Compact([100, 1, 0, 33, 500], [50, 1, 0, 32, 499], dtype=dtype, d=d, hkv=3, per_head=per_head,
            seed=d).run()


@pytest.mark.parametrize("p", [1, 5, 16, 48, 256])
def test_compact_block_sizes(p):
    Compact([300, 5 * p, p], [120, 4 * p, 1], p=p, seed=p).run()


@pytest.mark.parametrize("pattern", ["random", "last", "first", "ends"])
@pytest.mark.parametrize("weights", [True, False])
def test_compact_patterns(pattern, weights):
    # "last" shifts every row by the same distance, one row among them
    for cut in (1, 2, 15, 700):
        Compact([3000, 901], [3000 - cut, 901 - cut], pattern=pattern, weights=weights, d=128,
                seed=cut).run()


@pytest.mark.parametrize("d", [8, 24, 96, 512])
def test_compact_head_dims(d):
    Compact([200, 77], [90, 40], d=d, hkv=2, seed=d).run()


def test_compact_accepted_paths():
    rng = np.random.default_rng(3)
    base = rng.integers(0, 200, 40)
    n = rng.integers(1, 65, 40)
    acc = [int(rng.integers(0, m + 1)) for m in n]
    Compact((base + n).tolist(), acc, base=base, per_head=False, d=128, hkv=4, weights=False,
            seed=3).run()
    Compact((base + n).tolist(), acc, base=base, per_head=True, d=128, hkv=4, seed=3).run()


def test_compact_to_nothing_clears_the_scores():
    for pad in (0, 2):  # a list with no room, and one of which nothing is used
        Compact([50, 7], [0, 0], pad=pad, seed=11).run()
        Compact([50, 7], [0, 0], pad=pad, base=[20, 7], seed=11).run()


def test_compact_long():
    Compact([40000, 12345], [17000, 12000], d=128, hkv=2, seed=4).run()


def test_compact_pool_past_2_31_elements():
    c = Compact([300, 77], [100, 60], d=128, hkv=8, seed=5, first_block=2**31 // (16 * 8 * 128) + 5)
    k0 = [c.cache.rows64(r, t) for r, t in enumerate(c.cache.lens)]
    c.call()
    assert pkv.get_device_error() == 0
    for r, n in enumerate(c.keep_lens):
        for x, x0 in zip(c.cache.rows64(r, n), k0[r]):
            for h in range(8):
                assert np.array_equal(x[:, h], x0[c.keep[r, h, :n], h])


def test_compact_refuses_bad_lists():
    for bad in ("high", "order", "equal", "negative", "low"):
        c = Compact([200, 60], [50, 20], seed=6, pattern="last", weights=False)
        row = c.keep[0, 1]
        row[10] = {"high": 200, "order": row[9] - 1, "equal": row[9], "negative": -1, "low": 9}[bad]
        raw = c.cache.raw()
        c.call()
        assert pkv.get_device_error() == pkv.DEVERR_KEEP, bad
        # the other head and the other sequence are as ever, and so are the
        # rows of the bad list up to the bad entry
        want = compact_plain(c.cache, raw, np.clip(c.keep, 0, 199), c.keep_lens, c.base)
        for got, ref in zip(c.cache.raw(), want):
            got, ref = got.reshape(ref.shape), ref
            for r, n in enumerate(c.keep_lens):
                s = c.cache.slots(r, np.arange(n))
                assert np.array_equal(got[s, 0], ref[s, 0])
                s = s if r else s[:10]
                assert np.array_equal(got[s, 1], ref[s, 1])


def test_compact_refuses_bad_lengths():
    for case in range(6):
        c = Compact([200, 60, 90], [50, 20, 30], base=[0, 10, 5], seed=7)
        raw, w0 = c.cache.raw(), c.w.clone()
        lens = list(c.cache.lens)
        if case == 0:
            c.keep_lens[1] = -1
        elif case == 1:
            c.keep_lens[1] = 51  # base 10 + 51 > 60, and within the list's width
        elif case == 2:
            c.base[1] = -1
        elif case == 3:
            c.base[1] = 61
        elif case == 4:
            c.keep_lens[1] = c.keep.shape[2] + 1
        else:
            c.w = w0 = c.w[:, :, :199].contiguous()  # shorter than sequence 0
        skip = 0 if case == 5 else 1
        kept = c.keep_lens.copy()
        c.call()
        assert pkv.get_device_error() == pkv.DEVERR_LENGTH, case
        kept[skip] = 0
        want = compact_plain(c.cache, raw, c.keep, kept, np.clip(c.base, 0, None))
        for got, ref in zip(c.cache.raw(), want):
            assert np.array_equal(got.reshape(-1), ref.reshape(-1))
        assert torch.equal(c.w[skip], w0[skip])
        assert lens == c.cache.lens


def test_compact_refuses_a_length_near_the_end_of_32_bits():
    # a table of 2^31 rows, of which the one kept row is in its place already
    k, v = [torch.randn(4, 256, 1, 8, device="cuda").bfloat16() for _ in range(2)]
    k0, v0 = k.clone(), v.clone()
    tables = torch.zeros(1, 2**23, dtype=torch.int32, device="cuda")
    one = torch.ones(1, dtype=torch.int32, device="cuda")
    for n, err in ((2**31 - 2**16, 0), (2**31 - 2**16 + 1, pkv.DEVERR_LENGTH)):
        pkv.kv_compact(k, v, tables, torch.tensor([n], dtype=torch.int32, device="cuda"),
                       torch.zeros(1, 1, 1, dtype=torch.int32, device="cuda"), one)
        assert pkv.get_device_error() == err
    assert torch.equal(k, k0) and torch.equal(v, v0)


def test_compact_bad_block():
    c = Compact([200, 60], [50, 20], seed=8, pattern="last", weights=False)
    good = c.cache.tables_np[0, 1]
    c.cache.tables[0, 1] = c.cache.k.shape[0]
    raw = c.cache.raw()
    c.call()
    assert pkv.get_device_error() == pkv.DEVERR_BLOCK
    want = compact_plain(c.cache, raw, c.keep, c.keep_lens, c.base)
    for got, ref in zip(c.cache.raw(), want):
        got = got.reshape(ref.shape)
        s = np.concatenate([c.cache.slots(0, np.arange(16)), c.cache.slots(0, np.arange(32, 50)),
                            c.cache.slots(1, np.arange(20))])
        assert np.array_equal(got[s], ref[s])
        before = raw[0].reshape(ref.shape)
    s = good * 16 + np.arange(16)
    assert np.array_equal(c.cache.raw()[0].reshape(before.shape)[s], before[s])


def test_compact_twice_captured():
    c = Compact([500], [300], d=128, seed=9, pattern="last")
    keep, kl = torch.from_numpy(c.keep).cuda(), torch.from_numpy(c.keep_lens).cuda()
    lens = torch.tensor(c.cache.lens, dtype=torch.int32, device="cuda")
    raw = c.cache.raw()
    g = torch.cuda.CUDAGraph()
    args = (c.cache.k, c.cache.v, c.cache.tables, lens, keep, kl)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        pkv.kv_compact(*args)
    for _ in range(2):
        g.replay()
        raw = compact_plain(c.cache, raw, c.keep, c.keep_lens, c.base)
        for got, ref in zip(c.cache.raw(), raw):
            assert np.array_equal(got.reshape(-1), ref.reshape(-1))
