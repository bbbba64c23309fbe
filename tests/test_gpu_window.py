"""pkv_paged_attention_decode_window against a plain 64-bit form: types, head
layouts, windows and sinks around every border, released blocks, streams and
graphs."""
import numpy as np
import pytest
import torch

from paged_kv_cache_41_gb300 import pkv

import serving_util as su

pytestmark = pytest.mark.gpu


class Window:
    """A cache whose hidden blocks are released (-1) and whose hidden rows in blocks
    that are held are NaN."""

    def __init__(self, lens, window, sinks, *, dtype="bf16", hq=4, hkv=2, d=64, p=16, seed=0, width=None,
                 first_block=0, release=True):
        self.c = c = su.Cache(lens, dtype=dtype, hkv=hkv, d=d, p=p, seed=seed, width=width, first_block=first_block)
        self.lens, self.window, self.sinks, self.hq = list(lens), window, sinks, hq
        self.q = c.randn(len(lens), hq, d)
        self.seen = [np.array([t < sinks or t >= n - window for t in range(n)], bool) for n in lens]
        self.k64, self.v64 = [], []
        for r, n in enumerate(lens):
            k, v = c.rows64(r, n)
            self.k64.append(k)
            self.v64.append(v)
        tables = c.tables_np.copy()
        dead = [int(s) for r, n in enumerate(lens) for s in c.slots(r, np.nonzero(~self.seen[r])[0])]
        if dead:
            at = torch.tensor(dead, device="cuda")
            for pool in (c.k, c.v):
                if dtype == "mxfp8":
                    pool.elements.view(-1, hkv, d)[at] = 0x7F
                else:
                    pool.view(-1, hkv, d)[at] = float("nan")
        if release:
            for r, n in enumerate(lens):
                for j in range(-(-n // p)):
                    if not self.seen[r][j * p:(j + 1) * p].any():
                        tables[r, j] = -1
        self.tables = torch.from_numpy(tables).cuda()
        self.lens_t = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.scale = su.softmax_scale(d)

    def call(self, **kw):
        out = torch.full_like(self.q, 77.0)
        lse = torch.full((len(self.lens), self.hq), 77.0, device="cuda")
        kw = {"out": out, "lse": lse, "window": self.window, "num_sinks": self.sinks, **kw}
        pkv.paged_attention_decode_window(self.q, self.c.k, self.c.v, self.tables, self.lens_t, self.scale, **kw)
        return kw["out"], kw["lse"]

    def check(self, out, lse):
        c = self.c
        out, lse = out.double().cpu().numpy(), None if lse is None else lse.double().cpu().numpy()
        q = self.q.double().cpu().numpy()
        g = self.hq // c.hkv
        for r, n in enumerate(self.lens):
            for h in range(self.hq):
                # the tensor-core decode rounds a weight to two bf16 terms
                o, l, _, absv, mag = su.attend64(q[r:r + 1, h], self.k64[r][:, h // g], self.v64[r][:, h // g],
                                                 self.seen[r][None], self.scale)
                su.check_attention(c.dtype, c.d, out[r:r + 1, h], None if lse is None else lse[r:r + 1, h], o, l,
                                   absv, mag, max(n, 1), f"sequence {r} ({n} rows) head {h}",
                                   p_bits=2.0 ** -16 if g == 8 and c.dtype != "f32" else 0.0)

    def run(self, **kw):
        out, lse = self.call(**kw)
        assert pkv.get_device_error() == 0
        self.check(out, lse)


LENS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 100, 127, 128, 129, 200, 257, 500, 1000]


@pytest.mark.parametrize("dtype", ["bf16", "f32", "mxfp8"])
@pytest.mark.parametrize("hq,hkv,d", [(1, 1, 64), (2, 1, 128), (4, 2, 64), (8, 2, 128), (16, 2, 128), (8, 1, 64)])
def test_types_and_heads(dtype, hq, hkv, d):
    if dtype == "mxfp8" and hq == 8 * hkv and d == 64:
        pytest.skip("refused: MXFP8 with eight query heads per kv head takes head_dim 128")
    Window(LENS, 50, 5, dtype=dtype, hq=hq, hkv=hkv, d=d, seed=hq).run()


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 31, 32, 33, 100, 127, 128, 129, 256, 999, 1000, 2**31 - 1])
@pytest.mark.parametrize("sinks", [0, 1, 4, 16, 17, 32, 40, 128, 130])
@pytest.mark.parametrize("heads", [(4, 2, "bf16", 64), (16, 2, "bf16", 128)])
def test_windows_and_sinks(window, sinks, heads):
    hq, hkv, dtype, d = heads
    Window(LENS, window, sinks, dtype=dtype, hq=hq, hkv=hkv, d=d, seed=window % 97).run()


@pytest.mark.parametrize("window,sinks", [(1, 0), (17, 3), (128, 16), (130, 40), (300, 129)])
@pytest.mark.parametrize("hq,d", [(4, 64), (8, 128), (16, 128)])
def test_windows_over_mxfp8(window, sinks, hq, d):
    Window(LENS, window, sinks, dtype="mxfp8", hq=hq, hkv=2, d=d, seed=window).run()


@pytest.mark.parametrize("p", [16, 32, 64, 96, 128, 160, 256])
@pytest.mark.parametrize("hq,dtype,d", [(4, "bf16", 64), (16, "bf16", 128), (4, "f32", 128), (4, "mxfp8", 64),
                                        (16, "mxfp8", 128)])
def test_block_sizes(p, hq, dtype, d):
    if dtype == "mxfp8" and hq == 16 and p in (96, 160):
        pytest.skip("refused: MXFP8 with eight query heads per kv head takes powers of two")
    for window, sinks in ((1, 1), (p, p), (p + 1, p - 1), (3 * p - 5, 2)):
        Window([1, p - 1, p, p + 1, 3 * p + 5, 700, 5 * p], window, sinks, dtype=dtype, hq=hq, hkv=2, d=d, p=p,
               seed=p).run()


@pytest.mark.parametrize("hq,dtype", [(4, "bf16"), (8, "bf16"), (16, "bf16"), (16, "mxfp8"), (8, "f32")])
def test_large_batches(hq, dtype):
    # many pieces a CTA: short windows, ends of pieces at every stage
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 700, 300)
    Window(lens, 90, 20, dtype=dtype, hq=hq, hkv=2, d=128, seed=9).run()


def test_more_sequences_than_a_scan_takes():
    rng = np.random.default_rng(6)
    Window(rng.integers(0, 120, 2200), 40, 3, hq=1, hkv=1, d=64, seed=3).run()


@pytest.mark.parametrize("hq", [4, 16])
def test_long_sequences_are_split(hq):
    Window([30000, 100, 20001], 10000, 64, hq=hq, hkv=2, d=128, seed=hq).run()


@pytest.mark.parametrize("dtype,hq", [("bf16", 4), ("bf16", 16), ("f32", 4), ("mxfp8", 16)])
def test_a_window_over_everything_is_the_decode(dtype, hq):
    w = Window([1, 50, 333, 1000], 1000, 0, dtype=dtype, hq=hq, hkv=2, d=128)
    out, lse = w.call()
    lse2 = torch.empty_like(lse)
    plain = pkv.paged_attention_decode(w.q, w.c.k, w.c.v, w.c.tables, w.lens_t, w.scale, lse=lse2)
    w.check(out, lse)
    w.check(plain, lse2)


def test_lengths_that_make_no_sense():
    for hq in (4, 16):
        w = Window([40, 70, 500], 30, 4, hq=hq, hkv=2, d=128)
        good, glse = w.call()
        w.lens_t = torch.tensor([-5, 70, 2**31 - 1], dtype=torch.int32, device="cuda")
        out, lse = w.call()
        assert pkv.get_device_error() & pkv.DEVERR_LENGTH
        assert (out[0] == 0).all() and (lse[0] == float("-inf")).all()
        assert torch.equal(out[1], good[1])


@pytest.mark.parametrize("hq,dtype", [(4, "bf16"), (16, "bf16"), (16, "mxfp8"), (4, "mxfp8"), (4, "f32")])
def test_bad_blocks_under_the_window_are_named(hq, dtype):
    w = Window([200, 333], 60, 4, dtype=dtype, hq=hq, hkv=2, d=128)
    good, _ = w.call()
    assert pkv.get_device_error() == 0
    w.tables[1, 333 // 16] = w.c.k.shape[0] + 5
    out, _ = w.call()
    assert pkv.get_device_error() == pkv.DEVERR_BLOCK
    assert torch.equal(out[0], good[0])


def test_without_lse_and_with_a_workspace_of_its_own():
    w = Window(LENS, 60, 4)
    out, _ = w.call(lse=None)
    w.check(out, None)
    n = pkv.decode_window_workspace_bytes(w.c.k, len(LENS), 4, w.tables.shape[1], 60, 4)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    w.run(workspace=ws)


def test_two_graphs_at_once_and_a_side_stream():
    ws = [Window(LENS, 60, 4, hq=4, seed=1), Window(LENS[::-1], 100, 17, hq=16, d=128, seed=2)]
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in ws]
    for w, st in zip(ws, streams):
        w.call()
        n = pkv.decode_window_workspace_bytes(w.c.k, len(LENS), w.hq, w.tables.shape[1], w.window, w.sinks)
        work = torch.empty(n, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=st):
                outs.append(w.call(workspace=work))
        graphs.append((g, work))
    torch.cuda.synchronize()
    for _ in range(5):
        for (g, _), st, (o, l) in zip(graphs, streams, outs):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert pkv.get_device_error() == 0
    for w, (o, l) in zip(ws, outs):
        w.check(o, l)
    # an eager call on a side stream, its memory its own
    side = torch.cuda.Stream()
    w = ws[0]
    out = pkv.paged_attention_decode_window(w.q, w.c.k, w.c.v, w.tables, w.lens_t, w.scale, window=w.window,
                                            num_sinks=w.sinks, stream=side)
    side.synchronize()
    w.check(out, None)


def test_large_offsets():
    # blocks past 2^31 elements of the pool
    first = 2**31 // (16 * 8 * 128) + 10
    for hq in (32, 64):
        Window([300, 40], 50, 4, hq=hq, hkv=8, d=128, first_block=first).run()


def test_the_scores_of_hidden_rows_do_not_matter():
    # infinities in hidden rows of blocks that are read
    w = Window([100, 290], 37, 5, dtype="f32", release=False)
    bad = torch.isnan(w.c.k)
    good, _ = w.call()
    w.c.k[bad] = float("inf")
    w.c.v[bad] = float("-inf")
    out, lse = w.call()
    assert torch.equal(out, good)
    w.check(out, lse)


@pytest.mark.parametrize("hq,d", [(1, 64), (4, 128), (8, 128)])
def test_scales_and_codes_at_the_ends_of_mxfp8(hq, d):
    # K scales of 2^-127, V scales past 2^7 (up to 2^14) in single groups: the ones
    # that chunks of rows without them do not pay for
    w = Window([5, 40, 64, 300], 120, 3, dtype="mxfp8", hq=hq, hkv=1, d=d, seed=hq)
    rng = np.random.default_rng(d)
    for pool, bytes_ in ((w.c.k, [0]), (w.c.v, [134, 135, 141])):
        scales = pool.scales.view(-1)
        at = torch.from_numpy(rng.choice(scales.numel(), scales.numel() // 12, replace=False)).cuda()
        scales[at] = torch.from_numpy(rng.choice(bytes_, at.numel())).to(torch.uint8).cuda()
    w.k64, w.v64 = zip(*(w.c.rows64(r, n) for r, n in enumerate(w.lens)))
    w.run()
    # a NaN code in a row that is seen: its column of V, every column by K
    good, _ = w.call()
    row = int(w.c.slots(3, np.array([250]))[0])
    v, k = w.c.v.elements.view(-1, d), w.c.k.elements.view(-1, d)
    was = int(v[row, 37])
    v[row, 37] = 0xFF
    out, _ = w.call()
    assert torch.isnan(out[3, :, 37]).all()
    out[3, :, 37] = good[3, :, 37]
    assert torch.equal(out, good)
    v[row, 37] = was
    k[row, 5] = 0x7F
    out, _ = w.call()
    assert torch.isnan(out[3]).all() and torch.equal(out[:3], good[:3])


@pytest.mark.parametrize("dtype,hq", [("bf16", 1), ("bf16", 8), ("f32", 1), ("f32", 8), ("mxfp8", 8)])
@pytest.mark.parametrize("window,lens", [(120, [5, 300]), (120, [5, 300] + [0] * 400), (2500, [5, 2600])])
def test_nan_scores_stay(dtype, hq, window, lens):
    # one CTA a segment, several, and (fp32) pieces of the balanced split
    w = Window(lens, window, 3, dtype=dtype, hq=hq, hkv=1, d=128, seed=hq)
    good, good_lse = w.call()
    row = int(w.c.slots(1, np.array([lens[1] - 30]))[0])
    if dtype == "mxfp8":
        w.c.k.elements.view(-1, 128)[row, 5] = 0x7F
    else:
        w.c.k.view(-1, 128)[row, 5] = float("nan")
    out, lse = w.call()
    assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()
    assert torch.equal(out[0], good[0]) and torch.equal(lse[0], good_lse[0])
    assert torch.equal(out[2:], good[2:]) and torch.equal(lse[2:], good_lse[2:])
    # every row that is seen
    rows = torch.from_numpy(w.c.slots(0, np.arange(5))).cuda()
    if dtype == "mxfp8":
        w.c.k.elements.view(-1, 128)[rows] = 0x7F
    else:
        w.c.k.view(-1, 128)[rows] = float("nan")
    out, lse = w.call()
    assert torch.isnan(out[:2]).all() and torch.isnan(lse[:2]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window,n", [(120, 300), (2500, 2600)])
def test_scores_of_minus_infinity_weigh_nothing(dtype, window, n):
    w = Window([n, 3], window, 0, dtype=dtype, hq=1, hkv=1, d=64, seed=n)
    w.q[:, 0, 7] = 1.0
    off = np.concatenate([np.arange(n - window, n - window + 70), [n - 20]])
    pool = w.c.k.view(-1, 64)
    pool[torch.from_numpy(w.c.slots(0, off)).cuda(), 7] = float("-inf")
    pool[torch.from_numpy(w.c.slots(1, np.arange(3))).cuda(), 7] = float("-inf")
    w.seen[0][off] = False  # what is left of the formula
    w.seen[1][:] = False
    out, lse = w.call()
    assert pkv.get_device_error() == 0
    w.check(out, lse)
    assert (out[1] == 0).all() and torch.isneginf(lse[1]).all()


@pytest.mark.parametrize("dtype", ["bf16", "mxfp8"])
@pytest.mark.parametrize("hq,hkv,d", [(4, 1, 128), (8, 1, 128), (2, 2, 64), (16, 2, 128)])
@pytest.mark.parametrize("window", [20, 100, 250, 1000, 6000])
def test_segments_of_several_ctas(dtype, hq, hkv, d, window):
    # parts of one cluster, of several, and sequences too short to have them all
    Window([7000, 0, 1, 33, 300, 5000, 255, 257], window, 5, dtype=dtype, hq=hq, hkv=hkv, d=d, seed=window).run()


@pytest.mark.parametrize("dtype", ["bf16", "mxfp8"])
def test_segments_of_several_ctas_in_several_waves(dtype):
    Window([9000] + [40] * 700, 8000, 3, dtype=dtype, hq=4, hkv=1, d=64, seed=5).run()


@pytest.mark.parametrize("dtype", ["bf16", "f32", "mxfp8"])
def test_wide_tables(dtype):
    Window([100, 0, 900] + [20] * 30, 2**31 - 1, 0, dtype=dtype, hq=4, hkv=1, d=64, width=100000, seed=6).run()
