"""pkv_draft_tree_attention against a plain 64-bit form: types, head layouts,
lengths, masks, bad data, streams and graphs."""
import numpy as np
import pytest
import torch

from paged_kv_cache_41_gb300 import pkv

import serving_util as su

pytestmark = pytest.mark.gpu


class Draft:
    """Sequences of ctx[r] committed and n[r] drafted rows, and their queries."""

    def __init__(self, ctx, n, masks="tree", *, dtype="bf16", hq=4, hkv=2, d=64, p=16, seed=0,
                 lead=0, trail=0, width=None, first_block=0):
        self.ctx, self.n, self.hq = list(ctx), list(n), hq
        self.cache = su.Cache([c + m for c, m in zip(ctx, n)], dtype=dtype, hkv=hkv, d=d, p=p,
                              seed=seed, width=width, first_block=first_block)
        rng = np.random.default_rng(seed + 1)
        self.words = []
        for m in n:
            if masks == "tree":
                self.words.append(su.tree_masks(m, rng))
            elif masks == "chain":
                self.words.append([(2 << i) - 1 for i in range(m)])
            elif masks == "random":  # any bits, those past n among them
                self.words.append([int(rng.integers(0, 1 << 63)) | (int(rng.integers(0, 2)) << 63)
                                   for _ in range(m)])
            else:
                self.words.append([masks] * m)
        self.ptr_np = lead + np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        self.rows = int(self.ptr_np[-1]) + trail
        self.q = self.cache.randn(self.rows, hq, d)
        flat = [w for ws in self.words for w in ws]
        self.masks = None if masks == "chain" else su.as_int64([0] * lead + flat + [0] * trail).cuda()
        self.ctx_t = torch.tensor(self.ctx, dtype=torch.int32, device="cuda")
        self.ptr = torch.from_numpy(self.ptr_np).cuda()
        self.max_draft = max(list(n) + [1])
        self.scale = su.softmax_scale(d)

    def call(self, out=None, lse=None, **kw):
        c = self.cache
        lse = torch.full((self.rows, self.hq), 77.0, device="cuda") if lse is None else lse
        out = torch.full_like(self.q, 77.0) if out is None else out
        kw = {"max_draft": self.max_draft, **kw}
        pkv.draft_tree_attention(self.q, c.k, c.v, c.tables, self.ctx_t, self.ptr, self.scale,
                                 masks=self.masks, out=out, lse=lse, **kw)
        return out, lse

    def check(self, out, lse, skip=()):
        """Against the plain form; rows of no sequence (or of skipped ones) untouched."""
        c = self.cache
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        q = self.q.double().cpu().numpy()
        mine = np.zeros(self.rows, bool)
        for r, (ctx, n) in enumerate(zip(self.ctx, self.n)):
            if n == 0 or r in skip:
                continue
            a, b = self.ptr_np[r], self.ptr_np[r + 1]
            mine[a:b] = True
            k, v = c.rows64(r, ctx + n)
            seen = np.ones((n, ctx + n), bool)
            seen[:, ctx:] = [[(w >> j) & 1 for j in range(n)] for w in self.words[r]]
            g = self.hq // c.hkv
            for h in range(self.hq):
                o, l, _, absv, mag = su.attend64(q[a:b, h], k[:, h // g], v[:, h // g], seen,
                                                 self.scale)
                su.check_attention(c.dtype, c.d, out[a:b, h], lse[a:b, h], o, l, absv, mag,
                                   ctx + n, f"sequence {r} head {h}",
                                   p_bits=0.0 if c.dtype == "f32" else 2.0 ** -8)
        assert (out[~mine] == 77.0).all() and (lse[~mine] == 77.0).all()

    def run(self, **kw):
        out, lse = self.call(**kw)
        assert pkv.get_device_error() == 0
        self.check(out, lse)


CTX = [0, 1, 15, 16, 17, 100, 127, 128, 129, 300, 0, 640]
N = [1, 64, 2, 16, 3, 0, 7, 1, 33, 20, 5, 63]


@pytest.mark.parametrize("dtype", ["bf16", "f32", "mxfp8"])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 2), (4, 2), (8, 2), (16, 2)])
@pytest.mark.parametrize("d", [64, 128])
def test_types_and_heads(dtype, hq, hkv, d):
    Draft(CTX, N, dtype=dtype, hq=hq, hkv=hkv, d=d, seed=hq + d).run()


@pytest.mark.parametrize("p", [16, 32, 64, 96, 128, 160, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f32", "mxfp8"])
def test_block_sizes(p, dtype):
    Draft([p - 1, 3 * p + 5, 0, 700, 2 * p], [2, 64, p % 60 + 1, 9, 30], dtype=dtype, p=p, d=128,
          hq=8, hkv=2, seed=p).run()


@pytest.mark.parametrize("masks", ["chain", "tree", "random", 0, (1 << 64) - 1])
@pytest.mark.parametrize("dtype", ["bf16", "f32", "mxfp8"])
def test_masks(masks, dtype):
    Draft([0, 5, 64, 200, 127], [3, 64, 31, 17, 2], masks, dtype=dtype, hq=8, hkv=2, d=128,
          seed=3).run()


@pytest.mark.parametrize("n", [1, 2, 4, 8, 16, 17, 32, 33, 64])
@pytest.mark.parametrize("dtype", ["bf16", "mxfp8"])
def test_draft_lengths(n, dtype):
    # every sequence alike: one to eight row tiles of the largest group
    Draft([250, 0, 1000], [n] * 3, dtype=dtype, hq=16, hkv=2, d=128, seed=n).run()


@pytest.mark.parametrize("dtype", ["bf16", "mxfp8"])
def test_one_sequence_many_splits(dtype):
    Draft([9001], [13], dtype=dtype, hq=8, hkv=2, d=128, seed=5).run()


@pytest.mark.parametrize("dtype", ["bf16", "f32", "mxfp8"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,n", [(1, 1), (2, 7), (8, 17), (8, 64)])
def test_one_long_segment(dtype, d, hq, n):
    # every CTA holds a piece of it
    Draft([20011], [n], dtype=dtype, hq=hq, hkv=1, d=d, seed=9 + n).run()


def test_many_sequences():
    rng = np.random.default_rng(6)
    Draft(rng.integers(0, 400, 300), rng.integers(0, 9, 300), hq=4, hkv=1, d=64, seed=6).run()


def test_ordinary_batch():
    rng = np.random.default_rng(7)
    Draft(rng.integers(512, 3000, 10), rng.integers(5, 28, 10), hq=32, hkv=8, d=128, seed=7).run()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_of_no_sequence_are_left(dtype):
    # query rows before the first sequence and behind the last, and a table
    # wider than any sequence needs
    Draft([40, 0, 129], [3, 0, 20], dtype=dtype, lead=5, trail=7, width=64, seed=8).run()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("ctx", [0, 50, 120, 128])
def test_hidden_rows_with_nan_and_inf(dtype, value, ctx):
    # drafted row 2 holds the value in K and V: its descendants see it, its
    # siblings must not
    dr = Draft([ctx], [12], dtype=dtype, hq=8, hkv=2, d=128, seed=9)
    words = [1 | 1 << i for i in range(12)]
    words[5] |= 4
    words[7] |= 4 | 32
    words[2] = 1  # not even itself
    dr.words = [words]
    dr.masks = su.as_int64(words).cuda()
    slot = int(dr.cache.slots(0, [ctx + 2])[0])
    dr.cache.v.view(-1, 2, 128)[slot, :, 3:40] = value
    out, lse = dr.call()
    assert pkv.get_device_error() == 0
    dr.check(out, lse)
    dr.cache.k.view(-1, 2, 128)[slot, :, 9] = value
    out, lse = dr.call()
    torch.cuda.synchronize()
    hidden = [i for i in range(12) if not words[i] & 4]
    assert torch.isfinite(out[hidden].float()).all() and torch.isfinite(lse[hidden]).all()
    ref = Draft([ctx], [12], dtype=dtype, hq=8, hkv=2, d=128, seed=9)
    ref.masks = dr.masks
    want, want_lse = ref.call()
    assert torch.equal(out[hidden], want[hidden]) and torch.equal(lse[hidden], want_lse[hidden])
    seers = [5, 7]
    if value != value:
        assert torch.isnan(out[seers].float()).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ctx", [3, 60, 125])
def test_nan_codes_of_a_quantized_pool(d, ctx):
    # drafted row 2 holds NaN codes: whoever sees it gets NaN there, nobody else
    dr = Draft([ctx], [9], dtype="mxfp8", hq=8, hkv=2, d=d, seed=21)
    words = [1 | 1 << i for i in range(9)]
    words[6] |= 4
    words[2] = 1
    dr.words, dr.masks = [words], su.as_int64(words).cuda()
    want, want_lse = dr.call()
    slot = int(dr.cache.slots(0, [ctx + 2])[0])
    dr.cache.v.elements.view(-1, 2, d)[slot, :, 5:40:3] = 0x7F
    dr.cache.v.elements.view(-1, 2, d)[slot, :, 6] = 0xFF
    out, lse = dr.call()
    assert pkv.get_device_error() == 0
    dr.check(out, lse)
    dr.cache.k.elements.view(-1, 2, d)[slot, 1, 9] = 0x7F
    out, lse = dr.call()
    hidden = [i for i in range(9) if i != 6]
    assert torch.equal(out[hidden], want[hidden]) and torch.equal(lse[hidden], want_lse[hidden])
    assert torch.isnan(out[6, 4:].float()).all() and torch.isnan(lse[6, 4:]).all()
    # in the context every row sees them
    dr.cache.v.elements.view(-1, 2, d)[int(dr.cache.slots(0, [0])[0]), :, 1] = 0x7F
    out, _ = dr.call()
    assert torch.isnan(out[:, :, 1].float()).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32", "mxfp8"])
def test_large_scores(dtype):
    # scores far apart: the running maximum moves in every tile
    dr = Draft([700, 3], [9, 9], dtype=dtype, hq=4, hkv=2, d=64, seed=10)
    dr.q *= 12
    dr.run()


def test_negative_and_zero_scale():
    for scale in (-0.3, 0.0):
        dr = Draft([300], [9], "tree", hq=4, hkv=2, d=64, seed=11)
        dr.scale = scale
        out, lse = dr.call()
        dr.scale = abs(scale)
        dr.q = -dr.q if scale < 0 else dr.q
        dr.check(out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_ranges_set_the_error_and_skip(dtype):
    dr = Draft([40, 30, 20, 10, 16], [4, 5, 6, 7, 3], dtype=dtype, seed=12)
    good = dr.ptr.clone(), dr.ctx_t.clone()
    for case in range(5):
        dr.ptr, dr.ctx_t = good[0].clone(), good[1].clone()
        skip = {1}
        if case == 0:
            dr.ctx_t[1] = -1
        elif case == 1:
            dr.ctx_t[1] = dr.cache.max_blocks * 16 - 4
        elif case == 2:
            dr.ptr[1], skip = 10, {0, 1}  # 0 has ten rows (> max_draft 7), 1 a descending range
        elif case == 3:
            dr.ptr[5], skip = dr.rows + 1, {4}
        else:
            dr.ctx_t[1] = 2**31 - 1
        out, lse = dr.call()
        assert pkv.get_device_error() == pkv.DEVERR_LENGTH, case
        dr.check(out, lse, skip=skip)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "mxfp8"])
def test_bad_block_sets_the_error(dtype):
    dr = Draft([200, 30], [4, 5], dtype=dtype, seed=13)
    for bad in (-1, dr.cache.k.shape[0], 2**31 - 1):
        dr.cache.tables[0, 3] = bad
        dr.call()
        assert pkv.get_device_error() == pkv.DEVERR_BLOCK
    out, _ = dr.call()
    pkv.get_device_error()
    want, _ = Draft([200, 30], [4, 5], dtype=dtype, seed=13).call()
    a, b = dr.ptr_np[1], dr.ptr_np[2]
    assert torch.equal(out[a:b], want[a:b])  # the other sequence is as ever


def test_pool_past_2_31_elements():
    # block ids whose element offsets pass 2^31 (and byte offsets 2^32)
    Draft([300, 77], [9, 4], hq=16, hkv=8, d=128, p=16, seed=14, first_block=2**31 // (16 * 8 * 128) + 5).run()


def test_repeats_are_bit_identical():
    dr = Draft([5000, 700, 64], [13, 30, 2], hq=32, hkv=8, d=128, seed=15)
    out, lse = dr.call()
    for _ in range(3):
        o, l = dr.call()
        assert torch.equal(o, out) and torch.equal(l, lse)


def test_side_stream_and_own_workspace():
    dr = Draft([900, 40], [8, 8], hq=8, hkv=2, d=128, seed=16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ws = torch.empty(pkv.draft_tree_workspace_bytes(dr.cache.k, 2, 8, 8, dr.cache.max_blocks),
                     dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF)
    out, lse = torch.full_like(dr.q, 77.0), torch.full((dr.rows, 8), 77.0, device="cuda")
    torch.cuda.synchronize()
    dr.call(out=out, lse=lse, workspace=ws, stream=s)
    s.synchronize()
    dr.check(out, lse)


def test_two_streams_at_once():
    a = Draft([3000, 40], [8, 8], hq=8, hkv=2, d=128, seed=17)
    b = Draft([10, 2500], [64, 5], hq=8, hkv=2, d=128, seed=18)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    got = [(torch.full_like(x.q, 77.0), torch.full((x.rows, 8), 77.0, device="cuda")) for x in (a, b)]
    ws = [torch.empty(pkv.draft_tree_workspace_bytes(x.cache.k, 2, 8, x.max_draft, x.cache.max_blocks),
                      dtype=torch.uint8, device="cuda") for x in (a, b)]
    torch.cuda.synchronize()
    for _ in range(5):
        for x, s, (o, l), w in zip((a, b), (sa, sb), got, ws):
            x.call(out=o, lse=l, workspace=w, stream=s)
    torch.cuda.synchronize()
    for x, (o, l) in zip((a, b), got):
        x.check(o, l)


def test_graph_replay_follows_its_inputs():
    dr = Draft([500, 64, 0], [7, 16, 2], hq=8, hkv=2, d=128, seed=19)
    out, lse = torch.full_like(dr.q, 77.0), torch.full((dr.rows, 8), 77.0, device="cuda")
    ws = torch.empty(pkv.draft_tree_workspace_bytes(dr.cache.k, 3, 8, 16, dr.cache.max_blocks),
                     dtype=torch.uint8, device="cuda")
    dr.call(out=out, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dr.call(out=out, lse=lse, workspace=ws)
    dr.q.copy_(dr.cache.randn(*dr.q.shape))
    dr.ctx_t[0] -= 3  # shorter: the drafted rows are read three rows earlier
    dr.ctx[0] -= 3
    ws.fill_(0xFF)
    out.fill_(77.0)
    g.replay()
    torch.cuda.synchronize()
    dr.check(out, lse)
    other, _ = dr.call()  # an eager call beside the live graph
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, other)


def test_chain_of_one_equals_the_decode():
    # a single drafted token that sees itself: the decode of its sequence
    dr = Draft([1000, 31, 8], [1, 1, 1], "chain", hq=8, hkv=2, d=128, seed=20)
    out, lse = dr.call()
    lens = dr.ctx_t + 1
    want_lse = torch.empty_like(lse)
    want = pkv.paged_attention_decode(dr.q, dr.cache.k, dr.cache.v, dr.cache.tables, lens, dr.scale,
                                      lse=want_lse)
    # both are held to the bounds against 64 bits elsewhere; here they must
    # agree to one bf16 step of each plus the rounded weights' half step
    dr.check(out, lse)
    dr.check(want, want_lse)
