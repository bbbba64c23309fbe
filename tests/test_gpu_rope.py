"""pkv_qk_norm_rope_append against a plain 64-bit form: types, head layouts,
rotated parts, axes, strides, bad data, streams and graphs."""
import numpy as np
import pytest
import torch

from paged_kv_cache_41_gb300 import pkv

import serving_util as su
from step_util import rotate64

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24


def table(rows, rot, base=10000.0):
    half = rot // 2
    angle = np.arange(rows)[:, None] * base ** (-np.arange(half) / half)
    return np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)


class Rope:
    def __init__(self, n, *, dtype="bf16", hq=4, hkv=2, d=64, p=16, rot=None, axes=1, axis_of=None, norm=True,
                 interleaved=False, eps=1e-6, far=1000, pad=0, seed=0, scale=2.0):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.n, self.dtype, self.hq, self.hkv, self.d, self.p = n, dtype, hq, hkv, d, p
        self.rot, self.inter, self.eps = d if rot is None else rot, interleaved, eps
        io = su.IO[dtype]
        heads = hq + 2 * hkv
        # the packed projection, tokens `pad` elements further apart than their heads
        wide = torch.randn(n, heads * d + pad, generator=g, device="cuda") * scale
        self.qkv = wide.to(io)[:, : heads * d]
        self.q, self.k, self.v = (x.unflatten(1, (-1, d)) for x in
                                  self.qkv.split([hq * d, hkv * d, hkv * d], 1))
        self.wq = self.wk = None
        if norm:
            self.wq, self.wk = (torch.randn(d, generator=g, device="cuda") for _ in range(2))
        self.axes = axes
        self.axis_of = axis_of or [j * axes // max(self.rot // 2, 1) for j in range(self.rot // 2)]
        self.pos = rng.integers(0, far, (axes, n)).astype(np.int32)
        self.table = table(far, self.rot) if self.rot else None
        nb = -(-n // p) + 3
        self.slots = rng.permutation(nb * p)[:n].astype(np.int64)
        self.shape = (nb, p, hkv, d)
        if dtype == "mxfp8":
            self.kc, self.vc = (pkv.MxPool(*self.shape, fill=0x55) for _ in range(2))
        else:
            self.kc, self.vc = (torch.full(self.shape, 77.0, dtype=io, device="cuda") for _ in range(2))

    def args(self):
        pos = torch.from_numpy(self.pos if self.axes > 1 else self.pos[0]).cuda()
        return (self.q, self.k, self.v, self.kc, self.vc, torch.from_numpy(self.slots).cuda(), pos,
                torch.from_numpy(self.table).cuda() if self.rot else None)

    def call(self, **kw):
        out = torch.full((self.n, self.hq, self.d), 55.0, dtype=self.q.dtype, device="cuda")
        return pkv.qk_norm_rope_append(*self.args(), **{"q_weight": self.wq, "k_weight": self.wk, "eps": self.eps,
                                                        "axis_of": self.axis_of if self.axes > 1 else None,
                                                        "interleaved": self.inter, "out": out, **kw})

    def check(self, out, live=None, stored=None):
        """live: tokens written at all; stored: those whose K and V are.  The bound,
        in half steps of fp32 relative to the terms that an element is the sum of:
        the sum of squares (a chain of 8, a tree over 16 lanes, mean and eps: 14,
        halved by the root), the inverse root (2 ulp: 4), and the products with
        weight, cosine and sine and their difference (5): 16; then the output's own."""
        n = self.n
        live = np.ones(n, bool) if live is None else live
        stored = live if stored is None else stored
        got = out.double().cpu().numpy()
        y, size = rotate64(self.q.double().cpu().numpy(), None if self.wq is None else self.wq.double().cpu().numpy(),
                           self.eps, self.table, np.where(live, self.pos, 0), self.axis_of, self.inter)
        su.check(got[live], y[live], (16 * U32 * size + su.HALF[self.dtype] * np.abs(y) + 1e-37)[live], "q")
        assert (got[~live] == 55.0).all()
        k, size = rotate64(self.k.double().cpu().numpy(), None if self.wk is None else self.wk.double().cpu().numpy(),
                           self.eps, self.table, np.where(live, self.pos, 0), self.axis_of, self.inter)
        nb, p, hkv, d = self.shape
        at = self.slots[stored]
        other = np.setdiff1d(np.arange(nb * p), at)
        if self.dtype != "mxfp8":
            kc = self.kc.double().cpu().numpy().reshape(-1, hkv, d)
            vc = self.vc.cpu().reshape(-1, hkv, d)
            bound = (16 * U32 * size + su.HALF[self.dtype] * np.abs(k) + 1e-37)[stored]
            su.check(kc[at], k[stored], bound, "k")
            assert torch.equal(vc[torch.from_numpy(at)], self.v.cpu()[torch.from_numpy(stored)])
            assert (kc[other] == 77.0).all() and (vc[torch.from_numpy(other)] == 77.0).all()
            return
        # V as kv_append quantises it; K within half a step of its group's scale
        want = pkv.MxPool(*self.shape, fill=0x55)
        slots = np.where(stored, self.slots, -1)
        pkv.kv_append(want, want, self.v.contiguous(), self.v.contiguous(), torch.from_numpy(slots).cuda())
        assert torch.equal(want.buf, self.vc.buf)
        codes = self.kc.elements.view(torch.float8_e4m3fn).double().cpu().numpy().reshape(-1, hkv, d)
        raw = self.kc.elements.cpu().numpy().reshape(-1, hkv, d)
        scales = self.kc.scales.permute(0, 2, 1, 3).cpu().numpy().reshape(-1, hkv, d // 32)
        assert (raw[other] == 0x55).all() and (scales[other] == 0x55).all()
        power = scales[at].astype(np.float64) - 127
        want_k, off = k[stored].reshape(-1, hkv, d // 32, 32), (16 * U32 * size)[stored].reshape(-1, hkv, d // 32, 32)
        top, slack = np.abs(want_k).max(-1), off.max(-1)
        # the smallest power of two with top / 2^e <= 448, or its neighbour where the
        # rounding of the 32-bit values decides
        assert ((top - slack) <= 448 * 2.0 ** power).all()
        assert ((top + slack) > 224 * 2.0 ** power)[power > -127].all()
        err = np.abs(codes[at].reshape(want_k.shape) * 2.0 ** power[..., None] - want_k)
        # e4m3: half a step is 2^-4 of the value, at least half of 2^-9
        assert (err <= np.maximum(2.0 ** -4 * np.abs(want_k), 2.0 ** -10 * 2.0 ** power[..., None]) * (1 + 1e-6) + off).all()

    def run(self, **kw):
        out = self.call(**kw)
        assert pkv.get_device_error() == 0
        self.check(out)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "mxfp8"])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 2), (8, 1), (32, 8), (5, 3)])
@pytest.mark.parametrize("d", [64, 128])
def test_types_and_heads(dtype, hq, hkv, d):
    Rope(33, dtype=dtype, hq=hq, hkv=hkv, d=d, seed=hq + d).run()


@pytest.mark.parametrize("d,rot", [(64, 0), (64, 16), (64, 32), (64, 48), (64, 64), (128, 0), (128, 16), (128, 48),
                                   (128, 64), (128, 96), (128, 112), (128, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_rotated_part(d, rot, interleaved, norm):
    for dtype in ("bf16", "f32", "mxfp8"):
        Rope(19, dtype=dtype, d=d, rot=rot, interleaved=interleaved, norm=norm, seed=rot).run()


@pytest.mark.parametrize("n", [1, 2, 3, 15, 16, 17, 100, 1000, 3000])
@pytest.mark.parametrize("dtype", ["bf16", "f32", "mxfp8"])
def test_tokens(n, dtype):
    # one head row a group of lanes below 20000 of them, four above
    Rope(n, dtype=dtype, hq=8, hkv=2, d=128, seed=n).run()


@pytest.mark.parametrize("axes", [2, 3])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_axes(axes, interleaved, d):
    for axis_of in (None, [j % axes for j in range(d // 2)], [(j // 5) % axes for j in range(d // 2)],
                    [axes - 1] * (d // 2)):
        Rope(40, hq=8, d=d, axes=axes, axis_of=axis_of, interleaved=interleaved, seed=axes).run()
        Rope(40, dtype="f32", d=d, axes=axes, axis_of=axis_of, interleaved=interleaved, seed=axes).run()


@pytest.mark.parametrize("p", [1, 7, 16, 96, 256])
@pytest.mark.parametrize("dtype", ["bf16", "mxfp8"])
def test_block_sizes(p, dtype):
    Rope(50, dtype=dtype, p=p, seed=p).run()


@pytest.mark.parametrize("dtype,pad", [("bf16", 8), ("bf16", 264), ("f32", 4), ("mxfp8", 16)])
def test_padded_tokens(dtype, pad):
    Rope(20, dtype=dtype, pad=pad).run()


def test_one_weight_alone_and_norms_of_small_and_large_rows():
    r = Rope(20, dtype="f32")
    r.wk = None
    r.run()
    r = Rope(20, dtype="f32", seed=1)
    r.wq = None
    r.run()
    for scale in (1e-12, 1e-3, 1e15):
        Rope(20, dtype="f32", scale=scale).run()
    Rope(20, dtype="f32", scale=0.0, eps=0.5).run()


def test_far_positions_lose_nothing():
    r = Rope(64, dtype="f32", far=200000, hq=2, hkv=1)
    r.pos[0] = np.arange(199936, 200000)
    r.run()


def test_rows_that_are_skipped():
    for dtype in ("bf16", "f32", "mxfp8"):
        r = Rope(30, dtype=dtype, axes=3, hq=8, hkv=2, d=64)
        r.slots[3] = r.slots[20] = -1   # rotated, not stored
        r.pos[0, 5] = -1                # no token: nothing at all, whatever its other positions
        r.pos[2, 6] = -7
        r.pos[1, 7] = 2**31 - 1
        r.pos[:, 8] = -1
        r.slots[8] = 10**12             # of no token, so not looked at
        out = r.call()
        assert pkv.get_device_error() == pkv.DEVERR_POSITION
        live = np.ones(30, bool)
        live[[5, 6, 7, 8]] = False
        stored = live & (r.slots >= 0)
        r.pos[:, ~live] = 0
        r.check(out, live, stored)


def test_errors_are_named():
    r = Rope(10)
    r.slots[4] = r.shape[0] * r.p
    out = r.call()
    assert pkv.get_device_error() == pkv.DEVERR_SLOT
    r.check(out, None, np.arange(10) != 4)
    r = Rope(10)
    r.pos[0, 9] = 1000
    out = r.call()
    assert pkv.get_device_error() == pkv.DEVERR_POSITION
    live = np.arange(10) != 9
    r.pos[0, 9] = 0
    r.check(out, live)


def test_no_tokens():
    r = Rope(4)
    out = pkv.qk_norm_rope_append(r.q[:0], r.k[:0], r.v[:0], r.kc, r.vc,
                                  torch.empty(0, dtype=torch.int64, device="cuda"),
                                  torch.empty(0, dtype=torch.int32, device="cuda"), torch.from_numpy(r.table).cuda())
    assert out.shape == (0, 4, 64) and (r.kc == 77.0).all()


def test_nan_and_infinity_stay_in_their_rows():
    r = Rope(12, dtype="f32", norm=True, hq=4, hkv=2)
    clean = r.call().clone()
    kc = r.kc.clone()
    r.qkv[3, 70] = float("nan")    # q head 1 of token 3
    r.qkv[5, 4 * 64 + 2] = float("inf")   # k head 0 of token 5
    out = r.call()
    assert pkv.get_device_error() == 0
    assert out[3, 1].isnan().all()
    out[3, 1] = clean[3, 1]
    assert torch.equal(out, clean)
    got = r.kc.view(-1, 2, 64)
    kc = kc.view(-1, 2, 64)
    got[r.slots[5], 0] = kc[r.slots[5], 0]
    assert torch.equal(got, kc)


def test_in_place_queries():
    r = Rope(25, dtype="bf16")
    q = r.q.contiguous()
    want = r.call()
    args = list(r.args())
    args[0] = q
    got = pkv.qk_norm_rope_append(*args, q_weight=r.wq, k_weight=r.wk, out=q)
    assert got is q and torch.equal(got, want)


def test_graph_side_stream_and_the_decode_behind_it():
    # the append of a step and the decode that reads it, on a side stream and replayed
    lens = [40, 5, 100]
    c = su.Cache([t - 1 for t in lens], hkv=2, d=64, width=8)
    r = Rope(3, hq=8, hkv=2, d=64)
    for i, t in enumerate(lens):  # their last row's slot, in blocks of the cache
        need = -(-t // 16)
        if c.tables_np[i, need - 1] < 0:
            c.tables_np[i, need - 1] = c.k.shape[0] - 1 - i
    c.tables = torch.from_numpy(c.tables_np).cuda()
    slots = torch.tensor([int(c.slots(i, [t - 1])[0]) for i, t in enumerate(lens)], device="cuda")
    pos = torch.tensor([t - 1 for t in lens], dtype=torch.int32, device="cuda")
    table_t = torch.from_numpy(r.table).cuda()
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, res = torch.empty(3, 8, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(3, 8, 64, dtype=torch.bfloat16,
                                                                                      device="cuda")

    def step():
        pkv.qk_norm_rope_append(r.q, r.k, r.v, c.k, c.v, slots, pos, table_t, q_weight=r.wq, k_weight=r.wk, out=out)
        pkv.paged_attention_decode(out, c.k, c.v, c.tables, lens_t, 0.125, out=res)

    step()
    torch.cuda.synchronize()
    want, want_q = res.clone(), out.clone()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step()
    for _ in range(3):
        res.zero_()
        out.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            g.replay()
        side.synchronize()
        assert torch.equal(res, want) and torch.equal(out, want_q)
    assert pkv.get_device_error() == 0


def test_large_offsets():
    # a pool past 2^31 elements: the last slots
    nb = (2**31 // (16 * 8 * 128)) + 64
    kc = torch.zeros(nb, 16, 8, 128, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    r = Rope(3, hq=8, hkv=8, d=128)
    r.slots = np.array([nb * 16 - 1, 0, nb * 16 - 17], np.int64)
    a = list(r.args())
    a[3], a[4] = kc, vc
    pkv.qk_norm_rope_append(*a, q_weight=r.wq, k_weight=r.wk)
    assert pkv.get_device_error() == 0
    small = Rope(3, hq=8, hkv=8, d=128)
    small.slots = np.array([2, 0, 1], np.int64)
    small.call()
    got = kc.view(-1, 8, 128)[torch.from_numpy(r.slots).cuda()]
    assert torch.equal(got, small.kc.view(-1, 8, 128)[[2, 0, 1]])
    assert torch.equal(vc.view(-1, 8, 128)[torch.from_numpy(r.slots).cuda()], r.v)


def test_more_lanes_than_32_bits_count():
    # three groups of sixteen lanes a token; all tokens but the ends are padding
    n, ends = (1 << 28) // 3 + 1000, 6
    if torch.cuda.mem_get_info()[0] < 90 << 30:
        pytest.skip("69 GB of rows")
    r = Rope(2 * ends, hq=1, hkv=1, d=128, seed=11)
    q, k, v = (torch.empty(n, 1, 128, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    slots = torch.full((n,), -1, dtype=torch.int64, device="cuda")
    pos = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    for big, small in ((q, r.q), (k, r.k), (v, r.v), (slots, torch.from_numpy(r.slots)), (pos, torch.from_numpy(r.pos[0]))):
        big[:ends], big[-ends:] = small[:ends].to(big.device), small[ends:].to(big.device)
    pkv.qk_norm_rope_append(q, k, v, r.kc, r.vc, slots, pos, torch.from_numpy(r.table).cuda(), q_weight=r.wq,
                            k_weight=r.wk, eps=r.eps, out=q)
    assert pkv.get_device_error() == 0
    r.check(torch.cat([q[:ends], q[-ends:]]))
