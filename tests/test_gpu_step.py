"""Speculative steps from lengths to lengths with nothing on the host between: blocks and
slots, norm, rotation and append, the draft-tree attention, the verdict, the
accepted rows moved together, the other blocks given back; then the windowed decode
over what has become of the cache."""
import numpy as np
import pytest
import torch

from paged_kv_cache_41_gb300 import pkv

import serving_util as su
from step_util import Blocks, verify

pytestmark = pytest.mark.gpu
I32 = torch.int32

VOCAB, B, HQ, HKV, D, P, WIDTH = 40, 5, 8, 2, 64, 16, 12
DEPTH = [0, 1, 1, 2, 2, 3]               # a root, two children, ...
WORDS = [1, 3, 5, 11, 21, 43]
N = len(WORDS)


class Serving:
    """Requests whose rows are a table of projections by token; the logits are a
    fixed projection of the attention's output."""

    def __init__(self, dtype):
        g = torch.Generator(device="cuda")
        g.manual_seed(5)
        io = su.IO[dtype]
        r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.dtype, self.emb = dtype, r(VOCAB, (HQ + 2 * HKV) * D).to(io)
        self.head = r(HQ * D, VOCAB) * 0.3
        self.wq, self.wk = 1 + 0.1 * r(D), 1 + 0.1 * r(D)
        angle = np.arange(500)[:, None] * 100.0 ** (-np.arange(D // 2) / (D // 2))
        self.angles = torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1)).float().cuda()
        nb = B * WIDTH
        if dtype == "mxfp8":
            self.k, self.v = (pkv.MxPool(nb, P, HKV, D, fill=0x7F) for _ in range(2))
        else:
            self.k, self.v = (torch.full((nb, P, HKV, D), float("nan"), dtype=io, device="cuda") for _ in range(2))
        perm = torch.randperm(nb, generator=g, device="cuda").to(I32)
        self.free, self.count = perm.clone(), torch.tensor([nb], dtype=I32, device="cuda")
        self.tables = torch.full((B, WIDTH), -1, dtype=I32, device="cuda")
        self.lens = torch.zeros(B, dtype=I32, device="cuda")
        self.root = torch.arange(B, dtype=I32, device="cuda")
        self.masks = torch.tensor(WORDS * B, device="cuda")
        self.depth = torch.tensor(DEPTH, dtype=I32, device="cuda")
        self.six = torch.full((B,), N, dtype=I32, device="cuda")
        self.drafted = torch.zeros(B, N, dtype=I32, device="cuda")   # this step's inputs
        self.u = torch.zeros(B * N, device="cuda")
        self.plain = Blocks(nb, P, self.tables.tolist(), self.free.tolist(), nb)
        self.said = [[] for _ in range(B)]                            # tokens whose rows are cached

    def step(self):
        drafted = torch.cat([self.root[:, None], self.drafted[:, 1:]], 1).view(-1)
        grown, ptr, slots, pos = pkv.kv_blocks_update(self.k, self.tables, self.lens, self.six, self.free, self.count,
                                                      base_lens=self.lens, num_rows=B * N)
        q, k, v = (x.unflatten(1, (-1, D)) for x in self.emb[drafted.long()].split([HQ * D, HKV * D, HKV * D], 1))
        turn = (self.lens[:, None] + self.depth).view(-1)   # a tree's rows: by depth
        q = pkv.qk_norm_rope_append(q, k, v, self.k, self.v, slots, turn, self.angles, q_weight=self.wq,
                                    k_weight=self.wk)
        out = pkv.draft_tree_attention(q, self.k, self.v, self.tables, self.lens, ptr, su.softmax_scale(D),
                                       max_draft=N, masks=self.masks)
        probs = torch.softmax(out.view(B * N, -1).float() @ self.head, -1)
        keep, keep_lens, nxt = pkv.draft_verify(probs, drafted, ptr, self.u, max_draft=N, masks=self.masks)
        pkv.kv_compact(self.k, self.v, self.tables, grown, keep, keep_lens, base_lens=self.lens)
        lens, _, _, _ = pkv.kv_blocks_update(self.k, self.tables, grown, keep_lens, self.free, self.count,
                                             base_lens=self.lens, num_rows=0)
        self.lens.copy_(lens)
        self.root.copy_(nxt)
        return drafted, slots, probs, keep, keep_lens, nxt

    def inputs(self, k):
        rng = np.random.default_rng(k)
        self.drafted.copy_(torch.from_numpy(rng.integers(0, VOCAB, (B, N)).astype(np.int32)))
        self.u.copy_(torch.from_numpy(rng.random(B * N).astype(np.float32) * 0.3))

    def check(self, lens_before, got):
        """One step against the plain forms, in Python."""
        drafted, slots, probs, keep, keep_lens, nxt = (x.cpu().numpy() for x in got)
        grown, _, want_slots, _ = self.plain.update(lens_before, lens_before, [N] * B, B * N)
        assert slots.tolist() == want_slots
        accepted = []
        for r in range(B):
            s = slice(r * N, r * N + N)
            path, token = verify(probs[s], None, drafted[s], WORDS, self.u.cpu().numpy()[s])
            assert keep[r, 0, : keep_lens[r]].tolist() == path and nxt[r] == token
            self.said[r] += [int(drafted[s][i]) for i in path]
            accepted.append(len(path))
        lens, _, _, _ = self.plain.update(grown, lens_before, accepted, 0)
        assert self.lens.tolist() == lens and self.tables.tolist() == self.plain.tables
        assert self.count.item() == self.plain.count and self.free.tolist() == self.plain.free
        return accepted

    def check_cache(self):
        """Every request's cached rows are those of the tokens that it has said, at
        their positions, bit for bit; and attended under a window."""
        longest = max(len(s) for s in self.said)
        # of the same width: the decode's work split, so its rounding, goes by it
        want = su.Cache([len(s) for s in self.said], dtype=self.dtype, hkv=HKV, d=D, p=P, width=WIDTH)
        q = torch.zeros(B, HQ, D, dtype=self.emb.dtype, device="cuda")
        for r, said in enumerate(self.said):
            rows = self.emb[torch.tensor(said, device="cuda")]
            q_, k_, v_ = (x.unflatten(1, (-1, D)) for x in rows.split([HQ * D, HKV * D, HKV * D], 1))
            slots = torch.from_numpy(want.slots(r, np.arange(len(said)))).cuda()
            q[r] = pkv.qk_norm_rope_append(q_, k_, v_, want.k, want.v, slots,
                                           torch.arange(len(said), dtype=I32, device="cuda"), self.angles,
                                           q_weight=self.wq, k_weight=self.wk)[-1]
        args = dict(window=20, num_sinks=3)
        lens = torch.tensor([len(s) for s in self.said], dtype=I32, device="cuda")
        a = pkv.paged_attention_decode_window(q, self.k, self.v, self.tables, lens, 0.125, **args)
        b = pkv.paged_attention_decode_window(q, want.k, want.v, want.tables, lens, 0.125, **args)
        assert longest > 20 and torch.equal(a, b) and not a.isnan().any()
        mine = su.Cache.__new__(su.Cache)
        mine.__dict__.update(want.__dict__, k=self.k, v=self.v, tables_np=self.tables.cpu().numpy())
        for r, said in enumerate(self.said):
            for x, y in zip(mine.rows64(r, len(said)), want.rows64(r, len(said))):
                assert np.array_equal(x, y)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "mxfp8"])
def test_speculative_steps(dtype):
    s = Serving(dtype)
    total = 0
    for k in range(30):
        s.inputs(k)
        before = s.lens.tolist()
        got = s.step()
        assert pkv.get_device_error() == 0
        total += sum(s.check(before, got))
    assert total > 30 * B  # some drafts were accepted
    s.check_cache()


def test_speculative_steps_in_a_graph():
    eager, s = Serving("bf16"), Serving("bf16")
    s.inputs(0)
    keep = {x: getattr(s, x).clone() for x in ("tables", "lens", "root", "free", "count", "k", "v")}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.step()                      # warm up, then back to the start
        for x, y in keep.items():
            getattr(s, x).copy_(y)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            out = s.step()
    torch.cuda.current_stream().wait_stream(side)
    for k in range(30):
        for x in (s, eager):
            x.inputs(k)
        before = s.lens.tolist()
        g.replay()
        got = [x.clone() for x in out]
        want = eager.step()
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)
        s.check(before, got)
    assert pkv.get_device_error() == 0
    s.check_cache()


def test_windowed_decode_steps_that_give_blocks_back():
    # one row a step for 200 steps, 40 rows seen: the pool would not hold the rest
    window, sinks, steps = 37, 3, 200
    c = 4
    k = torch.full((c * 5, P, HKV, D), float("nan"), dtype=torch.float32, device="cuda")
    v = torch.full_like(k, float("nan"))
    free, count = torch.arange(c * 5, dtype=I32, device="cuda"), torch.tensor([c * 5], dtype=I32, device="cuda")
    tables = torch.full((c, 16), -1, dtype=I32, device="cuda")
    lens, one = torch.zeros(c, dtype=I32, device="cuda"), torch.ones(c, dtype=I32, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    qkv = torch.randn(steps, c, (HQ + 2 * HKV) * D, generator=g, device="cuda")
    outs, qs = [], []
    for i in range(steps):
        lens, _, slots, pos = pkv.kv_blocks_update(k, tables, lens, one, free, count, base_lens=lens, num_rows=c,
                                                   window=window, num_sinks=sinks)
        q, kk, vv = (x.unflatten(1, (-1, D)) for x in qkv[i].split([HQ * D, HKV * D, HKV * D], 1))
        qs.append(pkv.qk_norm_rope_append(q, kk, vv, k, v, slots, pos, None))
        outs.append(pkv.paged_attention_decode_window(qs[-1], k, v, tables, lens, 0.125, window=window,
                                                      num_sinks=sinks))
    assert pkv.get_device_error() == 0
    rows = qkv.double().cpu().numpy()
    for i in (0, 36, 37, 39, 40, 41, 55, 100, 199):
        seen = [t for t in range(i + 1) if t < sinks or t >= i + 1 - window]
        for r in range(c):
            kv = rows[seen, r, HQ * D:].reshape(len(seen), 2, HKV, D)
            for h in range(HQ):
                o, _, _, absv, mag = su.attend64(rows[i, r, h * D:(h + 1) * D][None], kv[:, 0, h // 4],
                                                 kv[:, 1, h // 4], np.ones((1, len(seen)), bool), 0.125)
                su.check_attention("f32", D, outs[i][r:r + 1, h].double().cpu().numpy(), None, o, None, absv, mag,
                                   len(seen), f"step {i}")
