"""The operators together, as a serving loop uses them: append drafted tokens,
verify them, commit the accepted path, decode and weigh, evict, go on."""
import numpy as np
import pytest
import torch

from paged_kv_cache_41_gb300 import pkv

import serving_util as su

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,hq,hkv,d", [("bf16", 8, 2, 128), ("f32", 4, 2, 64), ("mxfp8", 8, 2, 128),
                                            ("bf16", 16, 2, 128)])
def test_speculate_commit_weigh_evict(dtype, hq, hkv, d):
    b, p, budget, sinks, recent = 3, 16, 96, 4, 16
    lens = [40, 130, 77]
    # every sequence owns a table row of 20 blocks; rows past its length are to come
    c = su.Cache([320] * b, dtype=dtype, hkv=hkv, d=d, p=p, seed=2, extra_blocks=0)
    scale = su.softmax_scale(d)
    rng = np.random.default_rng(3)
    g = hq // hkv
    # the logical rows every (sequence, kv head) should hold, in binary64
    held = [list(c.rows64(r, t)) for r, t in enumerate(lens)]
    scores = np.zeros((b, hkv, 320))
    w = torch.zeros(b, hkv, 320, device="cuda")
    p_bits = 0.0 if dtype == "f32" else 2.0 ** -8
    for step in range(6):
        # ---- speculate: a tree of drafted tokens each
        n = [int(rng.integers(1, 20)) for _ in range(b)]
        words = [su.tree_masks(m, rng) for m in n]
        ptr = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        slots = np.concatenate([c.slots(r, lens[r] + np.arange(n[r])) for r in range(b)])
        c.append(c.randn(int(ptr[-1]), hkv, d), c.randn(int(ptr[-1]), hkv, d), slots)
        q = c.randn(int(ptr[-1]), hq, d)
        ctx_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
        out = pkv.draft_tree_attention(q, c.k, c.v, c.tables, ctx_t, torch.from_numpy(ptr).cuda(),
                                       scale, max_draft=max(n),
                                       masks=su.as_int64(sum(words, [])).cuda())
        q64 = q.double().cpu().numpy()
        paths = []
        for r in range(b):
            drafted = [x[lens[r]:] for x in c.rows64(r, lens[r] + n[r])]
            k, v = [np.concatenate([x, y]) for x, y in zip(held[r], drafted)]
            seen = np.ones((n[r], lens[r] + n[r]), bool)
            seen[:, lens[r]:] = [[(x >> j) & 1 for j in range(n[r])] for x in words[r]]
            for h in range(hq):
                o, l, _, absv, mag = su.attend64(q64[ptr[r]:ptr[r + 1], h], k[:, h // g], v[:, h // g],
                                                 seen, scale)
                su.check_attention(dtype, d, out[ptr[r]:ptr[r + 1], h].double().cpu().numpy(), None, o, l,
                                   absv, mag, len(k), f"step {step} draft", p_bits=p_bits)
            leaf = words[r][int(rng.integers(0, n[r]))]
            paths.append([j for j in range(n[r]) if (leaf >> j) & 1])
            held[r] = [np.concatenate([x, y[paths[r]]]) for x, y in zip(held[r], drafted)]
        # ---- commit the accepted paths
        keep = np.full((b, 1, max(n)), -1, np.int32)
        for r, path in enumerate(paths):
            keep[r, 0, :len(path)] = path
        acc = np.array([len(x) for x in paths], np.int32)
        pkv.kv_compact(c.k, c.v, c.tables,
                       torch.tensor([t + m for t, m in zip(lens, n)], dtype=torch.int32, device="cuda"),
                       torch.from_numpy(keep).cuda(), torch.from_numpy(acc).cuda(), base_lens=ctx_t)
        lens = [t + int(a) for t, a in zip(lens, acc)]
        # ---- one weighing decode over what is held
        q = c.randn(b, hq, d)
        lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
        lse = torch.empty(b, hq, device="cuda")
        out = pkv.paged_attention_decode_weights(q, c.k, c.v, c.tables, lens_t, w, scale, lse=lse,
                                                 decay=0.95)
        q64 = q.double().cpu().numpy()
        for r in range(b):
            scores[r, :, :lens[r]] *= 0.95
            for h in range(hkv):
                mine = slice(h * g, (h + 1) * g)
                k, v = held[r][0][:, h], held[r][1][:, h]
                o, l, pw, absv, mag = su.attend64(q64[r, mine], k, v, np.ones((g, len(k)), bool), scale)
                su.check_attention(dtype, d, out[r, mine].double().cpu().numpy(),
                                   lse[r, mine].double().cpu().numpy(), o, l, absv, mag, len(k),
                                   f"step {step} decode",
                                   p_bits=2.0 ** -16 if g == 8 else 0.0)
                scores[r, h, :lens[r]] += pw.sum(0)
        # every weight within 1e-4 relative: score_error stays below 4e-5 here
        got = w.double().cpu().numpy()
        assert (np.abs(got - scores) <= 1e-4 * scores + 1e-30).all()
        # ---- evict down to the budget, by the kernel's own scores
        keep_t, new_t = pkv.kv_evict_select(w, lens_t, budget, num_sinks=sinks, num_recent=recent)
        pkv.kv_compact(c.k, c.v, c.tables, lens_t, keep_t, new_t, weights=w)
        keep, new = keep_t.cpu().numpy(), new_t.cpu().numpy()
        for r in range(b):
            assert new[r] == min(lens[r], budget)
            held[r] = [np.stack([x[keep[r, h, :new[r]], h] for h in range(hkv)], 1) for x in held[r]]
            for h in range(hkv):
                s = scores[r, h, keep[r, h, :new[r]]]
                scores[r, h] = 0
                scores[r, h, :new[r]] = s
            for x, y in zip(c.rows64(r, int(new[r])), held[r]):
                assert np.array_equal(x, y)
        lens = [int(x) for x in new]
        assert pkv.get_device_error() == 0


class Small:
    """Inputs of every operator over one small cache."""

    def __init__(self, seed, dtype="bf16"):
        lens, n = [300, 33, 700], [5, 0, 17]
        self.c = su.Cache([t + m for t, m in zip(lens, n)], dtype=dtype, hkv=2, d=128, p=16, seed=seed)
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.ptr = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device="cuda")
        rng = np.random.default_rng(seed)
        self.masks = su.as_int64(sum((su.tree_masks(m, rng) for m in n if m), [])).cuda()
        self.q = self.c.randn(sum(n), 8, 128)
        self.q1 = self.c.randn(3, 8, 128)
        self.w0 = torch.rand(3, 2, 720, device="cuda")
        self.scale = su.softmax_scale(128)

    def run(self, stream=None, ws=(None, None)):
        c, w = self.c, self.w0.clone()
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        out = pkv.draft_tree_attention(self.q, c.k, c.v, c.tables, self.lens, self.ptr, self.scale, max_draft=17,
                                       masks=self.masks, workspace=ws[0], stream=stream)
        out1 = pkv.paged_attention_decode_weights(self.q1, c.k, c.v, c.tables, self.lens, w, self.scale,
                                                  workspace=ws[1], stream=stream)
        keep, new = pkv.kv_evict_select(w, self.lens, 200, num_sinks=4, num_recent=20, stream=stream)
        return out, out1, keep, new, w

    def workspaces(self):
        k, nb = self.c.k, self.c.tables.shape[1]
        return [torch.empty(n, dtype=torch.uint8, device="cuda") for n in
                (pkv.draft_tree_workspace_bytes(k, 3, 8, 17, nb), pkv.decode_weights_workspace_bytes(k, 3, 8, nb))]


@pytest.mark.parametrize("dtype", ["bf16", "f32", "mxfp8"])
def test_results_belong_to_the_launching_stream(dtype):
    x = Small(4, dtype)
    want = x.run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = x.run(s)
    owners = {}
    for seg in torch.cuda.memory_snapshot():
        for t in got[:4]:
            if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
                owners[t.data_ptr()] = seg["stream"]
    s.synchronize()
    assert sorted(owners) == sorted(t.data_ptr() for t in got[:4])
    assert set(owners.values()) == {s.cuda_stream}
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_two_graphs_replayed_at_once():
    xs = [Small(5), Small(6, "mxfp8")]
    want = [x.run() for x in xs]
    torch.cuda.synchronize()
    graphs, got = [], []
    for x in xs:
        ws = x.workspaces()  # one for each graph
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(x.run(ws=ws))
        graphs.append((g, ws))
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(20):
        for (g, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert pkv.get_device_error() == 0
    for a, b in zip(want, got):
        for t, u in zip(a, b):
            assert torch.equal(t, u)
