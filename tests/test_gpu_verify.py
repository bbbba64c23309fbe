"""pkv_draft_verify against exact fractions: every answer is a whole number, so
everything must be equal; and the distribution of what it emits."""
import numpy as np
import pytest
import torch

from paged_kv_cache_41_gb300 import pkv

import serving_util as su
from step_util import verify

pytestmark = pytest.mark.gpu
I32 = torch.int32


def softmax(x):
    e = np.exp(x - x.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


class Verify:
    def __init__(self, n, vocab, *, tree=True, sampled=True, peak=2.0, noise=0.7, pad=0, lead=0, trail=0, seed=0,
                 max_draft=None):
        rng = np.random.default_rng(seed)
        self.n, self.vocab, self.pad = list(n), vocab, pad
        self.ptr = lead + np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        rows = self.rows = int(self.ptr[-1]) + trail
        x = rng.standard_normal((rows, vocab)) * peak
        self.p = softmax(x)
        self.q = softmax(x + noise * rng.standard_normal((rows, vocab))) if sampled else None
        self.words = [su.tree_masks(m, rng) if tree else [(2 << i) - 1 for i in range(m)] for m in n]
        self.masks = [0] * lead + [w for ws in self.words for w in ws] + [0] * trail if tree else None
        self.tok = rng.integers(0, vocab, rows).astype(np.int32)
        for r, m in enumerate(n):
            for i in range(1, m):
                older = self.words[r][i] & ((1 << i) - 1)
                row = self.ptr[r] + older.bit_length() - 1
                d = (self.q if sampled else self.p)[row].astype(np.float64)
                # its children: samples of the draft, or likely tokens of the target
                self.tok[self.ptr[r] + i] = rng.choice(vocab, p=d / d.sum()) if sampled else rng.choice(
                    np.argsort(-d)[:6])
        self.u = rng.random(rows).astype(np.float32)
        self.u[self.u >= 1] = 0
        self.max_draft = max_draft or max(list(n) + [1])

    def wide(self, x):
        out = torch.full((self.rows, self.vocab + self.pad), float("nan"), device="cuda")
        out[:, : self.vocab] = torch.from_numpy(x).cuda()
        return out[:, : self.vocab]

    def tensors(self):
        return (self.wide(self.p), torch.from_numpy(self.tok).cuda(), torch.from_numpy(self.ptr).cuda(),
                torch.from_numpy(self.u).cuda()), dict(
            max_draft=self.max_draft, draft_probs=None if self.q is None else self.wide(self.q),
            masks=None if self.masks is None else su.as_int64(self.masks).cuda())

    def call(self, **kw):
        a, k = self.tensors()
        return pkv.draft_verify(*a, **{**k, **kw})

    def want(self):
        out = []
        for r, m in enumerate(self.n):
            s = slice(self.ptr[r], self.ptr[r] + m)
            out.append(verify(self.p[s], None if self.q is None else self.q[s], self.tok[s],
                              None if self.masks is None else self.words[r], self.u[s]))
        return out

    def check(self, got):
        keep, lens, nxt = (x.cpu().numpy() for x in got)
        assert keep.shape == (len(self.n), 1, self.max_draft)
        for r, (path, token) in enumerate(self.want()):
            assert lens[r] == len(path), r
            assert keep[r, 0].tolist() == path + [-1] * (self.max_draft - len(path)), r
            assert nxt[r] == token, r

    def run(self, **kw):
        got = self.call(**kw)
        assert pkv.get_device_error() == 0
        self.check(got)


N = [1, 2, 5, 0, 17, 64, 33, 3, 9, 1]


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("sampled", [False, True])
@pytest.mark.parametrize("vocab", [1, 2, 7, 128, 500, 1031])
def test_trees_and_chains(tree, sampled, vocab):
    for seed in range(3):
        Verify(N, vocab, tree=tree, sampled=sampled, seed=seed).run()


@pytest.mark.parametrize("vocab", [4095, 4096, 4097, 8193, 20000, 33000, 70001])
@pytest.mark.parametrize("sampled", [False, True])
def test_vocabularies(vocab, sampled):
    # one to eight CTAs a request, segments that end anywhere
    Verify([4, 1, 6], vocab, sampled=sampled, peak=1.0, seed=vocab).run()


@pytest.mark.parametrize("batch", [65, 130, 300, 700])
def test_batches(batch):
    Verify([1 + r % 5 for r in range(batch)], 600, seed=batch).run()
    Verify([1 + r % 5 for r in range(batch)], 9000, seed=batch, peak=3.0, sampled=False).run() if batch < 100 else None


@pytest.mark.parametrize("pad", [1, 2, 3, 4, 61])
def test_rows_of_a_wider_buffer(pad):
    Verify([5, 9, 2], 1001, pad=pad, seed=pad).run()
    Verify([5, 9, 2], 1000, pad=pad, sampled=False, seed=pad).run()


def test_rows_before_and_behind_are_not_read():
    v = Verify([4, 0, 9], 300, lead=2, trail=3)
    v.p[:2] = v.p[-3:] = np.nan
    v.tok[:2] = v.tok[-3:] = -5
    v.run()


def test_max_draft_above_what_is_drafted():
    Verify([4, 9], 300, max_draft=64).run()


# ------------------------------------------------------------------- borders
def crafted(p, q, tokens, u, masks=None):
    """One request with given rows."""
    v = Verify([len(tokens)], len(p[0]), tree=masks is not None, sampled=q is not None)
    v.p = np.array(p, np.float32)
    v.q = None if q is None else np.array(q, np.float32)
    v.tok, v.u = np.array(tokens, np.int32), np.array(u, np.float32)
    if masks is not None:
        v.words, v.masks = [masks], masks
    v.run()
    keep, lens, nxt = v.call()
    return keep[0, 0, : int(lens)].tolist(), int(nxt)


def test_a_number_on_the_border_is_turned_down():
    # u q = p: strictly below is wanted; the next token is then of max(p - q, 0)
    p, q = [[0.25, 0.75, 0, 0]] * 2, [[0.5, 0.5, 0, 0]] * 2
    assert crafted(p, q, [0, 0], [0.0, 0.5]) == ([0], 1)
    below = np.nextafter(np.float32(0.5), np.float32(0))
    assert crafted(p, q, [0, 0], [0.3, below]) == ([0, 1], 1)


def test_the_next_token_on_a_border():
    p = [[0.25, 0.25, 0.0, 0.5]]
    for u, want in ((0.0, 0), (0.25, 1), (0.5, 3), (0.999, 3), (1.0, 3), (2.0, 3), (-1.0, 0), (float("nan"), 0)):
        assert crafted(p, None, [0], [u]) == ([0], want)


def test_zero_probabilities():
    # p(x) = 0 is never accepted, q(x) = 0 with p(x) > 0 always
    assert crafted([[0.0, 1.0]] * 2, [[0.5, 0.5]] * 2, [0, 0], [0.4, 0.0]) == ([0], 1)
    assert crafted([[0.0, 1.0]] * 2, [[1.0, 0.0]] * 2, [0, 1], [0.4, 0.999]) == ([0, 1], 1)
    assert crafted([[0.0, 1.0]] * 2, None, [0, 0], [0.4, 0.0]) == ([0], 1)
    assert crafted([[0.0, 1.0]] * 2, None, [0, 1], [0.4, 0.999]) == ([0, 1], 1)


def test_nothing_left():
    # p = q, turned down by an impossible number: the target's own distribution
    assert crafted([[0.5, 0.5]] * 2, [[0.5, 0.5]] * 2, [0, 1], [0.7, 1.0])[0] == [0, 1]
    v = [[0.0, 0.0, 0.0]] * 2
    assert crafted(v, [[0.0, 1.0, 0.0]] * 2, [0, 1], [0.5, 0.5]) == ([0], -1)
    assert crafted(v, None, [0, 1], [0.5, 0.5]) == ([0], -1)
    # every token of p turned down outright
    m = [1, 3, 5]
    assert crafted([[0.5, 0.5, 0.0]] * 3, None, [0, 2, 2], [0.5, 0.0, 0.0], m) == ([0], 1)


def test_siblings_of_the_same_token():
    m = [1, 3, 5, 9]
    crafted([[0.4, 0.3, 0.2, 0.1]] * 4, [[0.1, 0.7, 0.1, 0.1]] * 4, [0, 1, 1, 1], [0.2, 0.9, 0.8, 0.7], m)
    crafted([[0.4, 0.3, 0.2, 0.1]] * 4, None, [0, 1, 1, 2], [0.2, 0.9, 0.0, 0.1], m)
    # sixty-three of a token that the target never takes: c grows past 2^5
    words = [1] + [1 | (1 << i) for i in range(1, 64)]
    crafted([[0.0, 0.25, 0.75]] * 64, [[1.0, 0.0, 0.0]] * 64, [0] * 64, [0.3] * 64, words)


def test_rows_that_are_not_distributions_stay_in_the_vocabulary():
    for bad in (np.nan, np.inf, -np.inf, -0.5, 7.0, 1e-45, 2.0 ** -80):
        for vocab in (3, 300):
            v = Verify([6, 6], vocab, seed=3)
            v.p[:, 1] = bad
            v.q[:, 2] = bad
            keep, lens, nxt = v.call()
            assert ((nxt >= -1) & (nxt < vocab)).all() and ((lens >= 1) & (lens <= 6)).all()
            if bad not in (2.0 ** -80, 1e-45):
                v.check((keep, lens, nxt))
    v = Verify([6, 6], 300, seed=4)   # sums far past what is held exactly
    v.p[:], v.q[:] = 1.0, 0.0
    for vocab_rows in (v, Verify([6, 6], 300, sampled=False, seed=4)):
        vocab_rows.p[:] = 1.0
        keep, lens, nxt = vocab_rows.call()
        assert ((nxt >= -1) & (nxt < 300)).all() and ((lens >= 1) & (lens <= 6)).all()
    assert pkv.get_device_error() == 0


def test_masks_that_are_no_tree():
    v = Verify([8, 8, 8], 50, seed=4)
    rng = np.random.default_rng(1)
    v.words = [[int(rng.integers(0, 1 << 62)) for _ in range(8)], [0] * 8, [(1 << 64) - 1] * 8]
    v.masks = [w for ws in v.words for w in ws]
    v.run()


# ------------------------------------------------------------------ refusals
def test_tokens_outside_the_vocabulary():
    v = Verify([6, 6, 6], 100, seed=2)
    v.tok[[1, 8]] = [100, -1]
    v.tok[12] = 1 << 30   # a root's is not read
    got = v.call()
    assert pkv.get_device_error() == pkv.DEVERR_TOKEN
    v.check(got)


def test_ranges_that_make_no_sense():
    v = Verify([6, 6, 6, 6], 100, seed=2)
    a, k = v.tensors()
    a = list(a)
    a[2] = torch.tensor([0, 6, 4, 40, 24], dtype=I32, device="cuda")
    keep, lens, nxt = pkv.draft_verify(*a, **k)
    assert pkv.get_device_error() == pkv.DEVERR_LENGTH
    assert lens[1:].tolist() == [0, 0, 0] and nxt[1:].tolist() == [-1, -1, -1] and (keep[1:] == -1).all()
    assert lens[0] >= 1
    a[2] = torch.tensor([-3, 3, 9, 12, 18], dtype=I32, device="cuda")
    _, lens, _ = pkv.draft_verify(*a, **{**k, "max_draft": 5})
    assert pkv.get_device_error() == pkv.DEVERR_LENGTH
    assert lens[[0, 1, 3]].tolist() == [0, 0, 0] and lens[2] >= 1


def test_no_rows():
    e = torch.empty(0, device="cuda")
    keep, lens, nxt = pkv.draft_verify(torch.empty(0, 50, device="cuda"), e.to(I32),
                                       torch.zeros(4, dtype=I32, device="cuda"), e, max_draft=3)
    assert (keep == -1).all() and (lens == 0).all() and (nxt == -1).all()


# ------------------------------------------------------------ the distribution
@pytest.mark.parametrize("sampled", [False, True])
def test_what_is_emitted_is_distributed_as_the_target(sampled):
    # two children of the root, 40000 requests: the first token emitted against p
    rng = np.random.default_rng(11)
    batch, vocab = 40000, 6
    p, q = softmax(rng.standard_normal(vocab) * 1.5), softmax(rng.standard_normal(vocab) * 1.5)
    rows = 3 * batch
    tok = (rng.choice(vocab, (batch, 3), p=q.astype(np.float64) / q.astype(np.float64).sum()) if sampled
           else np.tile(np.argsort(-q)[:3], (batch, 1)))
    nxt_row = softmax(rng.standard_normal(vocab))
    probs = np.tile(np.stack([p, nxt_row, nxt_row]), (batch, 1))
    tok_t = torch.from_numpy(tok.reshape(-1).astype(np.int32)).cuda()
    keep, lens, nxt = pkv.draft_verify(
        torch.from_numpy(probs).cuda(), tok_t, torch.arange(batch + 1, dtype=I32, device="cuda") * 3,
        torch.from_numpy(rng.random(rows).astype(np.float32)).clamp(max=1 - 2.0 ** -24).cuda(), max_draft=3,
        draft_probs=torch.from_numpy(np.tile(q, (rows, 1))).cuda() if sampled else None,
        masks=torch.tensor([1, 3, 5] * batch, device="cuda"))
    assert pkv.get_device_error() == 0
    lens, keep, nxt = lens.cpu().numpy(), keep.cpu().numpy()[:, 0], nxt.cpu().numpy()
    first = np.where(lens > 1, tok[np.arange(batch), np.clip(keep[:, 1], 0, 2)], nxt)
    count = np.bincount(first, minlength=vocab)
    sigma = np.sqrt(batch * p * (1 - p))
    assert (np.abs(count - batch * p) < 5 * sigma).all(), (count / batch, p)
    assert 0.05 < (lens > 1).mean() < 0.999


# ----------------------------------------------------------- graphs, streams
def test_graphs_and_a_side_stream():
    vs = [Verify([5, 9, 64, 1], 5000, seed=1), Verify([3] * 20, 40000, sampled=False, seed=2)]
    graphs, streams = [], [torch.cuda.Stream() for _ in vs]
    for v, st in zip(vs, streams):
        a, k = v.tensors()
        v.call()
        b = len(v.n)
        out = [torch.zeros(b, 1, v.max_draft, dtype=I32, device="cuda"), torch.zeros(b, dtype=I32, device="cuda"),
               torch.zeros(b, dtype=I32, device="cuda")]
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=st):
                pkv.draft_verify(*a, **k, keep=out[0], keep_lens=out[1], next_tokens=out[2])
        graphs.append((g, out, a, k))
    torch.cuda.synchronize()
    for _ in range(4):
        for (g, *_), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for v, (_, out, _, _) in zip(vs, graphs):
        v.check(out)
    a, k = vs[0].tensors()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = pkv.draft_verify(*a, **k, stream=side)
    side.synchronize()
    vs[0].check(got)
    assert pkv.get_device_error() == 0


def test_large_offsets():
    # rows past 2^31 elements of the buffer
    vocab, rows = 131072, 2**31 // 131072 + 3
    p = torch.zeros(rows, vocab, device="cuda")
    p[:, 77] = 0.5
    p[:, 131071] = 0.5
    u = torch.full((rows,), 0.9, device="cuda")
    tok = torch.full((rows,), 77, dtype=I32, device="cuda")
    keep, lens, nxt = pkv.draft_verify(p, tok, torch.tensor([rows - 2, rows], dtype=I32, device="cuda"), u,
                                       max_draft=2)
    assert keep.tolist() == [[[0, -1]]] and nxt.tolist() == [131071]
    assert pkv.get_device_error() == 0
