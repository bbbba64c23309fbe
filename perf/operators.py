"""Operators of a serving loop over a paged K/V cache that verifies drafted
tokens and keeps the cache inside a budget: their cases, their plain forms and
the calls of the framework's own kernels.

* ``draft``: attention of every sequence's drafted tokens (a chain or a tree,
  at most 64) over its cached context and their drafted ancestors.
* ``weigh``: one decode step that also adds each cached row's attention weight,
  summed over the query heads of its kv head, to a running score.
* ``select``: per sequence and kv head, the rows to keep within a budget: the
  first ``sinks``, the last ``recent`` and the highest scores between them.
* ``compact``: move the kept rows of K and V (and their scores) together, in
  place; ``commit`` is the same call for the accepted path of a draft.

The cache is one pool per tensor, [blocks, block size, kv heads, head dim],
read through block tables (int32 [sequences, blocks], -1 padded).  Lengths are
spread evenly over a case's range and dealt out by the seed, so that a case's
work does not depend on it.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "mxfp8": torch.uint8}


# ---------------------------------------------------------------- the cases
def _case(op, dtype, batch, heads, d, p, lo, hi, **more):
    hq, hkv = heads
    return {"op": op, "dtype": dtype, "batch": batch, "hq": hq, "hkv": hkv, "d": d, "p": p,
            "lo": lo, "hi": hi, **more}


def listed():
    def named(name, c):
        return {"name": name, **c}

    return [
        # one request on a short chat, a chain of four drafted tokens: latency
        named("draft, 1 chat, chain 4",
              _case("draft", "bf16", 1, (32, 8), 128, 16, 300, 300, n_lo=4, n_hi=4, tree=False)),
        # an ordinary speculative step: ragged trees of 5 to 27 nodes over ordinary contexts
        named("draft, 16 requests, trees",
              _case("draft", "bf16", 16, (32, 8), 128, 16, 512, 8192, n_lo=5, n_hi=27, tree=True)),
        # the largest: the full decode batch, every tree at the limit of 64 nodes
        named("draft, 64 requests, trees of 64",
              _case("draft", "bf16", 64, (32, 8), 128, 16, 512, 8192, n_lo=64, n_hi=64, tree=True)),
        # eight query heads per kv head over a quantized pool, odd tree sizes
        named("draft, MXFP8 pool, 64/8 heads",
              _case("draft", "mxfp8", 12, (64, 8), 128, 32, 700, 5001, n_lo=3, n_hi=17, tree=True)),
        # a few short fp32 sequences: latency, and the precise type
        named("weigh, fp32, 4 short",
              _case("weigh", "f32", 4, (4, 2), 64, 16, 1, 100)),
        # the decode batch that the framework is measured on
        named("weigh, 64 requests",
              _case("weigh", "bf16", 64, (32, 8), 128, 16, 512, 8192)),
        # long contexts, the ones whose cache has to be cut
        named("weigh, 8 long contexts",
              _case("weigh", "bf16", 8, (32, 8), 128, 64, 32768, 65536)),
        # the decode batch brought down to 1024 rows each
        named("select, 64 requests",
              _case("select", "f32", 64, (8, 8), 128, 16, 512, 8192, budget=1024, sinks=4, recent=128)),
        # long contexts brought down to 16384 rows each
        named("select, 8 long contexts",
              _case("select", "f32", 8, (8, 8), 128, 64, 32768, 65536, budget=16384, sinks=16,
                    recent=1000)),
        # the accepted paths of a speculative step, every head alike: latency
        named("commit, 64 requests",
              _case("commit", "bf16", 64, (32, 8), 128, 16, 512, 8192, n_lo=16, n_hi=16, acc_hi=6)),
        # the eviction that follows "select, 64 requests", a list per kv head
        named("compact, 64 requests",
              _case("compact", "bf16", 64, (32, 8), 128, 16, 512, 8192, budget=1024, sinks=4,
                    recent=128)),
        # a few long fp32 sequences: few chains of rows, each a long one
        named("compact, fp32, 3 long",
              _case("compact", "f32", 3, (4, 2), 64, 32, 9000, 30001, budget=7777, sinks=1,
                    recent=64)),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["draft", "draft", "weigh", "select", "commit", "compact"])
    dtype = "f32" if op == "select" else rng.choice(["bf16", "bf16", "bf16", "f32", "mxfp8"])
    if op in ("commit", "compact") and dtype == "mxfp8":
        dtype = "bf16"
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 8])
    d = rng.choice([64, 128, 128])
    if dtype == "mxfp8" and hq == 8 * hkv:
        d = 128  # what the quantized decode takes
    p = rng.choice([16, 16, 32, 64, 128])
    batch = _log(rng, 1, 64)
    # rows of the whole batch, well inside the largest listed cases'
    rows = 200000 if dtype == "bf16" else 60000
    hi = max(2, _log(rng, 20, min(65536, max(40, rows // batch))))
    lo = rng.randint(1, hi)
    c = _case(op, dtype, batch, (hq, hkv), d, p, lo, hi)
    if op == "draft":
        n_hi = _log(rng, 1, 64)
        c.update(n_lo=rng.randint(1, n_hi), n_hi=n_hi, tree=rng.random() < 0.7)
    elif op == "commit":
        n_hi = _log(rng, 2, 64)
        c.update(n_lo=rng.randint(1, n_hi), n_hi=n_hi, acc_hi=rng.randint(1, 8))
    elif op in ("select", "compact"):
        budget = max(2, _log(rng, max(2, hi // 8), hi))
        sinks = rng.randint(0, min(16, budget // 2))
        c.update(budget=budget, sinks=sinks, recent=rng.randint(0, (budget - sinks) // 2))
    return c


def _spread(lo, hi, n):
    """n whole numbers spread evenly over [lo, hi]."""
    if n == 1:
        return [(lo + hi) // 2]
    return [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _lens(case):
    return _spread(case["lo"], case["hi"], case["batch"])


def _drafts(case):
    return _spread(case["n_lo"], case["n_hi"], case["batch"])


def _elem(case):
    # MXFP8: one byte, and one scale byte for 32 elements
    return {"bf16": 2.0, "f32": 4.0, "mxfp8": 1.0 + 1.0 / 32.0}[case["dtype"]]


def work(case):
    hq, hkv, d, lens = case["hq"], case["hkv"], case["d"], _lens(case)
    io = 4 if case["dtype"] == "f32" else 2
    row = hkv * d * _elem(case)  # one token's K, or V
    if case["op"] == "draft":
        n = _drafts(case)
        keys = sum(lens) + sum(n)
        per = sum(n) / len(n)
        nbytes = 2 * keys * row + sum(n) * hq * (2 * d * io + 4) + 8 * sum(n)
        return {"bytes": nbytes, "flops": 4 * d * hq * per * keys}
    if case["op"] == "weigh":
        nbytes = 2 * sum(lens) * row + len(lens) * hq * (2 * d * io + 4) + 8 * hkv * sum(lens)
        return {"bytes": nbytes, "flops": 4 * d * hq * sum(lens)}
    if case["op"] == "select":
        kept = sum(min(t, case["budget"]) for t in lens)
        return {"bytes": 4 * hkv * (sum(lens) + kept), "flops": hkv * sum(lens)}
    if case["op"] == "commit":
        kept = sum(_accepted(case))  # the root is in its place already
        return {"bytes": 4 * kept + 4 * row * (kept - case["batch"]), "flops": 0}
    # rows before the first dropped one need not move: the sinks
    moved = sum(max(0, case["budget"] - case["sinks"]) for t in lens if t > case["budget"])
    dropped = sum(max(0, t - case["budget"]) for t in lens)
    listed_rows = sum(min(t, case["budget"]) for t in lens)
    nbytes = 4 * hkv * listed_rows + moved * (4 * row + hkv * 8) + 4 * hkv * dropped
    return {"bytes": nbytes, "flops": 0}


def _accepted(case):
    return [1 + i % min(case["acc_hi"], n) for i, n in enumerate(_drafts(case))]


# ---------------------------------------------------------------- the inputs
def _pool(case, g, blocks):
    shape = (blocks, case["p"], case["hkv"], case["d"])
    if case["dtype"] != "mxfp8":
        return torch.randn(shape, generator=g, device="cuda",
                           dtype=torch.float32).to(DTYPES[case["dtype"]])
    # E4M3 codes of N(0, 1) rows over scales of 1/64 to 1/32: the element plane,
    # then the plane of scale bytes
    n = math.prod(shape)
    x = torch.randn(n, generator=g, device="cuda") * 48.0
    codes = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    scales = torch.randint(121, 123, (n // 32,), generator=g, device="cuda", dtype=torch.uint8)
    return torch.cat([codes, scales])


def _tree_masks(case, rng, drafts):
    """One 64-bit word a drafted token: itself and its ancestors."""
    words = []
    for n in drafts:
        mine = []
        for i in range(n):
            if case["tree"]:
                parent = -1 if i == 0 else rng.randint(max(0, i - 5), i - 1)
            else:
                parent = i - 1
            mine.append((1 << i) | (mine[parent] if parent >= 0 else 0))
        words += mine
    return torch.tensor([w - (1 << 64) if w >> 63 else w for w in words], dtype=torch.int64,
                        device="cuda")


def prepare(case, seed):
    rng = random.Random(seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    lens = _lens(case)
    rng.shuffle(lens)
    drafts = _drafts(case) if "n_lo" in case else [0] * len(lens)
    accepted = _accepted(case) if case["op"] == "commit" else None
    if accepted:
        both = list(zip(drafts, accepted))
        rng.shuffle(both)
        drafts, accepted = [list(x) for x in zip(*both)]
    else:
        rng.shuffle(drafts)
    p, batch, hkv = case["p"], case["batch"], case["hkv"]
    i32 = dict(dtype=torch.int32, device="cuda")
    s = {"case": case, "lens": torch.tensor(lens, **i32),
         "scale": 1.0 / math.sqrt(case["d"])}
    total = [t + n for t, n in zip(lens, drafts)]
    if case["op"] != "select":
        need = [-(-t // p) for t in total]
        blocks = max(1, math.ceil(1.25 * sum(need)))
        placed = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
        width = max(need)
        start = torch.tensor([sum(need[:r]) for r in range(batch)], device="cuda")[:, None]
        col = torch.arange(width, device="cuda")[None]
        held = col < torch.tensor(need, device="cuda")[:, None]
        at = (start + col).clamp(max=blocks - 1)
        s["tables"] = torch.where(held, placed[at], -1).contiguous()
        s["k"], s["v"] = _pool(case, g, blocks), _pool(case, g, blocks)
    io = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    if case["op"] in ("draft", "weigh"):
        rows = sum(drafts) if case["op"] == "draft" else batch
        s["q"] = torch.randn(rows, case["hq"], case["d"], generator=g, device="cuda").to(io)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(rows, case["hq"], device="cuda")
    longest = max(total)
    live = torch.arange(longest, device="cuda")[None, None] < s["lens"][:, None, None]
    if case["op"] == "draft":
        s["ptr"] = torch.tensor([sum(drafts[:r]) for r in range(batch + 1)], **i32)
        s["masks"] = _tree_masks(case, rng, drafts)
        s["max_draft"] = case["n_hi"]
    elif case["op"] == "commit":
        # the accepted path: the root, then nodes in ascending order
        keep = [[0] + sorted(rng.sample(range(1, n), a - 1)) for n, a in zip(drafts, accepted)]
        width = max(drafts)
        s["keep"] = torch.tensor([k + [-1] * (width - len(k)) for k in keep], **i32)[:, None]
        s["keep_lens"] = torch.tensor(accepted, **i32)
        s["base"], s["lens"] = s["lens"], torch.tensor(total, **i32)
    else:
        # scores as decoding leaves them: heavy-tailed, zero where nothing looked yet
        w = torch.randn(batch, hkv, longest, generator=g, device="cuda").mul_(2).exp_()
        unseen = torch.rand(batch, hkv, longest, generator=g, device="cuda") < 0.02
        s["weights"] = w.masked_fill_(unseen | ~live, 0.0)
    if case["op"] in ("select", "compact"):
        keep, new = _choose(s["weights"], s["lens"], case)
        if case["op"] == "compact":
            s["keep"], s["keep_lens"] = keep, new
        else:
            s["keep"], s["new_lens"] = torch.zeros_like(keep), torch.zeros_like(new)
    return s


# ---------------------------------------------------------------- plain forms
def _values(s, pool):
    """A pool's rows in 32 bits: [blocks * block size, kv heads, head dim]."""
    c = s["case"]
    hkv, d, p = c["hkv"], c["d"], c["p"]
    if c["dtype"] != "mxfp8":
        return pool.view(-1, hkv, d).float()
    n = pool.numel() * 32 // 33
    x = pool[:n].view(torch.float8_e4m3fn).float().view(-1, p, hkv, d // 32, 32)
    e = torch.exp2(pool[n:].float() - 127).view(-1, hkv, p, d // 32).transpose(1, 2)
    return (x * e[..., None]).view(-1, hkv, d)


def _slots(s, positions):
    """Pool rows of the positions [batch, n] of every sequence."""
    p = s["case"]["p"]
    blocks = torch.gather(s["tables"].long(), 1, (positions // p).clamp(max=s["tables"].shape[1] - 1))
    return blocks * p + positions % p


def _history(s, longest):
    """K and V of every sequence in 32 bits, [batch, kv heads, longest, head dim]; rows past
    a sequence's blocks are some other row's."""
    at = torch.arange(longest, device="cuda").expand(s["case"]["batch"], -1)
    rows = _slots(s, at).clamp(min=0)
    return (_values(s, s["k"])[rows].transpose(1, 2), _values(s, s["v"])[rows].transpose(1, 2))


def _attend(scores, seen):
    """Softmax weights of the seen places, and the log of their sum."""
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True).clamp(min=-3.0e38)
    e = torch.exp(scores - top)
    total = e.sum(-1, keepdim=True)
    return e / total.clamp(min=1e-38), (torch.log(total) + top).squeeze(-1)


def _draft(s):
    c = s["case"]
    batch, hq, hkv, d = c["batch"], c["hq"], c["hkv"], c["d"]
    n = s["max_draft"]
    longest = s["tables"].shape[1] * c["p"]
    k, v = _history(s, longest)
    ptr = s["ptr"].long()
    rows = (ptr[:-1, None] + torch.arange(n, device="cuda")).clamp(max=int(s["q"].shape[0]) - 1)
    q = s["q"].float()[rows].view(batch, n, hkv, hq // hkv, d)
    q = q.permute(0, 2, 3, 1, 4).reshape(batch, hkv, -1, d)
    scores = (q @ k.transpose(-1, -2)).view(batch, hkv, hq // hkv, n, longest) * s["scale"]
    at = torch.arange(longest, device="cuda") - s["lens"].long()[:, None]
    held = (ptr[1:] - ptr[:-1])[:, None]
    bit = (s["masks"][rows][:, :, None] >> at.clamp(0, 63)[:, None, :]) & 1
    seen = (at < 0)[:, None, :] | ((at < held)[:, None, :] & (at >= 0)[:, None, :] & (bit == 1))
    w, lse = _attend(scores, seen[:, None, None])
    out = (w.view(batch, hkv, -1, longest) @ v.masked_fill((at >= held)[:, None, :, None], 0.0))
    out = out.view(batch, hkv, hq // hkv, n, d).permute(0, 3, 1, 2, 4).reshape(batch, n, hq, d)
    lse = lse.permute(0, 3, 1, 2).reshape(batch, n, hq)
    mine = torch.arange(n, device="cuda") < held
    return out[mine].to(s["q"].dtype), lse[mine]


def _weigh(s):
    c = s["case"]
    batch, hq, hkv, d = c["batch"], c["hq"], c["hkv"], c["d"]
    longest = s["weights"].shape[2]
    k, v = _history(s, longest)
    q = s["q"].float().view(batch, hkv, hq // hkv, d)
    scores = (q @ k.transpose(-1, -2)) * s["scale"]
    seen = torch.arange(longest, device="cuda") < s["lens"][:, None]
    w, lse = _attend(scores, seen[:, None, None])
    out = w @ v.masked_fill(~seen[:, None, :, None], 0.0)
    s["weights"] += w.sum(2)
    return out.view(batch, hq, d).to(s["q"].dtype), lse.view(batch, hq), s["weights"]


def _choose(weights, lens, case):
    """Rows kept, ascending and -1 padded, [batch, kv heads, budget], and how many."""
    budget, n = case["budget"], weights.shape[2]
    at = torch.arange(n, device="cuda")
    lens = lens.long()[:, None, None]
    forced = (at < case["sinks"]) | (at >= lens - case["recent"])
    w = weights.masked_fill(forced, math.inf).masked_fill(at >= lens, -math.inf)
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices
    new = lens.clamp(max=budget)
    rank = torch.empty_like(order).scatter_(2, order, at.expand_as(order))
    kept = torch.sort(torch.where(rank < new, at, n), dim=-1).values[..., :budget]
    if kept.shape[2] < budget:
        kept = torch.nn.functional.pad(kept, (0, budget - kept.shape[2]), value=n)
    kept = torch.where(kept < n, kept, -1).to(torch.int32)
    return kept.contiguous(), new.view(-1).to(torch.int32)


def _compact(s):
    c = s["case"]
    j = torch.arange(s["keep"].shape[2], device="cuda")
    r, h, at = (j < s["keep_lens"][:, None, None]).expand_as(s["keep"]).nonzero(as_tuple=True)
    base = s["base"].long()[r] if "base" in s else 0
    src, dst = s["keep"][r, h, at].long() + base, at + base
    p, tables = c["p"], s["tables"].long()
    from_, to = (tables[r, x // p] * p + x % p for x in (src, dst))
    k, v = s["k"].view(-1, c["hkv"], c["d"]), s["v"].view(-1, c["hkv"], c["d"])
    if s["keep"].shape[1] == 1:
        k[to], v[to] = k[from_], v[from_]
    else:
        k[to, h], v[to, h] = k[from_, h], v[from_, h]
    if "weights" in s:
        w = s["weights"]
        moved = w[r, h, src]
        place = torch.arange(w.shape[2], device="cuda")[None, None]
        w.masked_fill_((place >= s["keep_lens"][:, None, None]) & (place < s["lens"][:, None, None]),
                       0.0)
        w[r, h, dst] = moved
        return s["k"], s["v"], w
    return s["k"], s["v"]


def _pools(s, pkv):
    """The pools as the framework takes them."""
    if s["case"]["dtype"] != "mxfp8":
        return s["k"], s["v"]
    if "mx" not in s:
        c = s["case"]
        nb = s["k"].numel() * 32 // 33 // (c["p"] * c["hkv"] * c["d"])
        s["mx"] = [pkv.MxPool(nb, c["p"], c["hkv"], c["d"], buf=s[x]) for x in ("k", "v")]
    return s["mx"]


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        if op == "draft":
            return _draft(s)
        if op == "weigh":
            return _weigh(s)
        if op == "select":
            return _choose(s["weights"], s["lens"], s["case"])
        return _compact(s)
    from paged_kv_cache_41_gb300 import pkv

    if op == "select":
        c = s["case"]
        pkv.kv_evict_select(s["weights"], s["lens"], c["budget"], num_sinks=c["sinks"],
                            num_recent=c["recent"], keep=s["keep"], new_lens=s["new_lens"])
        return s["keep"], s["new_lens"]
    k, v = _pools(s, pkv)
    if op == "draft":
        if "ws" not in s:
            n = pkv.draft_tree_workspace_bytes(k, s["tables"].shape[0], s["q"].shape[1],
                                               s["max_draft"], s["tables"].shape[1])
            s["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        pkv.draft_tree_attention(s["q"], k, v, s["tables"], s["lens"], s["ptr"], s["scale"],
                                 max_draft=s["max_draft"], masks=s["masks"], out=s["out"],
                                 lse=s["lse"], workspace=s["ws"])
        return s["out"], s["lse"]
    if op == "weigh":
        if "ws" not in s:
            n = pkv.decode_weights_workspace_bytes(k, s["tables"].shape[0], s["q"].shape[1],
                                                   s["tables"].shape[1])
            s["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        pkv.paged_attention_decode_weights(s["q"], k, v, s["tables"], s["lens"], s["weights"],
                                           s["scale"], out=s["out"], lse=s["lse"],
                                           workspace=s["ws"])
        return s["out"], s["lse"], s["weights"]
    pkv.kv_compact(k, v, s["tables"], s["lens"], s["keep"], s["keep_lens"],
                   base_lens=s.get("base"), weights=s.get("weights"))
    return (s["k"], s["v"], s["weights"]) if "weights" in s else (s["k"], s["v"])


# ---------------------------------------------------------------- in 64 bits
def exact(case, seed):
    if case["op"] == "select":
        return None  # whole numbers
    s = prepare(case, seed)
    if case["op"] in ("commit", "compact"):
        # bytes moved, nothing computed; the scores by a gather row by row
        if "weights" not in s:
            return None
        w = s["weights"].double()
        for r, t in enumerate(s["lens"].tolist()):
            n = int(s["keep_lens"][r])
            kept = torch.gather(w[r], 1, s["keep"][r, :, :n].long())
            w[r, :, :t] = 0
            w[r, :, :n] = kept
        return None, None, w
    hq, hkv, d, p = case["hq"], case["hkv"], case["d"], case["p"]

    def rows64(pool, table, t):
        """Rows 0 .. t - 1 of one sequence, [kv heads, t, head dim]."""
        ids = table[: -(-t // p)].long()
        if case["dtype"] != "mxfp8":
            return pool[ids].reshape(-1, hkv, d)[:t].double().transpose(0, 1)
        n = pool.numel() // 33 * 32
        codes = pool[:n].view(-1, p, hkv, d)[ids].view(torch.float8_e4m3fn).double()
        power = pool[n:].view(-1, hkv, p, d // 32)[ids].double() - 127.0
        power = power.permute(0, 2, 1, 3).repeat_interleave(32, dim=3)
        return torch.ldexp(codes, power).reshape(-1, hkv, d)[:t].transpose(0, 1)

    outs, lses = [], []
    weights = s["weights"].double() if case["op"] == "weigh" else None
    for r, t in enumerate(s["lens"].tolist()):
        if case["op"] == "draft":
            a, b = s["ptr"][r : r + 2].tolist()
            words = [int(w) for w in s["masks"][a:b]]
            grid = [[(w >> j) & 1 for j in range(b - a)] for w in words]
            seen = torch.ones(b - a, t + b - a, dtype=torch.bool, device="cuda")
            seen[:, t:] = torch.tensor(grid, dtype=torch.bool, device="cuda")
        else:
            a, b = r, r + 1
            seen = torch.ones(1, t, dtype=torch.bool, device="cuda")
        k, v = (rows64(s[x], s["tables"][r], seen.shape[1]) for x in ("k", "v"))
        out = torch.empty(b - a, hq, d, dtype=torch.float64, device="cuda")
        lse = torch.empty(b - a, hq, dtype=torch.float64, device="cuda")
        for h in range(hkv):
            mine = slice(h * hq // hkv, (h + 1) * hq // hkv)
            q = s["q"][a:b, mine].double() * s["scale"]
            x = torch.einsum("igd,td->igt", q, k[h])
            x = torch.where(seen[:, None, :], x, -math.inf)
            lse[:, mine] = torch.logsumexp(x, -1)
            x = torch.exp(x - lse[:, mine, None])
            out[:, mine] = torch.einsum("igt,td->igd", x, v[h])
            if case["op"] == "weigh":
                weights[r, h, :t] += x[0].sum(0)
        outs.append(out)
        lses.append(lse)
    if case["op"] == "weigh":
        return torch.cat(outs), torch.cat(lses), weights
    return torch.cat(outs), torch.cat(lses)
