"""Operators of a whole serving step on the GPU around the paged K/V cache: their
cases, their plain forms and the calls of the framework's own kernels.

* ``blocks``: block tables and slot maps from request lengths.  Growing requests
  take blocks from a stack of free ids, shrinking ones give theirs back.
* ``rope``: RMS norms of the queries and keys of every head, the rotation by their
  positions (one axis, or time, height and width), and the append of K and V.
* ``window``: a decode in which a token sees the first ``sinks`` rows and the last
  ``window`` ones.
* ``verify``: drafted tokens (a chain or a tree) against the target's
  probabilities, from given random numbers: the accepted path and the next token.

The cache is one pool per tensor, [blocks, block size, kv heads, head dim], read
through block tables (int32 [sequences, blocks], -1 padded).  Lengths are spread
evenly over a case's range and dealt out by the seed, so that a case's work does
not depend on it.  A pass can be repeated on its state: what it changes it brings
back, or writes again.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "mxfp8": torch.bfloat16}  # of q, k, v and out
ROPE_ROWS = 131072  # positions that the table of angles covers


# ---------------------------------------------------------------- the cases
def _blocks(kind, batch, p, lo, hi, n_lo=1, n_hi=1):
    return {"op": "blocks", "kind": kind, "batch": batch, "p": p, "lo": lo, "hi": hi, "n_lo": n_lo,
            "n_hi": n_hi}


def _rope(dtype, batch, n, heads, d, p, rot, axes=1, norm=True, interleaved=False):
    return {"op": "rope", "dtype": dtype, "batch": batch, "n": n, "hq": heads[0], "hkv": heads[1],
            "d": d, "p": p, "rot": rot, "axes": axes, "norm": norm, "interleaved": interleaved}


def _window(dtype, batch, heads, d, p, lo, hi, window, sinks):
    return {"op": "window", "dtype": dtype, "batch": batch, "hq": heads[0], "hkv": heads[1], "d": d,
            "p": p, "lo": lo, "hi": hi, "window": window, "sinks": sinks}


def _verify(batch, n_lo, n_hi, vocab, tree, sampled, pad=0):
    return {"op": "verify", "batch": batch, "n_lo": n_lo, "n_hi": n_hi, "vocab": vocab, "tree": tree,
            "sampled": sampled, "pad": pad}


def listed():
    def named(name, c):
        return {"name": name, **c}

    return [
        # an ordinary decode step: one new row a request, a block for one in sixteen
        named("blocks, 64 requests, one row", _blocks("grow", 64, 16, 512, 8192)),
        # a speculative step whose drafts are all turned down: blocks come and go
        named("blocks, 256 requests, drafts", _blocks("drafts", 256, 16, 64, 16384, 1, 16)),
        # long contexts preempted and resumed: every block goes and comes, slots for every row
        named("blocks, 8 long resumed", _blocks("resume", 8, 64, 32768, 65536)),
        # the decode step of the batch that the framework is measured on: latency
        named("rope, 64 tokens", _rope("bf16", 64, 1, (32, 8), 128, 16, 128)),
        # an image prompt of three axes into a quantized pool, 64/8 heads
        named("rope, MXFP8 pool, 3 axes", _rope("mxfp8", 1, 1441, (64, 8), 128, 32, 128, axes=3)),
        # prompts of a whole batch: bandwidth
        named("rope, 32768 tokens", _rope("bf16", 8, 4096, (32, 8), 128, 16, 128)),
        # one chat: latency
        named("window, 1 chat", _window("bf16", 1, (32, 8), 128, 16, 2000, 2000, 512, 4)),
        # the decode batch, most of it longer than what it sees
        named("window, 64 requests", _window("bf16", 64, (32, 8), 128, 16, 512, 8192, 1024, 4)),
        # long contexts with eight query heads per kv head
        named("window, 8 long, 64/8 heads", _window("bf16", 8, (64, 8), 128, 16, 32768, 65536, 16384, 64)),
        # one chat with a chain of four drafted tokens behind its root: latency
        named("verify, 1 chat, chain 5", _verify(1, 5, 5, 32000, False, True)),
        # trees whose tokens are the draft's best ones, over an odd vocabulary
        named("verify, 16 requests, trees", _verify(16, 5, 27, 100003, True, False, pad=61)),
        # the decode batch, every request with a sampled chain
        named("verify, 64 requests, chain 9", _verify(64, 9, 9, 131072, False, True)),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["blocks", "rope", "window", "verify"])
    p = rng.choice([16, 16, 32, 64, 128])
    if op == "blocks":
        kind = rng.choice(["grow", "drafts", "resume"])
        batch = _log(rng, 1, 512)
        hi = _log(rng, 20, min(65536, 400000 // batch))
        n_hi = _log(rng, 1, 64)
        return _blocks(kind, batch, p, rng.randint(1, hi), hi, rng.randint(0, n_hi), n_hi)
    hkv = rng.choice([1, 2, 4, 8])
    heads = (hkv * rng.choice([1, 2, 4, 8]), hkv)
    d = rng.choice([64, 128, 128])
    dtype = rng.choice(["bf16", "bf16", "f32", "mxfp8"])
    if op == "rope":
        batch = _log(rng, 1, 64)
        n = _log(rng, 1, (1400 if dtype == "mxfp8" else 8000) // batch)
        rot = rng.choice([d, d, d // 2, d // 4])
        return _rope(dtype, batch, n, heads, d, p, rot, rng.choice([1, 1, 2, 3]), rng.random() < 0.7,
                     rng.random() < 0.3)
    if op == "window":
        if dtype == "mxfp8" and heads[0] == 8 * hkv:
            d = 128  # what the quantized decode takes
        batch = _log(rng, 1, 64)
        rows = 200000 if dtype == "bf16" else 60000
        hi = max(2, _log(rng, 20, min(65536, max(40, rows // batch))))
        return _window(dtype, batch, heads, d, p, rng.randint(1, hi), hi,
                       _log(rng, 1, max(2, hi)), rng.choice([0, 1, 4, 16, 100]))
    vocab = _log(rng, 900, 131072)
    batch = _log(rng, 1, 64)
    n_hi = _log(rng, 1, max(1, min(64, 4000000 // (batch * vocab))))
    return _verify(batch, rng.randint(1, n_hi), n_hi, vocab, rng.random() < 0.5, rng.random() < 0.5,
                   rng.choice([0, 0, 3, 64]))


def _spread(lo, hi, n):
    """n whole numbers spread evenly over [lo, hi]."""
    if n == 1:
        return [(lo + hi) // 2]
    return [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _elem(case):
    # MXFP8: one byte, and one scale byte for 32 elements
    return {"bf16": 2.0, "f32": 4.0, "mxfp8": 1.0 + 1.0 / 32.0}[case["dtype"]]


def work(case):
    op, batch = case["op"], case["batch"]
    if op == "blocks":
        p, lens = case["p"], _spread(case["lo"], case["hi"], batch)
        if case["kind"] == "resume":
            ids, rows = sum(-(-t // p) for t in lens), sum(lens)
            return {"bytes": 24 * batch + 20 * ids + 12 * rows, "flops": rows}
        n = _spread(case["n_lo"], case["n_hi"], batch)
        ids = sum(n) / p * (1 if case["kind"] == "grow" else 2.5)
        return {"bytes": 16 * batch + 8 * ids + 12 * sum(n), "flops": sum(n)}
    if op == "verify":
        n = _spread(case["n_lo"], case["n_hi"], batch)
        rows = 2 if case["sampled"] else 1  # of p, and of q
        return {"bytes": 4 * case["vocab"] * rows * batch + 24 * sum(n), "flops": 2 * case["vocab"] * batch}
    io = 4 if case["dtype"] == "f32" else 2
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if op == "rope":
        n = batch * case["n"]
        token = (2 * hq + 2 * hkv) * d * io + 2 * hkv * d * _elem(case) + 4 * case["axes"] + 8
        return {"bytes": n * token + 4 * case["rot"] * min(n, ROPE_ROWS), "flops": 8 * n * (hq + hkv) * d}
    seen = [min(t, case["window"] + case["sinks"]) for t in _spread(case["lo"], case["hi"], batch)]
    nbytes = 2 * sum(seen) * hkv * d * _elem(case) + batch * hq * (2 * d * io + 4)
    return {"bytes": nbytes, "flops": 4 * d * hq * sum(seen)}


# ---------------------------------------------------------------- the inputs
def _tables(need, blocks, g):
    """A block table with need[r] ids in row r, and the order the ids were dealt in."""
    placed = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    first = [0]
    for n in need:
        first.append(first[-1] + n)
    col = torch.arange(max(need + [1]), device="cuda")[None]
    held = col < torch.tensor(need, device="cuda")[:, None]
    at = (torch.tensor(first[:-1], device="cuda")[:, None] + col).clamp(max=blocks - 1)
    return torch.where(held, placed[at], -1).contiguous(), placed


def _tree(case, rng, drafts):
    """Parents within each request (the root's is -1), and one 64-bit word a node: itself and
    its ancestors."""
    parents, words = [], []
    for n in drafts:
        mine, up = [], []
        for i in range(n):
            up.append(-1 if i == 0 else rng.randint(max(0, i - 4), i - 1) if case["tree"] else i - 1)
            mine.append((1 << i) | (mine[up[i]] if i else 0))
        parents.append(up)
        words += mine
    signed = [w - (1 << 64) if w >> 63 else w for w in words]
    return parents, torch.tensor(signed, dtype=torch.int64, device="cuda")


def prepare(case, seed):
    rng = random.Random(seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": case}
    make = {"blocks": _prepare_blocks, "rope": _prepare_rope, "window": _prepare_window,
            "verify": _prepare_verify}[case["op"]]
    make(case, s, rng, g)
    return s


def _prepare_blocks(case, s, rng, g):
    i32 = dict(dtype=torch.int32, device="cuda")
    batch, p = case["batch"], case["p"]
    lens = _spread(case["lo"], case["hi"], batch)
    rng.shuffle(lens)
    n = lens if case["kind"] == "resume" else _spread(case["n_lo"], case["n_hi"], batch)
    if case["kind"] != "resume":
        rng.shuffle(n)
    need = [-(-t // p) for t in lens]
    width = -(-(max(lens) + max(n)) // p)
    blocks = max(math.ceil(1.25 * sum(need)), sum(need) + sum(-(-k // p) + 1 for k in n))
    table, placed = _tables(need, blocks, g)
    s["tables"] = torch.full((batch, width), -1, **i32)
    s["tables"][:, : table.shape[1]] = table[:, :width]
    s["free"] = placed.flip(0).contiguous()  # what is dealt out stands behind the free ids
    s["count"] = torch.tensor([blocks - sum(need)], **i32)
    s["count_out"] = torch.zeros_like(s["count"])
    s["lens"], s["add"] = torch.tensor(lens, **i32), torch.tensor(n, **i32)
    s["zeros"] = torch.zeros(batch, **i32)
    s["pool"] = torch.empty(blocks, p, 1, 8, dtype=torch.bfloat16, device="cuda")  # its shape counts
    s["rows"] = sum(n) + (0 if case["kind"] == "resume" else 3)  # a padded batch
    for x in ("a", "b"):
        rows = s["rows"] if x == "a" else 0
        s[x] = dict(out_lens=torch.zeros(batch, **i32), row_ptr=torch.zeros(batch + 1, **i32),
                    slots=torch.zeros(rows, dtype=torch.int64, device="cuda"),
                    positions=torch.zeros(rows, **i32))


def _prepare_rope(case, s, rng, g):
    batch, n, p, hkv, d = case["batch"], case["n"], case["p"], case["hkv"], case["d"]
    total, heads = batch * n, case["hq"] + 2 * hkv
    io = DTYPES[case["dtype"]]
    s["qkv"] = (torch.randn(total, heads * d, generator=g, device="cuda") * 2).to(io)  # of the projection
    per = -(-(n + p - 1) // p)  # a request's rows start anywhere in its first block
    placed = torch.randperm(batch * per, generator=g, device="cuda")
    off = torch.randint(0, p, (batch, 1), generator=g, device="cuda") + torch.arange(n, device="cuda")
    at = torch.arange(batch, device="cuda")[:, None] * per + off // p
    s["slots"] = (placed[at] * p + off % p).view(-1).contiguous()
    start = torch.randint(0, ROPE_ROWS - n - 40, (batch, 1), generator=g, device="cuda")
    pos = start + torch.arange(n, device="cuda")
    if case["axes"] > 1:  # pictures of 24 columns between stretches of text
        i = torch.arange(n, device="cuda")
        t = start + torch.where(i // 384 % 2 == 1, i // 384 * 384, i)
        h, w = t + (i // 384 % 2) * (i % 384 // 24), t + (i // 384 % 2) * (i % 24)
        pos = torch.stack([t, h, w][: case["axes"]])
    s["positions"] = pos.reshape(-1, total).to(torch.int32).contiguous()
    half = case["rot"] // 2
    s["axis_of"] = [min(j * case["axes"] // half, case["axes"] - 1) for j in range(half)]
    s["axes"] = torch.tensor(s["axis_of"], device="cuda")
    freq = 1e6 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    angle = torch.arange(ROPE_ROWS, device="cuda", dtype=torch.float64)[:, None] * freq
    s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    s["wq"] = s["wk"] = None
    if case["norm"]:
        s["wq"], s["wk"] = (1 + 0.2 * torch.randn(2, d, generator=g, device="cuda")).unbind(0)
    shape = (batch * per, p, hkv, d)
    if case["dtype"] == "mxfp8":
        s["k"], s["v"] = (torch.zeros(math.prod(shape) * 33 // 32, dtype=torch.uint8, device="cuda")
                          for _ in range(2))
    else:
        s["k"], s["v"] = (torch.zeros(shape, dtype=io, device="cuda") for _ in range(2))
    s["shape"] = shape
    s["out"] = torch.empty(total, case["hq"], d, dtype=io, device="cuda")


def _prepare_window(case, s, rng, g):
    batch, p, hkv, d = case["batch"], case["p"], case["hkv"], case["d"]
    lens = _spread(case["lo"], case["hi"], batch)
    rng.shuffle(lens)
    need = [-(-t // p) for t in lens]
    blocks = max(1, math.ceil(1.25 * sum(need)))
    s["tables"], _ = _tables(need, blocks, g)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    io = DTYPES[case["dtype"]]
    s["shape"] = (blocks, p, hkv, d)
    for x in ("k", "v"):
        if case["dtype"] == "mxfp8":  # codes of N(0, 1) rows over scales of 1/64 to 1/32
            n = math.prod(s["shape"])
            codes = (torch.randn(n, generator=g, device="cuda") * 48).clamp(-448, 448)
            scales = torch.randint(121, 123, (n // 32,), generator=g, device="cuda", dtype=torch.uint8)
            s[x] = torch.cat([codes.to(torch.float8_e4m3fn).view(torch.uint8), scales])
        else:
            s[x] = torch.randn(s["shape"], generator=g, device="cuda", dtype=torch.float32).to(io)
    s["q"] = torch.randn(batch, case["hq"], d, generator=g, device="cuda").to(io)
    s["out"], s["lse"] = torch.empty_like(s["q"]), torch.empty(batch, case["hq"], device="cuda")
    s["scale"] = 1.0 / math.sqrt(d)


def _prepare_verify(case, s, rng, g):
    i32 = dict(dtype=torch.int32, device="cuda")
    batch, vocab = case["batch"], case["vocab"]
    n = _spread(case["n_lo"], case["n_hi"], batch)
    rng.shuffle(n)
    parents, masks = _tree(case, rng, n)
    s["masks"] = masks if case["tree"] else None
    ptr = [sum(n[:r]) for r in range(batch + 1)]
    s["ptr"], s["max_draft"] = torch.tensor(ptr, **i32), case["n_hi"]
    rows, wide = ptr[-1], vocab + case["pad"]
    # the target's and the draft's distributions: peaked, and alike
    target = torch.randn(rows, wide, generator=g, device="cuda").mul_(3.0)
    draft = target + 0.8 * torch.randn(rows, wide, generator=g, device="cuda")
    s["p"] = target.softmax(-1).narrow(1, 0, vocab)  # a padded vocabulary's front part
    draft = draft.softmax(-1).narrow(1, 0, vocab)
    up = torch.tensor([ptr[r] + max(0, u) for r in range(batch) for u in parents[r]], device="cuda")
    if case["sampled"]:
        s["q"] = draft
        s["tokens"] = torch.multinomial(draft[up], 1, generator=g).view(-1).to(torch.int32)
    else:  # the draft's best tokens, each child of a node its own
        s["q"] = None
        best = draft.topk(8, -1).indices
        rank, seen = [], {}
        for r in range(batch):
            for u in parents[r]:
                rank.append(min(seen.get((r, u), 0), 7))
                seen[r, u] = seen.get((r, u), 0) + 1
        s["tokens"] = best[up, torch.tensor(rank, device="cuda")].to(torch.int32)
    s["u"] = torch.rand(rows, generator=g, device="cuda")
    s["keep"] = torch.zeros(batch, 1, s["max_draft"], **i32)
    s["keep_lens"], s["next"] = torch.zeros(batch, **i32), torch.zeros(batch, **i32)
    parent = [u + [-1] * (s["max_draft"] - len(u)) for u in parents]
    s["parent"] = torch.tensor(parent, device="cuda")


# ---------------------------------------------------------------- plain forms
def _update(s, lens, base, add, count, rows):
    """New lengths base + add: blocks given back, blocks taken, the new rows' slots."""
    p, table, free = s["case"]["p"], s["tables"], s["free"]
    total = free.numel()
    lens, new = lens.long(), (base + add).long()
    held, want = (lens + p - 1) // p, (new + p - 1) // p
    col = torch.arange(table.shape[1], device="cuda")
    goes = ((col >= want[:, None]) & (col < held[:, None]) & (table >= 0)).flatten().flip(0)
    rank = goes.long().cumsum(0)
    place = torch.where(goes, count.long() + rank - 1, total)
    spare = torch.cat([free, free[:1]])
    spare[place] = table.flatten().flip(0)
    free.copy_(spare[:total])
    avail = count.long() + rank[-1]
    table.masked_fill_(goes.flip(0).view_as(table), -1)
    demand = (want - held).clamp(min=0)
    upto = demand.cumsum(0)
    served = (demand == 0) | (upto <= avail)
    taken = torch.where(served, upto, 0).amax()
    comes = (col >= held[:, None]) & (col < want[:, None]) & served[:, None]
    at = avail - 1 - (upto - demand)[:, None] - (col - held[:, None])
    table.copy_(torch.where(comes, free[at.clamp(0, total - 1)], table))
    ptr = torch.nn.functional.pad((new - lens).clamp(min=0).cumsum(0), (1, 0))
    i = torch.arange(rows, device="cuda")
    r = torch.searchsorted(ptr[1:], i, right=True).clamp(max=lens.numel() - 1)
    pos = lens[r] + i - ptr[r]
    real = (i < ptr[-1]) & served[r]
    block = table[r, (pos // p).clamp(max=table.shape[1] - 1)].long()
    slots = torch.where(real, block * p + pos % p, -1)
    pos = torch.where(real, pos, -1).to(torch.int32)
    new = torch.where(served, new, lens).to(torch.int32)
    return new, ptr.to(torch.int32), slots, pos, (avail - taken).to(torch.int32).view(1)


def _plain_blocks(s):
    kind, zeros = s["case"]["kind"], s["zeros"]
    if kind == "resume":
        lens, _, _, _, count = _update(s, s["lens"], zeros, zeros, s["count"], 0)
        lens, ptr, slots, pos, count = _update(s, lens, zeros, s["lens"], count, s["rows"])
        return s["tables"], s["free"], lens, ptr, slots, pos, count
    lens, ptr, slots, pos, count = _update(s, s["lens"], s["lens"], s["add"], s["count"], s["rows"])
    if kind == "drafts":
        lens, _, _, _, count = _update(s, lens, s["lens"], zeros, count, 0)
    return s["tables"], s["free"], lens, ptr, slots, pos, count


def _split(s):
    c = s["case"]
    q, k, v = s["qkv"].split([c["hq"] * c["d"], c["hkv"] * c["d"], c["hkv"] * c["d"]], 1)
    return (x.unflatten(1, (-1, c["d"])) for x in (q, k, v))


def _rotate(s, x, weight):
    c = s["case"]
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * weight
    rot, half = c["rot"], c["rot"] // 2
    at = s["positions"].long()[s["axes"]].t()  # the position of each pair
    pair = torch.arange(half, device="cuda")
    cos, sin = s["cos_sin"][at, pair][:, None], s["cos_sin"][at, half + pair][:, None]
    if c["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _quantize(x):
    """E4M3 codes and E8M0 scale bytes of x [.., head dim] in groups of 32: the smallest power of
    two that brings a group's largest element to 448 or below."""
    x = x.unflatten(-1, (-1, 32))
    m, e = torch.frexp(x.abs().amax(-1))
    e = torch.where(m > 0, e - 9 + (m > 0.875).int(), -127).clamp(min=-127)
    codes = torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8).flatten(-2), (e + 127).to(torch.uint8)


def _planes(s, x):
    """The element and the scale plane of a quantized pool as the values that they stand for."""
    n = math.prod(s["shape"])
    return s[x][:n].view(torch.float8_e4m3fn), s[x][n:].view(torch.float8_e8m0fnu)


def _rope_outputs(s, out):
    if s["case"]["dtype"] == "mxfp8":
        return (out, *_planes(s, "k"), *_planes(s, "v"))
    return out, s["k"], s["v"]


def _plain_rope(s):
    c, (q, k, v) = s["case"], _split(s)
    out, k = _rotate(s, q, s["wq"]).to(q.dtype), _rotate(s, k, s["wk"])
    for x, y in (("k", k), ("v", v.float())):
        if c["dtype"] != "mxfp8":
            s[x].view(-1, c["hkv"], c["d"])[s["slots"]] = y.to(v.dtype)
            continue
        blocks, p, hkv, d = s["shape"]
        n = math.prod(s["shape"])
        codes, scales = _quantize(y)
        s[x][:n].view(-1, hkv, d)[s["slots"]] = codes
        s[x][n:].view(blocks, hkv, p, d // 32)[s["slots"] // p, :, s["slots"] % p] = scales
    return _rope_outputs(s, out)


def _plain_window(s):
    c = s["case"]
    batch, hq, hkv, d, p = c["batch"], c["hq"], c["hkv"], c["d"], c["p"]
    lens, sinks = s["lens"].long()[:, None], min(c["sinks"], c["hi"])
    width = min(c["window"], c["hi"])
    at = torch.cat([torch.arange(sinks, device="cuda").expand(batch, -1),
                    lens - width + torch.arange(width, device="cuda")], 1)
    first = torch.arange(sinks + width, device="cuda") < sinks
    seen = (at >= 0) & (at < lens) & (first | (at >= sinks))  # a sink inside the window counts once
    at = at.clamp(min=0).minimum(lens - 1)
    rows = torch.gather(s["tables"].long(), 1, at // p) * p + at % p

    def history(pool):
        if c["dtype"] != "mxfp8":
            return pool.view(-1, hkv, d)[rows].float().transpose(1, 2)
        n = math.prod(s["shape"])
        codes = pool[:n].view(-1, hkv, d)[rows].view(torch.float8_e4m3fn).float()
        scales = pool[n:].view(-1, hkv, p, d // 32)[rows // p, :, rows % p].float()
        return (codes * torch.exp2(scales - 127).repeat_interleave(32, -1)).transpose(1, 2)

    q = s["q"].float().view(batch, hkv, hq // hkv, d)
    x = (q @ history(s["k"]).transpose(-1, -2)) * s["scale"]
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True)
    out = (e / total) @ history(s["v"])
    lse = (torch.log(total) + top).view(batch, hq)
    return out.view(batch, hq, d).to(s["q"].dtype), lse


def _plain_verify(s):
    c, n = s["case"], s["max_draft"]
    batch = c["batch"]
    ptr, r = s["ptr"].long(), torch.arange(batch, device="cuda")
    node = torch.arange(n, device="cuda")
    row = (ptr[:-1, None] + node).clamp(max=s["tokens"].numel() - 1)
    held = (ptr[1:] - ptr[:-1])[:, None]
    up = torch.where(node < held, s["parent"], -1)
    tok, u = s["tokens"].long()[row], s["u"].double()[row]
    above = row.gather(1, up.clamp(min=0))  # the parent's row
    p = s["p"][above, tok].double()
    q = s["q"][above, tok].double() if c["sampled"] else torch.ones_like(p)
    if not c["tree"]:
        ok = (u * q < p) & (up >= 0)
        ok[:, 0] = True
        kept = ok.long().cumprod(1).bool()
        at = kept.sum(1) - 1
        last = (at + 1 < held[:, 0])  # a token was turned down there
        less = last.double()
        gone = torch.zeros(batch, n, dtype=torch.bool, device="cuda")
        gone.scatter_(1, (at + 1).clamp(max=n - 1)[:, None], last[:, None])
    else:
        # children in ascending order: one that is accepted is the node to go on from
        at = torch.zeros(batch, dtype=torch.long, device="cuda")
        kept, gone = (torch.zeros(batch, n, dtype=torch.bool, device="cuda") for _ in range(2))
        kept[:, 0] = True
        less, mass = (torch.full((batch,), x, dtype=torch.float64, device="cuda") for x in (0.0, 1.0))
        for i in range(1, n):
            child = up[:, i] == at
            if c["sampled"]:
                part = (p[:, i] - less * q[:, i]).clamp(min=0)
            else:
                twice = (gone & (tok == tok[:, i : i + 1])).any(1)
                part = torch.where(twice, 0.0, p[:, i])
            yes = child & (u[:, i] * q[:, i] * mass < part)
            no = child & ~yes
            kept[:, i] = yes
            gone[:, i] = no
            gone &= ~yes[:, None]
            if c["sampled"]:
                less = torch.where(yes, 0.0, less + torch.where(no, mass, 0.0))
                here = row[r, at]
                rest = s["p"][here].double() - less[:, None] * s["q"][here].double()
                mass = torch.where(yes, 1.0, torch.where(no, rest.clamp_(min=0).sum(1), mass))
            else:
                mass = torch.where(yes, 1.0, mass - torch.where(no, part, 0.0))
            at = torch.where(yes, i, at)
    here = row[r, at]
    whole = s["p"][here].double()
    if c["sampled"]:
        rest = (whole - less[:, None] * s["q"][here].double()).clamp_(min=0)
    else:
        rest = whole.scatter_reduce(1, tok, torch.where(gone, 0.0, math.inf).double(), "amin")
    rest = torch.where(rest.sum(1, keepdim=True) > 0, rest, whole)
    upto = rest.cumsum(1)
    target = u[:, :1] * upto[:, -1:]
    token = (upto <= target).sum(1).clamp(max=c["vocab"] - 1).to(torch.int32)
    some = held[:, 0] > 0
    kept &= node < held
    keep = torch.sort(torch.where(kept, node, n), dim=1).values
    keep = torch.where(keep < n, keep, -1).to(torch.int32)[:, None]
    return keep, kept.sum(1).to(torch.int32), torch.where(some, token, -1)


# ---------------------------------------------------------------- the framework's calls
def _pools(s, pkv):
    """The pools as the framework takes them."""
    if s["case"]["dtype"] != "mxfp8":
        return s["k"], s["v"]
    if "mx" not in s:
        s["mx"] = [pkv.MxPool(*s["shape"], buf=s[x]) for x in ("k", "v")]
    return s["mx"]


def _own_blocks(s, pkv):
    kind, zeros, pool, table, free = s["case"]["kind"], s["zeros"], s["pool"], s["tables"], s["free"]
    if kind == "resume":
        lens, _, _, _, = pkv.kv_blocks_update(pool, table, s["lens"], zeros, free, s["count"],
                                              free_count_out=s["count_out"], **s["b"])
        lens, ptr, slots, pos = pkv.kv_blocks_update(pool, table, lens, s["lens"], free, s["count_out"],
                                                     **s["a"])
        return table, free, lens, ptr, slots, pos, s["count_out"]
    lens, ptr, slots, pos = pkv.kv_blocks_update(pool, table, s["lens"], s["add"], free, s["count"],
                                                 base_lens=s["lens"], free_count_out=s["count_out"],
                                                 **s["a"])
    if kind == "drafts":
        lens, _, _, _ = pkv.kv_blocks_update(pool, table, lens, zeros, free, s["count_out"],
                                             base_lens=s["lens"], **s["b"])
    return table, free, lens, ptr, slots, pos, s["count_out"]


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"blocks": _plain_blocks, "rope": _plain_rope, "window": _plain_window,
                "verify": _plain_verify}[op](s)
    from paged_kv_cache_41_gb300 import pkv

    if op == "blocks":
        return _own_blocks(s, pkv)
    if op == "rope":
        q, k, v = _split(s)
        pkv.qk_norm_rope_append(q, k, v, *_pools(s, pkv), s["slots"], s["positions"], s["cos_sin"],
                                q_weight=s["wq"], k_weight=s["wk"], eps=1e-6, axis_of=s["axis_of"],
                                interleaved=s["case"]["interleaved"], out=s["out"])
        return _rope_outputs(s, s["out"])
    if op == "window":
        c, (k, v) = s["case"], _pools(s, pkv)
        if "ws" not in s:
            n = pkv.decode_window_workspace_bytes(k, c["batch"], c["hq"], s["tables"].shape[1],
                                                  c["window"], c["sinks"])
            s["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        pkv.paged_attention_decode_window(s["q"], k, v, s["tables"], s["lens"], s["scale"],
                                          window=c["window"], num_sinks=c["sinks"], out=s["out"],
                                          lse=s["lse"], workspace=s["ws"])
        return s["out"], s["lse"]
    pkv.draft_verify(s["p"], s["tokens"], s["ptr"], s["u"], max_draft=s["max_draft"], draft_probs=s["q"],
                     masks=s["masks"], keep=s["keep"], keep_lens=s["keep_lens"], next_tokens=s["next"])
    return s["keep"], s["keep_lens"], s["next"]


# ---------------------------------------------------------------- in 64 bits
def exact(case, seed):
    if case["op"] in ("blocks", "verify"):
        return None  # whole numbers
    s = prepare(case, seed)
    hq, hkv, d, p = case["hq"], case["hkv"], case["d"], case["p"]
    if case["op"] == "rope":
        n, rot = s["qkv"].shape[0], case["rot"]
        x = s["qkv"].double().view(n, hq + 2 * hkv, d)
        for lo, hi, w in ((0, hq, s["wq"]), (hq, hq + hkv, s["wk"])):
            if w is not None:
                y = x[:, lo:hi]
                x[:, lo:hi] = y / torch.sqrt((y * y).sum(-1, keepdim=True) / d + 1e-6) * w.double()
        angles = torch.empty(n, rot, dtype=torch.float64, device="cuda")
        for j, axis in enumerate(s["axis_of"]):
            at = s["positions"][axis].long()
            angles[:, j] = s["cos_sin"][at, j].double()
            angles[:, rot // 2 + j] = s["cos_sin"][at, rot // 2 + j].double()
        turned = x.clone()
        for j in range(rot // 2):
            a, b = (2 * j, 2 * j + 1) if case["interleaved"] else (j, rot // 2 + j)
            z = torch.complex(x[:, : hq + hkv, a], x[:, : hq + hkv, b])
            z = z * torch.complex(angles[:, j], angles[:, rot // 2 + j])[:, None]
            turned[:, : hq + hkv, a], turned[:, : hq + hkv, b] = z.real, z.imag
        out = [turned[:, :hq]]
        for rows in (turned[:, hq : hq + hkv], turned[:, hq + hkv :]):
            blocks = s["shape"][0]
            if case["dtype"] != "mxfp8":
                pool = torch.zeros(blocks * p, hkv, d, dtype=torch.float64, device="cuda")
                pool[s["slots"]] = rows
                out.append(pool.view(s["shape"]))
                continue
            groups = rows.reshape(n, hkv, d // 32, 32)
            # a group whose largest element is 448 times a power of two takes that power
            power = torch.ceil(torch.log2(groups.abs().amax(-1) / 448).clamp(min=-127) - 1e-12)
            codes = (groups / torch.exp2(power)[..., None]).float().to(torch.float8_e4m3fn).double()
            plane = torch.zeros(blocks * p, hkv, d, dtype=torch.float64, device="cuda")
            plane[s["slots"]] = codes.view(n, hkv, d)
            scales = torch.full((blocks, hkv, p, d // 32), 2.0 ** -127, dtype=torch.float64, device="cuda")
            scales[s["slots"] // p, :, s["slots"] % p] = torch.exp2(power)
            out += [plane.flatten(), scales.flatten()]
        return tuple(out)

    def rows64(pool, ids):
        if case["dtype"] != "mxfp8":
            return pool[ids].reshape(-1, hkv, d).double()
        n = pool.numel() // 33 * 32
        codes = pool[:n].view(-1, p, hkv, d)[ids].view(torch.float8_e4m3fn).double()
        power = pool[n:].view(-1, hkv, p, d // 32)[ids].double().permute(0, 2, 1, 3) - 127.0
        return torch.ldexp(codes, power.repeat_interleave(32, dim=3)).reshape(-1, hkv, d)

    outs, lses = [], []
    for r, t in enumerate(s["lens"].tolist()):
        ids = s["tables"][r, : -(-t // p)].long()
        at = torch.arange(t, device="cuda")
        at = at[(at < case["sinks"]) | (at >= t - case["window"])]
        k, v = (rows64(s[x], ids)[at] for x in ("k", "v"))
        q = s["q"][r].double().view(hkv, hq // hkv, d) * s["scale"]
        x = torch.einsum("hgd,thd->hgt", q, k)
        lse = torch.logsumexp(x, -1)
        outs.append(torch.einsum("hgt,thd->hgd", torch.exp(x - lse[..., None]), v).reshape(hq, d))
        lses.append(lse.reshape(hq))
    return torch.stack(outs), torch.stack(lses)
