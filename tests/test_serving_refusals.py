"""What the draft-tree and eviction calls refuse before any launch (no GPU)."""
import ctypes

import pytest
import torch

from paged_kv_cache_41_gb300 import pkv

P = ctypes.c_void_p
A = P(1 << 20)       # a 16- and 256-byte aligned address, never followed
ODD = P((1 << 20) + 8)
BIG = 1 << 60


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_41_gb300 import build
    build.build_all()
    return pkv.load_library()


def desc(nb=64, p=16, hkv=2, d=64, dtype=pkv.PKV_BF16):
    return pkv.CacheDesc(nb, p, hkv, d, dtype)


BAD, UNSUP = pkv.PKV_ERR_INVALID_ARG, pkv.PKV_ERR_UNSUPPORTED


def draft(lib, c=None, out=A, lse=A, q=A, k=A, v=A, tables=A, mb=4, ctx=A, ptr=A, masks=A, b=2, rows=6,
          n=3, hq=4, scale=0.1, ws=A, wsb=BIG):
    c = c or desc()
    return lib.pkv_draft_tree_attention(ctypes.byref(c), out, lse, q, k, v, tables, mb, ctx, ptr, masks, b,
                                        rows, n, hq, scale, ws, wsb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(out=None), BAD), (dict(q=None), BAD), (dict(k=None), BAD), (dict(v=None), BAD),
    (dict(tables=None), BAD), (dict(ctx=None), BAD), (dict(ptr=None), BAD), (dict(ws=None), BAD),
    (dict(out=ODD), BAD), (dict(q=ODD), BAD), (dict(k=ODD), BAD), (dict(v=ODD), BAD), (dict(ws=ODD), BAD),
    (dict(wsb=0), BAD), (dict(mb=0), BAD), (dict(b=-1), BAD), (dict(rows=-1), BAD), (dict(n=0), BAD),
    (dict(n=65), BAD), (dict(hq=3), BAD), (dict(hq=0), BAD), (dict(hq=6), UNSUP), (dict(hq=32), UNSUP),
    (dict(scale=float("nan")), BAD), (dict(scale=float("inf")), BAD), (dict(b=65536), UNSUP),
    (dict(c=desc(d=96)), UNSUP), (dict(c=desc(p=8)), UNSUP), (dict(c=desc(p=48)), UNSUP),
    (dict(c=desc(p=512)), UNSUP), (dict(c=desc(dtype=7)), BAD), (dict(c=desc(nb=0)), BAD),
    (dict(b=0), 0), (dict(rows=0), 0)])
def test_draft_arguments(lib, kw, want):
    assert draft(lib, **kw) == want


def test_draft_workspace_size(lib):
    c = desc()
    size = lib.pkv_draft_tree_workspace_bytes(ctypes.byref(c), 2, 4, 3, 4)
    assert size > 0
    assert draft(lib, wsb=size - 1) == BAD
    for args in ((0, 4, 3, 4), (2, 3, 3, 4), (2, 4, 0, 4), (2, 4, 65, 4), (2, 4, 3, 0), (65536, 4, 3, 4)):
        assert lib.pkv_draft_tree_workspace_bytes(ctypes.byref(c), *args) == 0


def weigh(lib, c=None, out=A, lse=A, w=A, ws_=10, decay=1.0, q=A, k=A, v=A, tables=A, mb=4, lens=A, b=2,
          hq=4, scale=0.1, ws=A, wsb=BIG):
    c = c or desc()
    return lib.pkv_paged_attention_decode_weights(ctypes.byref(c), out, lse, w, ws_, decay, q, k, v, tables,
                                                  mb, lens, b, hq, scale, ws, wsb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(w=None), BAD), (dict(ws_=0), BAD), (dict(decay=float("nan")), BAD),
    (dict(decay=float("inf")), BAD), (dict(out=None), BAD), (dict(q=None), BAD), (dict(k=None), BAD),
    (dict(v=None), BAD), (dict(tables=None), BAD), (dict(lens=None), BAD), (dict(ws=None), BAD),
    (dict(ws=ODD), BAD), (dict(wsb=0), BAD), (dict(q=ODD), BAD), (dict(out=ODD), BAD), (dict(mb=0), BAD),
    (dict(b=-1), BAD), (dict(hq=3), BAD), (dict(hq=6), UNSUP), (dict(scale=float("nan")), BAD),
    (dict(c=desc(d=96)), UNSUP), (dict(c=desc(dtype=pkv.PKV_MXFP8), hq=16), UNSUP), (dict(b=65536), UNSUP),
    (dict(b=0), 0)])
def test_weigh_arguments(lib, kw, want):
    assert weigh(lib, **kw) == want


def test_weigh_workspace_size(lib):
    c = desc()
    size = lib.pkv_decode_weights_workspace_bytes(ctypes.byref(c), 2, 4, 4)
    assert size > 0
    assert weigh(lib, wsb=size - 1) == BAD
    assert lib.pkv_decode_weights_workspace_bytes(ctypes.byref(c), 0, 4, 4) == 0
    assert lib.pkv_decode_weights_workspace_bytes(ctypes.byref(c), 2, 5, 4) == 0


def select(lib, w=A, stride=100, lens=A, b=2, hkv=2, budget=10, sinks=1, recent=2, keep=A, new=A):
    return lib.pkv_kv_evict_select(w, stride, lens, b, hkv, budget, sinks, recent, keep, new, None)


@pytest.mark.parametrize("kw,want", [
    (dict(w=None), BAD), (dict(lens=None), BAD), (dict(keep=None), BAD), (dict(new=None), BAD),
    (dict(stride=0), BAD), (dict(b=-1), BAD), (dict(hkv=0), BAD), (dict(budget=0), BAD),
    (dict(sinks=-1), BAD), (dict(recent=-1), BAD), (dict(sinks=9), BAD), (dict(recent=10), BAD),
    (dict(sinks=2**31 - 1, recent=2**31 - 1), BAD), (dict(b=65536), UNSUP), (dict(hkv=65536), UNSUP),
    (dict(b=0), 0)])
def test_select_arguments(lib, kw, want):
    assert select(lib, **kw) == want


def test_select_refuses_new_lengths_over_the_old_and_rows_past_32_bits(lib):
    for off in (-4, 0, 4):  # two sequences: eight bytes each
        assert select(lib, new=P((1 << 20) + off)) == BAD
    far = P(1 << 21)
    assert select(lib, stride=2**31 - 2**16 + 1, new=far) == UNSUP
    assert select(lib, budget=2**31 - 2**16 + 1, new=far) == UNSUP


def compact(lib, c=None, k=A, v=A, w=None, stride=0, tables=A, mb=4, lens=A, base=None, keep=A, heads=2,
            ks=10, kl=A, b=2):
    c = c or desc()
    return lib.pkv_kv_compact(ctypes.byref(c), k, v, w, stride, tables, mb, lens, base, keep, heads, ks, kl,
                              b, None)


@pytest.mark.parametrize("kw,want", [
    (dict(k=None), BAD), (dict(v=None), BAD), (dict(tables=None), BAD), (dict(lens=None), BAD),
    (dict(keep=None), BAD), (dict(kl=None), BAD), (dict(k=ODD), BAD), (dict(v=ODD), BAD),
    (dict(heads=3), BAD), (dict(heads=0), BAD), (dict(ks=-1), BAD), (dict(mb=0), BAD), (dict(b=-1), BAD),
    (dict(w=A, stride=0), BAD), (dict(c=desc(d=4)), UNSUP), (dict(c=desc(d=3, dtype=0)), UNSUP),
    (dict(c=desc(d=48, dtype=pkv.PKV_MXFP8)), UNSUP), (dict(c=desc(d=16384)), UNSUP),
    (dict(b=65536), UNSUP), (dict(c=desc(nb=2**31)), UNSUP), (dict(b=0), 0), (dict(ks=0), 0)])
def test_compact_arguments(lib, kw, want):
    assert compact(lib, **kw) == want


def test_compact_refuses_pools_that_overlap(lib):
    c = desc()  # 64 * 16 * 2 * 64 bf16 elements: 262144 bytes a pool
    for off in (0, 16, 262144 - 16):
        assert compact(lib, c=c, k=A, v=P((1 << 20) + off)) == BAD
        assert compact(lib, c=c, k=P((1 << 20) + off), v=A) == BAD
    mx = desc(dtype=pkv.PKV_MXFP8)  # 131072 codes, 4096 scales
    assert compact(lib, c=mx, k=A, v=P((1 << 20) + 131072)) == BAD


def test_draft_refuses_a_bf16_pool_past_its_coordinates(lib):
    assert draft(lib, c=desc(nb=2**30 + 8)) == UNSUP
    assert lib.pkv_draft_tree_workspace_bytes(ctypes.byref(desc(nb=2**30 + 8)), 2, 4, 3, 4) == 0


# ------------------------------------------------------------ the binding
def host(nb=8, p=16, hkv=2, d=64, dtype=torch.bfloat16):
    return torch.zeros(nb, p, hkv, d, dtype=dtype)


I32 = torch.int32


def test_binding_refuses_host_tensors_and_wrong_shapes(lib):
    k = host()
    t, n = torch.zeros(2, 4, dtype=I32), torch.zeros(2, dtype=I32)
    q = torch.zeros(6, 4, 64, dtype=torch.bfloat16)
    ptr = torch.zeros(3, dtype=I32)
    w = torch.zeros(2, 2, 70)
    good = [
        lambda **o: pkv.draft_tree_attention(*[o.get(x, y) for x, y in zip(
            ("q", "k", "v", "t", "n", "ptr"), (q, k, k, t, n, ptr))], 0.1, max_draft=3,
            masks=o.get("masks"), out=o.get("out"), lse=o.get("lse")),
        lambda **o: pkv.paged_attention_decode_weights(*[o.get(x, y) for x, y in zip(
            ("q", "k", "v", "t", "n", "w"), (q[:2], k, k, t, n, w))], 0.1, out=o.get("out"), lse=o.get("lse")),
        lambda **o: pkv.kv_evict_select(o.get("w", w), o.get("n", n), 10, keep=o.get("keep"),
                                        new_lens=o.get("new")),
        lambda **o: pkv.kv_compact(*[o.get(x, y) for x, y in zip(
            ("k", "v", "t", "n", "keep", "kl"), (k, k, t, n, torch.zeros(2, 2, 5, dtype=I32), n))],
            weights=o.get("w"), base_lens=o.get("base")),
    ]
    for f in good:  # every shape right: refused for being on the host
        with pytest.raises(ValueError, match="current CUDA device"):
            f()
    wrong = [
        (0, dict(q=q.float())), (0, dict(q=q[:, :, :32])), (0, dict(q=q.transpose(0, 1))),
        (0, dict(v=host(nb=9))), (0, dict(v=host(dtype=torch.float32))), (0, dict(t=t.long())),
        (0, dict(n=n[:1])), (0, dict(ptr=ptr[:2])), (0, dict(masks=torch.zeros(5, dtype=torch.int64))),
        (0, dict(masks=torch.zeros(6, dtype=I32))), (0, dict(out=q[:5])), (0, dict(lse=torch.zeros(6, 3))),
        (1, dict(w=w.double())), (1, dict(w=w[:1])), (1, dict(w=torch.zeros(2, 2, 70).transpose(1, 2))),
        (1, dict(w=torch.zeros(2, 2, 140)[:, :, ::2])), (1, dict(w=torch.zeros(2, 3, 70)[:, :2])),
        (1, dict(n=n.long())), (1, dict(out=q)), (1, dict(t=t[:1])),
        (2, dict(w=w.half())), (2, dict(n=n[:1])), (2, dict(keep=torch.zeros(2, 2, 9, dtype=I32))),
        (2, dict(new=n.long())),
        (3, dict(keep=torch.zeros(1, 2, 5, dtype=I32))), (3, dict(kl=n.long())), (3, dict(base=n[:1])),
        (3, dict(w=w[:, :1])), (3, dict(v=host(hkv=1))),
    ]
    for i, o in wrong:
        with pytest.raises(ValueError) as e:
            good[i](**o)
        assert "current CUDA device" not in str(e.value), o


def test_mxpool_over_a_buffer():
    buf = torch.zeros(2 * 16 * 2 * 64 * 33 // 32, dtype=torch.uint8)
    pool = pkv.MxPool(2, 16, 2, 64, buf=buf)
    assert pool.buf is buf and pool.elements.shape == (2, 16, 2, 64)
    for bad in (buf[:-1], buf.float(), buf.view(2, -1)):
        with pytest.raises(ValueError):
            pkv.MxPool(2, 16, 2, 64, buf=bad)
