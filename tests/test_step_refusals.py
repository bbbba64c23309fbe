"""What the calls of the step around the cache refuse before any launch (no GPU)."""
import ctypes

import pytest
import torch

from paged_kv_cache_41_gb300 import pkv

P = ctypes.c_void_p
A = P(1 << 20)       # a 16- and 256-byte aligned address, never followed
FAR = P(1 << 24)
ODD = P((1 << 20) + 8)
BIG = 1 << 60
BAD, UNSUP = pkv.PKV_ERR_INVALID_ARG, pkv.PKV_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_41_gb300 import build
    build.build_all()
    return pkv.load_library()


def desc(nb=64, p=16, hkv=2, d=64, dtype=pkv.PKV_BF16):
    return pkv.CacheDesc(nb, p, hkv, d, dtype)


def blocks(lib, c=None, tables=A, mb=4, lens=A, base=None, add=A, b=2, sinks=0, window=0, free=A, cin=A,
           cout=A, out=FAR, ptr=A, slots=A, pos=A, rows=5):
    c = c or desc()
    return lib.pkv_kv_blocks_update(ctypes.byref(c), tables, mb, lens, base, add, b, sinks, window, free, cin,
                                    cout, out, ptr, slots, pos, rows, None)


@pytest.mark.parametrize("kw,want", [
    (dict(tables=None), BAD), (dict(lens=None), BAD), (dict(add=None), BAD), (dict(free=None), BAD),
    (dict(cin=None), BAD), (dict(cout=None), BAD), (dict(out=None), BAD), (dict(ptr=None), BAD),
    (dict(slots=None), BAD), (dict(mb=0), BAD), (dict(b=-1), BAD), (dict(sinks=-1), BAD),
    (dict(window=-1), BAD), (dict(rows=-1), BAD), (dict(c=desc(nb=0)), BAD), (dict(c=desc(p=0)), BAD),
    (dict(b=65536), UNSUP), (dict(rows=2**31), UNSUP), (dict(c=desc(nb=2**31)), UNSUP),
    (dict(out=A), BAD), (dict(out=P((1 << 20) + 4)), BAD), (dict(out=P((1 << 20) - 4)), BAD),
    (dict(base=FAR), BAD), (dict(add=P((1 << 24) + 4)), BAD)])
def test_blocks_arguments(lib, kw, want):
    assert blocks(lib, **kw) == want


def rope(lib, c=None, out=A, k=A, v=A, q=A, qs=256, kk=A, ks=128, vv=A, vs=128, slots=A, pos=A, ps=10, axes=1,
         axis=None, table=A, far=100, rot=64, inter=0, qw=A, kw_=A, eps=1e-6, n=3, hq=4):
    c = c or desc()
    return lib.pkv_qk_norm_rope_append(ctypes.byref(c), out, k, v, q, qs, kk, ks, vv, vs, slots, pos, ps, axes,
                                       axis, table, far, rot, inter, qw, kw_, eps, n, hq, None)


@pytest.mark.parametrize("kw,want", [
    (dict(out=None), BAD), (dict(k=None), BAD), (dict(v=None), BAD), (dict(q=None), BAD), (dict(kk=None), BAD),
    (dict(vv=None), BAD), (dict(slots=None), BAD), (dict(pos=None), BAD), (dict(table=None), BAD),
    (dict(far=0), BAD), (dict(far=-1), BAD),
    (dict(out=ODD), BAD), (dict(k=ODD), BAD), (dict(v=ODD), BAD), (dict(q=ODD), BAD), (dict(kk=ODD), BAD),
    (dict(vv=ODD), BAD), (dict(table=ODD), BAD), (dict(qw=ODD), BAD), (dict(kw_=ODD), BAD),
    (dict(qs=255), BAD), (dict(qs=260), BAD), (dict(ks=127), BAD), (dict(ks=132), BAD), (dict(vs=0), BAD),
    (dict(c=desc(dtype=pkv.PKV_F32), vs=130), BAD),
    (dict(axes=0), BAD), (dict(axes=4), UNSUP), (dict(axes=2, ps=2), BAD),
    (dict(rot=-16), BAD), (dict(rot=80), BAD), (dict(rot=8), UNSUP), (dict(rot=24), UNSUP),
    (dict(axis=bytes([0] * 31 + [1])), BAD), (dict(axes=3, axis=bytes([2] * 31 + [3])), BAD),
    (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD), (dict(eps=float("inf")), BAD),
    (dict(n=-1), BAD), (dict(hq=0), BAD), (dict(c=desc(d=96)), UNSUP), (dict(c=desc(d=256)), UNSUP),
    (dict(c=desc(dtype=9)), BAD), (dict(n=2**40), UNSUP), (dict(n=0), 0)])
def test_rope_arguments(lib, kw, want):
    assert rope(lib, **kw) == want


def window(lib, c=None, out=A, lse=A, q=A, k=A, v=A, tables=A, mb=4, lens=A, b=2, hq=4, scale=0.1, w=20, sinks=4,
           ws=A, wsb=BIG):
    c = c or desc()
    return lib.pkv_paged_attention_decode_window(ctypes.byref(c), out, lse, q, k, v, tables, mb, lens, b, hq,
                                                 scale, w, sinks, ws, wsb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(w=0), BAD), (dict(w=-1), BAD), (dict(sinks=-1), BAD), (dict(out=None), BAD), (dict(q=None), BAD),
    (dict(k=None), BAD), (dict(v=None), BAD), (dict(tables=None), BAD), (dict(lens=None), BAD),
    (dict(ws=None), BAD), (dict(ws=ODD), BAD), (dict(wsb=0), BAD), (dict(q=ODD), BAD), (dict(out=ODD), BAD),
    (dict(mb=0), BAD), (dict(b=-1), BAD), (dict(hq=3), BAD), (dict(hq=6), UNSUP),
    (dict(scale=float("nan")), BAD), (dict(c=desc(d=96)), UNSUP), (dict(c=desc(p=48)), UNSUP),
    (dict(c=desc(dtype=pkv.PKV_MXFP8), hq=16), UNSUP), (dict(b=65536), UNSUP), (dict(b=0), 0)])
def test_window_arguments(lib, kw, want):
    assert window(lib, **kw) == want


def test_window_workspace_size(lib):
    c = ctypes.byref(desc())
    size = lib.pkv_decode_window_workspace_bytes
    need = size(c, 2, 4, 4, 20, 4)
    assert need > 0 and window(lib, wsb=need - 1) == BAD
    # a few rows seen of a long table ask for no more than a short table does
    assert size(c, 2, 4, 100000, 20, 4) == size(c, 2, 4, 8, 20, 4)
    # and a window over everything, where the plain decode's split is taken, what that does
    f32 = ctypes.byref(desc(dtype=pkv.PKV_F32))
    assert size(f32, 2, 4, 100000, 2**31 - 1, 2**31 - 1) == lib.pkv_decode_workspace_bytes(f32, 2, 4, 100000, 0)
    assert size(c, 2, 4, 100000, 2**31 - 1, 2**31 - 1) > need
    for args in ((0, 4, 4, 20, 4), (2, 3, 4, 20, 4), (2, 4, 0, 20, 4), (2, 4, 4, 0, 4), (2, 4, 4, 20, -1)):
        assert size(c, *args) == 0


def verify(lib, p=A, ps=100, q=A, qs=100, vocab=100, tok=A, ptr=A, masks=A, u=A, b=2, rows=6, n=3, keep=A, kl=A,
           nxt=A):
    return lib.pkv_draft_verify(p, ps, q, qs, vocab, tok, ptr, masks, u, b, rows, n, keep, kl, nxt, None)


@pytest.mark.parametrize("kw,want", [
    (dict(p=None), BAD), (dict(tok=None), BAD), (dict(ptr=None), BAD), (dict(u=None), BAD), (dict(keep=None), BAD),
    (dict(kl=None), BAD), (dict(nxt=None), BAD), (dict(ps=99), BAD), (dict(qs=99), BAD), (dict(vocab=0), BAD),
    (dict(b=-1), BAD), (dict(rows=-1), BAD), (dict(n=0), BAD), (dict(n=65), BAD), (dict(b=65536), UNSUP),
    (dict(vocab=2**30 + 1, ps=2**31, qs=2**31), UNSUP), (dict(b=0), 0)])
def test_verify_arguments(lib, kw, want):
    assert verify(lib, **kw) == want


# ------------------------------------------------------------ the binding
I32, I64 = torch.int32, torch.int64


def test_binding_refuses_host_tensors_and_wrong_shapes(lib):
    k = torch.zeros(8, 16, 2, 64, dtype=torch.bfloat16)
    t, n, one = torch.zeros(2, 4, dtype=I32), torch.zeros(2, dtype=I32), torch.zeros(1, dtype=I32)
    qkv = torch.zeros(3, 512, dtype=torch.bfloat16)
    q, kk, vv = (x.unflatten(1, (-1, 64)) for x in qkv.split([256, 128, 128], 1))
    probs, ptr = torch.zeros(6, 100), torch.zeros(3, dtype=I32)

    def blocks(**o):
        o = {"tables": t, "lens": n, "add": n, "free": torch.zeros(8, dtype=I32), "count": one, **o}
        pkv.kv_blocks_update(k, o.pop("tables"), o.pop("lens"), o.pop("add"), o.pop("free"), o.pop("count"),
                             **{"num_rows": 5, **o})

    def rope(**o):
        o = {"q": q, "k": kk, "v": vv, "kc": k, "vc": k, "slots": torch.zeros(3, dtype=I64),
             "pos": torch.zeros(3, dtype=I32), "table": torch.zeros(9, 64), **o}
        pkv.qk_norm_rope_append(*[o.pop(x) for x in ("q", "k", "v", "kc", "vc", "slots", "pos", "table")], **o)

    def window(**o):
        o = {"q": torch.zeros(2, 4, 64, dtype=torch.bfloat16), "k": k, "v": k, "tables": t, "lens": n, **o}
        pkv.paged_attention_decode_window(*[o.pop(x) for x in ("q", "k", "v", "tables", "lens")], 0.1,
                                          **{"window": 20, **o})

    def verify(**o):
        o = {"p": probs, "tok": torch.zeros(6, dtype=I32), "ptr": ptr, "u": torch.zeros(6), **o}
        pkv.draft_verify(*[o.pop(x) for x in ("p", "tok", "ptr", "u")], **{"max_draft": 3, **o})

    for f in (blocks, rope, window, verify):  # every shape right: refused for being on the host
        with pytest.raises(ValueError, match="current CUDA device"):
            f()
    wrong = [
        (blocks, dict(tables=t.long())), (blocks, dict(lens=n[:1])), (blocks, dict(add=n.long())),
        (blocks, dict(free=torch.zeros(7, dtype=I32))), (blocks, dict(count=n)), (blocks, dict(base_lens=n[:1])),
        (blocks, dict(out_lens=n.long())), (blocks, dict(row_ptr=n)), (blocks, dict(slots=torch.zeros(5, dtype=I32))),
        (blocks, dict(num_rows=4, slots=torch.zeros(5, dtype=I64))), (blocks, dict(num_rows=None)),
        (blocks, dict(positions=torch.zeros(5, dtype=I64))), (blocks, dict(free_count_out=n)),
        (blocks, dict(tables=torch.zeros(4, 2, dtype=I32).t())),
        (rope, dict(q=q.float())), (rope, dict(q=q[:, :, :32])), (rope, dict(q=q[:, ::2])),
        (rope, dict(k=kk[:, :1])), (rope, dict(v=vv.transpose(0, 1))), (rope, dict(slots=n)),
        (rope, dict(pos=torch.zeros(3, dtype=I64))), (rope, dict(pos=torch.zeros(2, 4, dtype=I32))),
        (rope, dict(pos=torch.zeros(3, 2, dtype=I32).t())), (rope, dict(table=torch.zeros(9, 64).double())),
        (rope, dict(axis_of=[0] * 31)), (rope, dict(q_weight=torch.zeros(32))),
        (rope, dict(k_weight=torch.zeros(64).bfloat16())), (rope, dict(out=q)),
        (rope, dict(vc=torch.zeros(9, 16, 2, 64, dtype=torch.bfloat16))),
        (window, dict(q=torch.zeros(2, 4, 64))), (window, dict(tables=t[:1])), (window, dict(lens=n.long())),
        (window, dict(lse=torch.zeros(2, 3))), (window, dict(v=k.float())),
        (verify, dict(p=probs.double())), (verify, dict(p=probs[:, ::2])), (verify, dict(tok=torch.zeros(5, dtype=I32))),
        (verify, dict(u=torch.zeros(6).double())), (verify, dict(draft_probs=probs[:5])),
        (verify, dict(masks=torch.zeros(6, dtype=I32))), (verify, dict(keep=torch.zeros(2, 3, dtype=I32))),
        (verify, dict(keep_lens=ptr)), (verify, dict(next_tokens=n.long())),
    ]
    for f, o in wrong:
        with pytest.raises(ValueError) as e:
            f(**o)
        assert "current CUDA device" not in str(e.value), o


@pytest.mark.parametrize("size", [2**31, 2**32 + 7, 2**40])
def test_binding_refuses_windows_past_32_bits(lib, size):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    kc = torch.zeros(4, 16, 2, 64)
    q = torch.zeros(1, 4, 64)
    for kw in (dict(window=size), dict(window=5, num_sinks=size)):
        with pytest.raises(ValueError, match="2\\*\\*31"):
            pkv.paged_attention_decode_window(q, kc, kc, i32(1, 2), i32(1), 1.0, **kw)
        with pytest.raises(ValueError, match="2\\*\\*31"):
            pkv.decode_window_workspace_bytes(kc, 1, 4, 2, kw["window"], kw.get("num_sinks", 0))
        with pytest.raises(ValueError, match="2\\*\\*31"):
            pkv.kv_blocks_update(kc, i32(1, 2), i32(1), i32(1), i32(4), i32(1), num_rows=1, **kw)
