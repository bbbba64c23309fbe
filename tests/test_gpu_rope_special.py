"""Norm, rotation and append: elements behind the rotated part meet no other
element.  What is infinite, NaN or a negative zero there stays where it is."""
import numpy as np
import pytest
import torch

from paged_kv_cache_41_gb300 import pkv

import serving_util as su
from test_gpu_rope import Rope

pytestmark = pytest.mark.gpu
SPOILT = [float("inf"), float("-inf"), float("nan"), -0.0]


def bits(t):
    return t.contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32)


def spoil(r):
    """One value of SPOILT in a head row of each token in turn, behind the rotated part;
    [token, head, element] of each."""
    rng = np.random.default_rng(r.rot + r.d)
    heads = r.qkv.view(r.n, -1, r.d) if r.qkv.is_contiguous() else r.qkv.unflatten(1, (-1, r.d))
    at = []
    for i in range(r.n):
        h, e = int(rng.integers(0, r.hq + r.hkv)), int(rng.integers(r.rot, r.d))
        heads[i, h, e] = SPOILT[i % len(SPOILT)]
        at.append((i, h, e))
    return at


@pytest.mark.parametrize("d,rot", [(64, 0), (64, 32), (64, 48), (128, 0), (128, 64), (128, 112)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [40, 1800])     # one head row a group of lanes, four
def test_not_rotated_elements_stay_by_themselves(d, rot, interleaved, norm, dtype, n):
    r = Rope(n, dtype=dtype, hq=8, hkv=2, d=d, rot=rot, interleaved=interleaved, norm=norm, seed=rot)
    clean = torch.cat([r.call(), r.kc.view(-1, 2, d)[torch.from_numpy(r.slots).cuda()]], 1)
    at = spoil(r)
    out = r.call()
    assert pkv.get_device_error() == 0
    with np.errstate(invalid="ignore"):
        r.check(out)
    got = torch.cat([out, r.kc.view(-1, 2, d)[torch.from_numpy(r.slots).cuda()]], 1)
    if not norm:
        # every element but the spoilt ones as without them, bit for bit; those as they are
        given = r.qkv.unflatten(1, (-1, d))
        for i, h, e in at:
            x = given[i, h, e]
            assert (x.isnan() and got[i, h, e].isnan()) or torch.equal(bits(x.view(1)), bits(got[i, h, e].view(1)))
            got[i, h, e] = clean[i, h, e]
        assert torch.equal(bits(got), bits(clean))
        return
    # a norm is over the whole row, the other rows are as they were
    for i, h, _ in at:
        got[i, h] = clean[i, h]
    assert torch.equal(bits(got), bits(clean))


@pytest.mark.parametrize("d,rot", [(64, 0), (64, 32), (128, 0), (128, 96)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n", [40, 8000])     # one head row a group of lanes, four
def test_not_rotated_keys_of_quantised_pools(d, rot, interleaved, n):
    # groups behind the rotated part hold what the plain append makes of them
    r = Rope(n, dtype="mxfp8", hq=8, hkv=2, d=d, rot=rot, interleaved=interleaved, norm=False, seed=rot)
    spoil(r)
    r.call()
    want = pkv.MxPool(*r.shape, fill=0x55)
    k = r.k.contiguous()
    pkv.kv_append(want, want, k, k, torch.from_numpy(r.slots).cuda())
    assert pkv.get_device_error() == 0
    assert torch.equal(r.kc.elements[..., rot:], want.elements[..., rot:])
    assert torch.equal(r.kc.scales[..., rot // 32:], want.scales[..., rot // 32:])


def test_a_key_of_minus_infinity_weighs_nothing_behind_the_append():
    # the score of that row is -infinity, so the windowed decode passes it over
    n, d = 40, 64
    r = Rope(n, dtype="f32", hq=2, hkv=1, d=d, rot=32, norm=False, p=16)
    r.slots = np.arange(n, dtype=np.int64)
    r.qkv.view(n, 4, d)[:, :, 50] = 1.0
    r.qkv.view(n, 4, d)[7, 2, 50] = float("-inf")     # the key's head
    q = r.call()[-1:].contiguous()
    tables = torch.arange(3, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    lse = torch.empty(1, 2, device="cuda")
    out = pkv.paged_attention_decode_window(q, r.kc, r.vc, tables, lens, su.softmax_scale(d), window=n, lse=lse)
    assert pkv.get_device_error() == 0
    k, v = (x.view(-1, d)[:n].double().cpu().numpy() for x in (r.kc, r.vc))
    seen = np.ones((1, n), bool)
    seen[0, 7] = False
    for h in range(2):
        o, l, _, absv, mag = su.attend64(q[:, h].double().cpu().numpy(), k, v, seen, su.softmax_scale(d))
        su.check_attention("f32", d, out[:, h].cpu().numpy(), lse[:, h].cpu().numpy(), o, l, absv, mag, n, f"head {h}")
