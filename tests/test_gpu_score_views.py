"""The calls that take scores, on views of wider buffers: nothing outside the
view is read or written, whatever the lengths on the device say."""
import numpy as np
import pytest
import torch

from paged_kv_cache_41_gb300 import pkv

from test_gpu_evict import Compact, Weigh, run_select, select_plain

pytestmark = pytest.mark.gpu

# (columns before the view, behind it): the last row of the last one ends where the buffer does
SIDES = [(0, 9), (5, 0), (4, 3), (1, 30)]


def view_of(x, before, behind, fill):
    buf = torch.full((*x.shape[:2], before + x.shape[2] + behind), fill, device="cuda")
    v = buf[:, :, before:before + x.shape[2]]
    v.copy_(x)
    return buf, v


def outside(buf, v, before):
    return torch.cat([buf[:, :, :before].flatten(), buf[:, :, before + v.shape[2]:].flatten()])


@pytest.mark.parametrize("before,behind", SIDES)
@pytest.mark.parametrize("g", [2, 8])
def test_weigh_stays_inside_its_view(g, before, behind):
    wg = Weigh([60, 100, 33], hq=2 * g, hkv=2, d=128, seed=6)
    w0 = wg.w.clone()
    wg.call()
    done = wg.w
    buf, wg.w = view_of(w0, before, behind, 3.0)
    wg.call()
    assert pkv.get_device_error() == 0
    assert torch.equal(wg.w, done) and (outside(buf, wg.w, before) == 3.0).all()
    # a sequence longer than the view, and shorter than the buffer's rows
    short = w0[:, :, :97]
    buf, wg.w = view_of(short, before, behind, 3.0)
    wg.call()
    assert pkv.get_device_error() == pkv.DEVERR_LENGTH
    assert torch.equal(wg.w, done[:, :, :97]) and (outside(buf, wg.w, before) == 3.0).all()


@pytest.mark.parametrize("before,behind", SIDES)
@pytest.mark.parametrize("n", [60, 9000, 400000])
def test_select_stays_inside_its_view(n, before, behind):
    w = torch.rand(3, 2, n, device="cuda")
    _, v = view_of(w, before, behind, 7.0)  # heavier than every weight of the view
    budget = n // 3
    run_select(v, [n, n // 2, 3], budget, 2, 5)
    if behind:  # a length past the view's rows is cut to them
        keep, new = pkv.kv_evict_select(v, torch.tensor([n + behind, n, 1], dtype=torch.int32, device="cuda"), budget,
                                        num_sinks=2, num_recent=5)
        assert pkv.get_device_error() == pkv.DEVERR_LENGTH
        want, want_new = select_plain(w.cpu().numpy(), np.array([n, n, 1]), budget, 2, 5)
        assert np.array_equal(keep.cpu().numpy(), want) and np.array_equal(new.cpu().numpy(), want_new)


@pytest.mark.parametrize("rows", [100, 8192, 30000])
def test_select_of_short_rows_in_a_wide_buffer(rows):
    buf = torch.rand(4, 2, 450000, device="cuda")
    run_select(buf[:, :, :rows], [rows, rows - 1, rows // 2, 0], rows // 4 + 1, 1, 3)


@pytest.mark.parametrize("before,behind", SIDES)
def test_compact_stays_inside_its_view(before, behind):
    c = Compact([200, 60, 90], [50, 20, 30], seed=7)
    c.w = c.w[:, :, :200].contiguous()
    w0 = c.w.clone()
    c.call()
    done = c.w
    assert pkv.get_device_error() == 0
    c = Compact([200, 60, 90], [50, 20, 30], seed=7)
    buf, c.w = view_of(w0, before, behind, 3.0)
    c.call()
    assert pkv.get_device_error() == 0
    assert torch.equal(c.w, done) and (outside(buf, c.w, before) == 3.0).all()
    # rows of 199 scores: sequence 0 does not fit them and is skipped
    c = Compact([200, 60, 90], [50, 20, 30], seed=7)
    buf, c.w = view_of(w0[:, :, :199], before, behind, 3.0)
    c.call()
    assert pkv.get_device_error() == pkv.DEVERR_LENGTH
    assert torch.equal(c.w[0], w0[0, :, :199]) and torch.equal(c.w[1:], done[1:, :, :199])
    assert (outside(buf, c.w, before) == 3.0).all()


def test_rows_of_no_scores():
    # torch gives an empty view no address, and the call refuses that; with an
    # address a row may hold nothing
    buf = torch.full((2, 2, 40), 3.0, device="cuda")
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(pkv.PkvError, match="invalid argument"):
        pkv.kv_evict_select(buf[:, :, 8:8], lens, 5)
    keep, new = torch.zeros(2, 2, 5, dtype=torch.int32, device="cuda"), lens + 9
    for n, err in ((0, 0), (1, pkv.DEVERR_LENGTH)):
        lens.fill_(n)
        assert pkv.load_library().pkv_kv_evict_select_view(
            buf.data_ptr(), 40, 0, lens.data_ptr(), 2, 2, 5, 1, 1, keep.data_ptr(), new.data_ptr(),
            torch.cuda.current_stream().cuda_stream) == 0
        assert pkv.get_device_error() == err
        assert (keep == -1).all() and (new == 0).all()
    assert (buf == 3.0).all()
