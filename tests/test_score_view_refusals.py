"""What the calls on a part of a wider score buffer refuse (no GPU), and the
bound that the binding hands them."""
import ctypes

import pytest
import torch

from paged_kv_cache_41_gb300 import pkv

from test_serving_refusals import A, BAD, BIG, UNSUP, P, desc, lib  # noqa: F401


@pytest.mark.parametrize("stride,rows,want", [
    (0, 0, BAD), (-1, 0, BAD), (10, -1, BAD), (10, 11, BAD), (10, 2**62, BAD)])
def test_rows_within_their_pitch(lib, stride, rows, want):  # noqa: F811
    c = ctypes.byref(desc())
    assert lib.pkv_paged_attention_decode_weights_view(c, A, A, A, stride, rows, 1.0, A, A, A, A, 4, A, 2, 4,
                                                       0.1, A, BIG, None) == want
    assert lib.pkv_kv_evict_select_view(A, stride, rows, A, 2, 2, 10, 1, 2, A, P(1 << 21), None) == want
    assert lib.pkv_kv_compact_view(c, A, P(1 << 24), A, stride, rows, A, 4, A, None, A, 2, 10, A, 2, None) == want


def test_row_numbers_are_bounded_by_the_rows_not_by_the_pitch(lib):  # noqa: F811
    far = P(1 << 21)
    assert lib.pkv_kv_evict_select_view(A, 2**40, 2**31 - 2**16 + 1, A, 2, 2, 10, 1, 2, A, far, None) == UNSUP
    # no sequences: everything else about the call is right
    assert lib.pkv_kv_evict_select_view(A, 2**40, 100, A, 0, 2, 10, 1, 2, A, far, None) == 0


def test_the_binding_bounds_a_view_by_its_own_rows():
    buf = torch.zeros(2, 3, 50)
    assert pkv._score_rows("w", buf, 2, 3) == (50, 50)
    assert pkv._score_rows("w", buf[:, :, 7:40], 2, 3) == (50, 33)
    assert pkv._score_rows("w", buf[:, :, :1], 2, 3) == (50, 1)
    assert pkv._score_rows("w", buf[:1, :, 40:], 1, 3) == (50, 10)
    assert pkv._score_rows("w", buf[:, :1, 4:], 2, 1) == (150, 46)
    assert pkv._score_rows("w", buf[:1, :1, 4:], 1, 1) == (46, 46)
