"""The binding refuses sizes that 32 bits would cut, on either side (no GPU)."""
import pytest
import torch

from paged_kv_cache_41_gb300 import pkv


def i32(*s):
    return torch.zeros(s, dtype=torch.int32)


@pytest.mark.parametrize("size", [-2**31 - 1, -2**32, -2**32 + 5, -2**40 + 5, 2**31, 2**32, 2**32 + 5])
@pytest.mark.parametrize("name", ["window", "num_sinks"])
def test_windows_past_32_bits(size, name):
    kc, q = torch.zeros(4, 16, 2, 64), torch.zeros(1, 4, 64)
    kw = {"window": 5, "num_sinks": 3, name: size}
    with pytest.raises(ValueError, match="2\\*\\*31"):
        pkv.paged_attention_decode_window(q, kc, kc, i32(1, 2), i32(1), 1.0, **kw)
    with pytest.raises(ValueError, match="2\\*\\*31"):
        pkv.decode_window_workspace_bytes(kc, 1, 4, 2, **kw)
    with pytest.raises(ValueError, match="2\\*\\*31"):
        pkv.kv_blocks_update(kc, i32(1, 2), i32(1), i32(1), i32(4), i32(1), num_rows=1, **kw)


@pytest.mark.parametrize("size", [2**31, 2**32 + 3])
def test_verified_drafts_past_32_bits(size):
    # of empty shapes, so that nothing large is made
    e, ptr = torch.empty(0), i32(1)
    with pytest.raises(ValueError, match="max_draft .*2\\*\\*31"):
        pkv.draft_verify(torch.empty(0, 5), i32(0), ptr, e, max_draft=size)
    with pytest.raises(ValueError, match="vocab .*2\\*\\*31"):
        pkv.draft_verify(torch.empty(0, size), i32(0), ptr, e, max_draft=3)
    with pytest.raises(ValueError, match="rows .*2\\*\\*31"):
        pkv.draft_verify(torch.empty(1, 1).expand(size, 1), i32(0), ptr, e, max_draft=3)


@pytest.mark.parametrize("size", [2**31, 2**32 + 3])
def test_tables_past_32_bits(size):
    kc, none = torch.zeros(4, 16, 2, 64), i32(0)
    with pytest.raises(ValueError, match="max_blocks .*2\\*\\*31"):
        pkv.kv_blocks_update(kc, i32(0, size), none, none, i32(4), i32(1), num_rows=1)
    with pytest.raises(ValueError, match="max_blocks .*2\\*\\*31"):
        pkv.paged_attention_decode_window(torch.zeros(0, 4, 64), kc, kc, i32(0, size), none, 1.0, window=5)
    with pytest.raises(ValueError, match="max_blocks_per_seq .*2\\*\\*31"):
        pkv.decode_window_workspace_bytes(kc, 1, 4, size, 5)
    q = torch.zeros(1, 4, 64)
    with pytest.raises(ValueError, match="positions .*2\\*\\*31"):
        pkv.qk_norm_rope_append(q, q[:, :2], q[:, :2], kc, kc, torch.zeros(1, dtype=torch.int64), i32(1),
                                torch.zeros(1, 16).expand(size, 16))
