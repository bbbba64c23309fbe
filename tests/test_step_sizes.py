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
