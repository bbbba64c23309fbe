"""The step's operators on either side of the sizes where another kernel takes over."""
import numpy as np
import pytest

from test_gpu_blocks import Step
from test_gpu_rope import Rope
from test_gpu_verify import Verify

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch", [1, 127, 128, 129])
@pytest.mark.parametrize("rows", [255, 256, 257, 2047, 2048, 2049])
def test_block_updates_of_so_many_rows(batch, rows):
    rng = np.random.default_rng(rows + batch)
    s = Step(rng.integers(0, 60, batch), 2100 // 16 + 60 // 16 + 2, spare=rows // 16 + batch + 1, seed=batch)
    add = np.bincount(rng.integers(0, batch, rows - 2), minlength=batch)
    old = s.lens_np.copy()
    s.update("lens", add, rows)                    # two rows of padding
    s.update(old, add // 2, 0)


@pytest.mark.parametrize("dtype,d,border", [("bf16", 128, 1100000), ("bf16", 64, 1100000), ("f32", 128, 1100000),
                                            ("f32", 64, 1100000), ("mxfp8", 128, 2200000), ("mxfp8", 64, 6000000)])
@pytest.mark.parametrize("rot", [0, 32, None])
def test_rotations_of_so_many_elements(dtype, d, border, rot):
    n = border // (d * 12)       # 8/2 heads: one head row a group of lanes up to here
    for tokens in (n, n + 1):
        Rope(tokens, dtype=dtype, hq=8, hkv=2, d=d, rot=rot, seed=tokens).run()


@pytest.mark.parametrize("vocab", [1023, 1024, 1025, 2047, 2048, 2049, 4096, 4097])
@pytest.mark.parametrize("sampled", [False, True])
def test_verifications_over_so_many_words(vocab, sampled):
    # one CTA a request, two, four, eight
    Verify([3, 1, 4], vocab, sampled=sampled, peak=1.0, seed=vocab).run()


@pytest.mark.parametrize("batch,vocab", [(70, 4100), (71, 4100), (140, 2100), (141, 2100), (280, 1100), (281, 1100)])
def test_verifications_of_so_many_requests(batch, vocab):
    Verify([1] * (batch - 2) + [3, 0], vocab, seed=batch).run()
