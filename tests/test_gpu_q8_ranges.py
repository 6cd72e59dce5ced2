"""The 8-bit block-scaled cache on the GPU where values, places and timing are far from ordinary:
scores and scales far apart, places near the ends of int32, warps that come late.  The reference
and the gates of test_gpu_q8.py, tighter where a test says so."""
import pytest
import torch

from compressed_domain_attention_tq_b200 import BlockKVCache, _lib
from conftest import require_cuda
from test_gpu_q8 import BF16, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,G,n", [(128, 4, 64), (128, 8, 8), (256, 4, 40), (64, 4, 64), (96, 2, 100), (64, 8, 4)])
def test_late_scales_change_nothing(d, G, n):
    """The warp that brings the blocks' scales is held up for longer than the products of several
    tiles take; the others have to wait for it, whatever the mode.  160 heads, so that a work
    item goes through five tiles and more."""
    require_cuda()
    B, H, T = 5, 32, 1100
    c, ctx = BlockKVCache(B, H, d, T, block=16), i32([1100, 1099, 900, 1024, 1100])
    g = torch.Generator("cuda").manual_seed(90)
    k, v = (torch.randn(B, H, T, d, generator=g, device="cuda", dtype=BF16) for _ in range(2))
    c.append(k, v, i32([0] * B))
    q = torch.randn(B, H * G, n, d, generator=g, device="cuda", dtype=BF16)
    good = c.attend(q, ctx, T)
    _lib.set_test_hooks(_lib.TEST_HOOK_SLOW_SCALES)
    try:
        late = c.attend(q, ctx, T)
    finally:
        _lib.set_test_hooks(0)
    assert torch.isfinite(good).all() and torch.equal(late, good)
