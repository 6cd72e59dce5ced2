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


GAPS = [100.0, 120.0, 127.6, 128.2, 129.0, 130.0, 200.0, 256.0, 270.0, 400.0]


@pytest.mark.parametrize("fmt", [torch.int8, torch.float8_e4m3fn])
@pytest.mark.parametrize("n", [20, 160])
@pytest.mark.parametrize("d", [64, 96, 128, 256])
def test_one_token_far_above_all_others(d, n, fmt):
    """Flat scores but for one token, 2^GAPS[b] above them in sequence b and at place h of 16
    tokens for kv head h, behind the first 64: its value is the output.  Its weight has 11 bits
    and so has the row's sum against it (2^-11 each at most), the output is rounded once.  The
    other 299 tokens weigh 2^-100 at most each, with values below 8: 299 * 8 * 2^-100 < 2^-88."""
    require_cuda()
    B, H, T = len(GAPS), 16, 300
    c = BlockKVCache(B, H, d, T, block=16, dtype=fmt)
    k = torch.zeros(B, H, T, d, device="cuda")
    at = 80 + torch.arange(H)
    k[:, torch.arange(H), at, 0] = 1.0
    v = torch.randn(B, H, T, d, generator=torch.Generator("cuda").manual_seed(92), device="cuda")
    c.append(k, v, i32([0] * B))
    values = c.read(None, T, dtype=torch.float32)[1]
    want = values[:, torch.arange(H), at][:, :, None].double()
    q = torch.zeros(B, H, n, d, device="cuda", dtype=BF16)
    q[..., 0] = torch.tensor(GAPS, device="cuda")[:, None, None].to(BF16)
    got = c.attend(q, i32([T] * B), T, attn_scale=0.6931471805599453)
    off = (got.double() - want).abs() > (2.0 ** -8 + 2.0 ** -10) * want.abs() + 2.0 ** -88
    assert values.abs().max() < 8
    assert not off.any(), sorted({(GAPS[b], int(h)) for b, h in off.nonzero()[:, :2].tolist()})


@pytest.mark.parametrize("block", [16, 128])
def test_appends_behind_the_capacity_wherever_they_begin(block):
    """Places up to the last int32, with more tokens than the cache has rows: nothing is written."""
    require_cuda()
    c = BlockKVCache(4, 2, 64, 50, block=block)
    x = torch.randn(4, 2, 300, 64, device="cuda")
    c.append(x[:, :, :50].contiguous(), x[:, :, :50].contiguous(), i32([0] * 4))
    before = [t.clone() for t in c.buffers[:4]]
    for n in (1, 20, 100, 300):
        y = (3 * x[:, :, :n]).contiguous()
        c.append(y, y, i32([50, 2 ** 31 - n // 2 - 1, 2 ** 31 - n, 2 ** 31 - 1]))
        c.append(y, y, i32([2 ** 31 - 1] * 4), n_valid=i32([n, 1, 2 ** 31 - 1, n // 2]))
    for a, b in zip(before, c.buffers[:4]):
        assert torch.equal(a, b)
