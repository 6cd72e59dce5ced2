"""The 8-bit block-scaled cache on the GPU where values, places and timing are far from ordinary:
scores and scales far apart, places near the ends of int32, warps that come late.  The reference
and the gates of test_gpu_q8.py, tighter where a test says so."""
import math

import pytest
import torch

from compressed_domain_attention_tq_b200 import BlockKVCache, TQError, _lib, context_parallel
from conftest import require_cuda
from test_gpu_q8 import BF16, F32, i32

pytestmark = pytest.mark.gpu


def definition(c, q, ctx, scale):
    """Attention of q [B][Hq][n][d] over the cache's values in 64 bits, every sequence of length ctx
    -> (outputs, the weights' sum of |v|, the largest score and the logarithm of the sum of weights in
    powers of two)."""
    k, v = (x.double() for x in c.read(None, ctx, dtype=F32))
    B, Hq, n, d = q.shape
    H = c.num_kv_heads
    s = (q.double().view(B, H, -1, d) @ k.transpose(-1, -2)).view(B, H, -1, n, ctx) * scale
    last = torch.arange(n, device="cuda") + ctx - n
    s.masked_fill_(torch.arange(ctx, device="cuda") > last[:, None], -torch.inf)
    p = torch.softmax(s, -1).view(B, H, -1, ctx)
    top, lse = s.amax(-1) / math.log(2), torch.logsumexp(s, -1) / math.log(2)
    return ((p @ v).view(B, Hq, n, d), (p @ v.abs()).view(B, Hq, n, d), top.view(B, Hq, n), lse.view(B, Hq, n))


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
    off = ~((got.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -10) * want.abs() + 2.0 ** -88)
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


@pytest.mark.parametrize("n", [1, 12])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_fp32_rows_behind_a_huge_block_keep_their_precision(d, n):
    """The first block's V is 1e5 to 1e20 times the others' and its keys score 69 nats below
    them, so that it adds nothing (e^-69 2^66 = 1e-10).  384 heads: a work item holds a whole context.
    fp32 queries: a score's error is 2^-20 of scale sum |q k| (22 bits of a query element, d / 16 sums in
    the tensor cores), a weight's that and 2^-20 for its exponent and its two parts; the outputs'
    twice a weight's of the weighted |v|."""
    require_cuda()
    B, H, T = 12, 32, 400
    g = torch.Generator("cuda").manual_seed(93)
    c = BlockKVCache(B, H, d, T, block=64)
    k, v = (torch.randn(B, H, T, d, generator=g, device="cuda") for _ in range(2))
    k[..., 0] = 0
    k[:, :, :64] = 0
    k[:, :, :64, 0] = -1
    v[:, :, :64] *= torch.tensor([1e5, 1e7, 1e10, 1e20], device="cuda").repeat(3)[:, None, None, None]
    c.append(k, v, i32([0] * B))
    q = torch.randn(B, 2 * H, n, d, generator=g, device="cuda")
    scale = d ** -0.5
    q[..., 0] = 69 / scale
    c.v_codes[1, :, :64] = 0  # (one sequence whose first block only has a large scale)
    want, size, *_ = definition(c, q, T, scale)
    got = (c.attend(q, i32([T] * B), T) if n > 1 else c.decode(q[:, :, 0].contiguous(), i32([T] * B), T)[:, :, None])
    kk = c.read(None, T, dtype=F32)[0][:, :, 64:].abs().double().repeat_interleave(2, 1)
    spread = scale * (q.abs().double() @ kk.transpose(-1, -2)).amax(-1, keepdim=True)
    off = ~((got.double() - want).abs() <= 2 * 2.0 ** -20 * (spread + 1) * size)
    assert not off.any(), off.sum((1, 2, 3)).tolist()


def filled(B, H, T, d, seed, size=1.0, block=64, positive=False):
    """A cache of normal draws, V (or |V|) times size (a number, or a tensor that broadcasts)."""
    require_cuda()
    g = torch.Generator("cuda").manual_seed(seed)
    c = BlockKVCache(B, H, d, T, block=block)
    k, v = (torch.randn(B, H, T, d, generator=g, device="cuda") for _ in range(2))
    c.append(k, (v.abs() if positive else v) * size, i32([0] * B))
    return c, g


@pytest.mark.parametrize("dtype,n", [(F32, 1), (F32, 9), (BF16, 20), (BF16, 160)])
@pytest.mark.parametrize("B,H", [(1, 2), (5, 32)])
def test_softmax_states_are_near_the_maximum(B, H, dtype, n):
    """lse = (M, L): M lies between one below the largest score and the logarithm of the sum, also where
    the row sees only blocks whose V is small beside another's; few heads (joined parts) and many
    (whole contexts).  M + log2(L) is the logarithm: scores of 11-bit queries, fp32 sums (4e-3 in bf16,
    whose weights have 11 bits of their own, as elsewhere)."""
    T, d = 1100, 128
    size = torch.ones(T, 1, device="cuda")
    size[:512] = 1e-20
    size[512:1024] = 1e-36
    c, g = filled(B, H, T, d, 94, size, block=16)
    q = torch.randn(B, 2 * H, n, d, generator=g, device="cuda").to(dtype)
    lse = torch.empty(B, 2 * H, n, 2, device="cuda")
    for ctx in (T, 1024, 512):
        _, _, top, want = definition(c, q, ctx, d ** -0.5)
        c.attend(q, i32([ctx] * B), T, lse=lse)
        M, L = lse.double().unbind(-1)
        assert ((M + torch.log2(L)) - want).abs().max() < (4e-3 if dtype == BF16 else 1e-4)
        assert (M > top - 1.01).all() and (M < want + 0.01).all(), (ctx, (M - top).min(), (M - want).max())


@pytest.mark.parametrize("size", [3e33, 1e-36])
@pytest.mark.parametrize("dtype,n", [(F32, 1), (F32, 9), (BF16, 20), (BF16, 160)])
@pytest.mark.parametrize("B,H,T,d", [(1, 2, 3000, 128), (5, 32, 4096, 64), (5, 32, 500, 256)])
def test_values_near_the_ends_of_the_range(B, H, T, d, dtype, n, size):
    """Sums of weights times V stay in fp32's range and keep its bits, positive as they are here.
    Tolerances of the fp32 rows behind a huge block (scores of normal draws: scale sum |q k| < 32) and
    of bf16 outputs, and half of bf16's last place below its normal numbers, 2^-134."""
    c, g = filled(B, H, T, d, 95, size, positive=True)
    q = (0.5 * torch.randn(B, H, n, d, generator=g, device="cuda")).to(dtype)
    got = c.attend(q, i32([T] * B), T).double()
    want, weighted, *_ = definition(c, q, T, d ** -0.5)
    tol = 2 * 2.0 ** -20 * 33 * weighted if dtype == F32 else 2.0 ** -8 * want.abs() + 2.0 ** -10 * weighted
    off = ~((got - want).abs() <= tol + 2.0 ** -134)
    assert torch.isfinite(got).all() and not off.any(), (off.sum().item(), off.numel())


@pytest.mark.parametrize("n", [20, 160])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_states_of_queries_that_attend_nothing(d, n):
    """Positions below 0, in tiles whose other tokens have blocks of zero V: (-inf, 0) and zeros, as of
    every row that attends nothing; 160 heads, so that contexts are not split."""
    B, H = 5, 32
    size = torch.ones(64, 1, device="cuda")
    size[16:] = 0
    c, g = filled(B, H, 64, d, 96, size, block=16)
    q = torch.randn(B, H, n, d, generator=g, device="cuda", dtype=BF16)
    for ctx in (5, 0, 19):
        lse = torch.full((B, H, n, 2), 5.0, device="cuda")
        got = c.attend(q, i32([ctx] * B), 64, lse=lse)
        none = max(0, n - ctx)
        assert torch.all(got[:, :, :none] == 0)
        assert torch.all(lse[:, :, :none, 0] == -torch.inf) and torch.all(lse[:, :, :none, 1] == 0)
        assert torch.all(lse[:, :, none:, 1] >= 1)


@pytest.mark.parametrize("size", [4e36, 3e-38])
@pytest.mark.parametrize("d,dtype,n", [(128, F32, 1), (64, F32, 9), (128, BF16, 1), (96, BF16, 20), (128, BF16, 160),
                                       (256, BF16, 40)])
def test_queries_near_the_ends_of_the_range(d, dtype, n, size):
    """Queries times size under an attention scale divided by it: ordinary scores, whose errors are those of
    the fp32 rows behind a huge block (queries below fp32's normal numbers are given as they are
    rounded), and of bf16 outputs (at least: decode gives fp32)."""
    c, g = filled(2, 4, 500, d, 97)
    q = (torch.randn(2, 8, n, d, generator=g, device="cuda") * size).to(dtype)
    scale = d ** -0.5 / size
    want, weighted, *_ = definition(c, q, 500, scale)
    got = (c.attend(q, i32([500] * 2), 500, attn_scale=scale) if n > 1 else
           c.decode(q[:, :, 0].contiguous(), i32([500] * 2), 500, attn_scale=scale)[:, :, None]).double()
    tol = 2 * 2.0 ** -20 * 33 * weighted
    if n > 1 and dtype == BF16:
        tol = tol + 2.0 ** -8 * want.abs() + 2.0 ** -10 * weighted
    off = ~((got - want).abs() <= tol)
    assert not off.any(), (off.sum().item(), off.numel())


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("fmt", [torch.int8, torch.float8_e4m3fn])
def test_append_keeps_the_sign_of_zeros(d, fmt):
    """Codes are those of fl32(x / s) bit for bit: an e4m3 code of -0 is 0x80, in a block that has an
    infinity as in one that has not (int8 has one zero)."""
    require_cuda()
    for dtype in (F32, BF16):
        c = BlockKVCache(1, 2, d, 64, block=16, dtype=fmt)
        x = torch.randn(1, 2, 64, d, device="cuda").to(dtype)
        x[..., ::3] = -0.0
        x[..., 1::3] = 0.0
        x[:, :, 20, 2], x[:, :, 21, 5] = torch.inf, -torch.inf
        x[:, :, 40, 2] = -1e-44  # underflows against the block's scale
        c.append(x, x, i32([0]))
        zero = x == 0
        want = torch.where(torch.signbit(x) & (fmt != torch.int8), 0x80, 0).to(torch.uint8)
        codes = c.k_codes.view(torch.uint8)
        assert torch.equal(codes[zero], want[zero]) and torch.equal(codes, c.v_codes.view(torch.uint8))
        assert (codes[:, :, 40, 2] == (0 if fmt == torch.int8 else 0x80)).all()


def test_lengths_beyond_the_cache_are_refused():
    """max_ctx is compared with the capacity as it is given, not by its low 32 bits."""
    c, _ = filled(1, 2, 40, 64, 98)
    x, one = torch.zeros(1, 2, 1, 64, device="cuda"), i32([1])
    for size in (41, 0, -1, (1 << 32) + 40, 1 << 31, 1 << 40):
        for f in (lambda: c.decode(x[:, :, 0], one, size), lambda: c.attend(x, one, size),
                  lambda: c.decode_append(x[:, :, 0], x, x, one, size)):
            with pytest.raises(TQError) as e:
                f()
            assert e.value.status == _lib.TQ_ERR_INVALID_ARG


def test_context_parallel_decode_takes_a_block_cache():
    """One rank's shard is the whole context: the call is decode and the merge of one part."""
    c, g = filled(2, 2, 700, 128, 99)
    q = torch.randn(2, 16, 128, generator=g, device="cuda", dtype=BF16)
    got = context_parallel.decode(c, q, i32([700, 300]), 700)
    torch.testing.assert_close(got, c.decode(q, i32([700, 300]), 700), rtol=2.0 ** -21, atol=0)


def test_long_sums_of_positive_values_keep_their_last_bits():
    """fp32 decode of positive values over 64K tokens, d = 256: each warp adds 256 and more steps.  Rounding
    to nearest, an addition is off by at most 2^-24 of a sum that grows evenly: 256 such errors come to
    256^(1/2) 2^-24 / 3^(1/2) < 2^-20.8 in the mean square, and six times that below 2^-18.  Cut off
    instead they add up to 256 2^-24 / 2 = 2^-17 on average."""
    require_cuda()
    B, H, T, d = 4, 16, 65536, 256
    c = BlockKVCache(B, H, d, T, block=128)
    g = torch.Generator("cuda").manual_seed(100)
    for at in range(0, T, 8192):
        k, v = (torch.randn(B, H, 8192, d, generator=g, device="cuda", dtype=BF16) for _ in range(2))
        c.append(k, v.abs(), i32([at] * B))
    q = torch.randn(B, 2 * H, d, generator=g, device="cuda")
    got = c.decode(q, i32([T] * B), T).double()
    for b in range(B):
        for h in range(H):
            k, v = ((x[b, h].double() * s[b, h].double().repeat_interleave(128)[:, None])
                    for x, s in ((c.k_codes, c.k_scales), (c.v_codes, c.v_scales)))
            want = torch.softmax(q[b, 2 * h:2 * h + 2].double() @ k.T / 16, -1) @ v
            assert ((got[b, 2 * h:2 * h + 2] / want - 1).abs().max() < 2.0 ** -18)


@pytest.mark.parametrize("place", [0, 5, 24])
@pytest.mark.parametrize("n", [1, 12])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_fp32_tokens_of_small_weight_and_huge_value_keep_their_precision(d, n, place):
    """One block of 16 tokens whose keys score 14 nats below the others' (weights of 1e-6) and whose V is
    1e5 to 1e20 times theirs, so that it is most of the output or all: at the beginning, between others,
    at the end.  Blocks of zeros, which score as the others do, around it in every second head.
    Tolerances of the fp32 rows behind a huge block."""
    require_cuda()
    B, H, T = 12, 32, 400
    g = torch.Generator("cuda").manual_seed(101)
    c = BlockKVCache(B, H, d, T, block=16)
    k, v = (torch.randn(B, H, T, d, generator=g, device="cuda") for _ in range(2))
    k[..., 0] = 0
    k[:, :, 16 * place:16 * place + 16, 0] = -1
    size = torch.tensor([1e5, 1e7, 1e10, 1e20], device="cuda").repeat(3)[:, None, None, None]
    v[:, :, 16 * place:16 * place + 16] *= size
    v[:, ::2, 32:64] = v[:, ::2, 320:352] = 0
    if place:
        v[:, ::2, :16] = 0
    c.append(k, v, i32([0] * B))
    q = torch.randn(B, 2 * H, n, d, generator=g, device="cuda")
    scale = d ** -0.5
    q[..., 0] = 14 / scale
    want, weighted, *_ = definition(c, q, T, scale)
    got = (c.attend(q, i32([T] * B), T) if n > 1 else c.decode(q[:, :, 0].contiguous(), i32([T] * B), T)[:, :, None])
    kk = c.read(None, T, dtype=F32)[0].abs().double().repeat_interleave(2, 1)
    spread = scale * (q.abs().double() @ kk.transpose(-1, -2)).amax(-1, keepdim=True)
    off = ~((got.double() - want).abs() <= 2 * 2.0 ** -20 * (spread + 1) * weighted)
    assert not off.any(), off.sum((1, 2, 3)).tolist()
