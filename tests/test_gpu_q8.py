"""The 8-bit block-scaled cache on the GPU against its definition in 64 bits.

Writes and reads are exact: codes, scales and values equal the reference's bit
for bit.  Attention with fp32 outputs passes the gates of the other decodes
(rel-L2 <= 1e-4 per row, max abs <= 1e-3 max|v|; helpers.py).  A bf16 output may
be off by its own rounding, 2^-8 |o|, and by the 11 bits of the weights, which
move the mean of the values by at most 2^-11 max|v| (numerator) and as much
(denominator): 2^-8 |o| + 2^-10 max|v|."""
import math

import numpy as np
import pytest
import torch

import compressed_domain_attention_tq_b200 as tq
from compressed_domain_attention_tq_b200 import BlockKVCache, _lib
from conftest import require_cuda
from helpers import MAX_ABS_GATE, REL_L2_GATE
from q8_reference import Cache, TORCH, f64

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def randn(shape, seed, dtype=F32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def pair(B, H, cap, d, block, fmt):
    require_cuda()
    return Cache(B, H, cap, d, block, fmt), BlockKVCache(B, H, d, cap, block=block, dtype=TORCH[fmt])


def assert_same_cache(ref, c):
    for w, (codes, scales) in enumerate(((c.k_codes, c.k_scales), (c.v_codes, c.v_scales))):
        np.testing.assert_array_equal(f64(scales), ref.scales[w], err_msg=f"scales {'KV'[w]}")
        np.testing.assert_array_equal(f64(codes), ref.codes[w], err_msg=f"codes {'KV'[w]}")


def spoil(c, ctx):
    """Garbage behind the end of each sequence: any bits in the codes, NaN in scales of blocks no row of which is live."""
    for b in range(c.batch):
        for t in (c.k_codes, c.v_codes):
            u = t.view(torch.uint8)
            u[b, :, ctx[b]:] = 0x7F if t.dtype == torch.float8_e4m3fn else 0x80
        for s in (c.k_scales, c.v_scales):
            s[b, :, -(-ctx[b] // c.block):] = float("nan")


def check(got, want, ref, ctx, q_lens, label=""):
    """got: tensor [B][Hq][n][d]; want: float64."""
    dtype, got = got.dtype, f64(got)
    B, Hq, n, d = want.shape
    for b in range(B):
        m = n if q_lens is None else q_lens[b]
        for h in range(Hq):
            vmax = ref.absmax_v(b, h // (Hq // ref.H), int(ctx[b]))
            for i in range(m):
                g, w = got[b, h, i], want[b, h, i]
                where = f"{label} b={b} h={h} i={i}"
                if dtype == F32:
                    rel = np.linalg.norm(g - w) / max(np.linalg.norm(w), 1e-300)
                    assert rel <= REL_L2_GATE or np.array_equal(g, w), f"{where}: rel-L2 {rel:.3e}"
                    assert np.max(np.abs(g - w)) <= MAX_ABS_GATE * vmax, where
                else:
                    assert np.all(np.abs(g - w) <= 2.0 ** -8 * np.abs(w) + 2.0 ** -10 * vmax), where


# ------------------------------------------------------------------ write and read

@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,block,H,n,pos", [
    (128, 64, 2, 1, [0, 63, 64]), (128, 64, 1, 200, [0, 1, 100]), (64, 16, 3, 17, [15, 16, 5]),
    (96, 16, 2, 33, [0, 31, 7]), (96, 128, 1, 130, [127, 0, 64]), (256, 128, 1, 129, [0, 128, 200]),
    (256, 32, 2, 3, [30, 31, 32])])
def test_append_is_exact(fmt, dtype, d, block, H, n, pos):
    cap = max(pos) + n + 3
    ref, c = pair(3, H, cap, d, block, fmt)
    # earlier rows, then the new ones: larger (the kept codes move) for the second head on
    size = torch.tensor([1.0, 30.0, 0.01])[:H].view(1, H, 1, 1)
    first, then = randn((3, H, cap, d), 1, dtype), (randn((3, H, n, d), 2) * size).to(dtype)
    for a, b, at in ((first, -first, [0, 0, 0]), (then, 2 * then, pos)):
        ref.append(f64(a), f64(b), at)
        c.append(a.cuda(), b.cuda(), i32(at))
        assert_same_cache(ref, c)
    # read back: any range, as fp32 exactly and as bf16 rounded once
    k32, v32 = c.read(i32([0, 1, 2]), cap - 2, dtype=F32)
    kb, vb = c.read(None, cap)
    for w, (x32, xb) in enumerate(((k32, kb), (v32, vb))):
        for b in range(3):
            for h in range(H):
                np.testing.assert_array_equal(f64(x32[b, h]), ref.values(w, b, h, b, b + cap - 2))
                want = torch.from_numpy(ref.values(w, b, h, 0, cap)).float().to(BF16)
                assert torch.equal(xb[b, h].cpu(), want)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_append_token_by_token_with_growing_values(fmt):
    """Each token larger than the last: every append moves the block's earlier codes."""
    ref, c = pair(1, 2, 40, 64, 32, fmt)
    x = randn((1, 2, 40, 64), 3) * torch.linspace(0.1, 9, 40).view(1, 1, 40, 1) ** 2
    for t in range(40):
        ref.append(f64(x[:, :, t:t + 1]), f64(-x[:, :, t:t + 1]), [t])
        c.append(x[:, :, t:t + 1].contiguous().cuda(), -x[:, :, t:t + 1].contiguous().cuda(), i32([t]))
    assert_same_cache(ref, c)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_append_infinities_nan_zeros_and_tiny(fmt, dtype):
    ref, c = pair(1, 1, 64, 64, 16, fmt)
    x = randn((1, 1, 64, 64), 4)
    x[..., 0:16, :] = 0
    x[0, 0, 17, 3], x[0, 0, 18, 5], x[0, 0, 19, 7] = float("inf"), -float("inf"), float("nan")
    x[0, 0, 33] = 1e-38       # in a block of ordinary values: code 0
    x[..., 48:, :] *= 1e-36   # a whole block of tiny ones
    x[0, 0, 50, :4] = torch.tensor([1e-40, -1e-42, 0.0, -0.0])
    y = x.flip(3).clone()
    y[..., 0:16, :] = float("nan")  # no finite value: scale 0, codes 0
    x, y = x.to(dtype), y.to(dtype)
    ref.append(f64(x), f64(y), [0])
    c.append(x.cuda(), y.cuda(), i32([0]))
    assert_same_cache(ref, c)
    assert torch.isfinite(c.k_scales).all() and torch.isfinite(c.read(None, 64, dtype=F32)[1]).all()
    # scales at the ends of fp32's range
    for size in (1e37, 2e-38, 1e-44):
        z = (randn((1, 1, 64, 64), 5) * size).to(dtype)
        ref.append(f64(z), f64(z), [0])
        c.append(z.cuda(), z.cuda(), i32([0]))
        assert_same_cache(ref, c)


def test_append_skips_what_it_should():
    ref, c = pair(5, 2, 50, 64, 16, "int8")
    x = randn((5, 2, 20, 64), 6, BF16)
    c.append(x.cuda(), x.cuda(), i32([0, 5, 5, 5, 5]))
    ref.append(f64(x), f64(x), [0, 5, 5, 5, 5])
    y = randn((5, 2, 20, 64), 7, BF16, 5.0)
    # a negative row, rows behind the capacity, no token, too large a count, some tokens
    pos, valid = [-1, 40, 10, 17, 25], [20, 20, 0, 99, 7]
    c.append(y.cuda(), y.cuda(), i32(pos), n_valid=i32(valid))
    ref.append(f64(y), f64(y), pos, valid)
    assert_same_cache(ref, c)
    c.append(y.cuda(), y.cuda(), i32([50, 2 ** 31 - 1, -2 ** 31, 60, 50]), n_valid=i32([20, 20, 20, -3, -(2 ** 31)]))
    assert_same_cache(ref, c)
    marks = torch.full((5, 2, 12, 64), 7.0, device="cuda")
    ko, vo = c.read(i32([-2, 45, 3, 50, 2 ** 31 - 1]), 12, n_valid=i32([12, 12, 5, 12, 12]), out=(marks, marks.clone()))
    for b, (at, m) in enumerate([(0, 0), (45, 5), (3, 5), (0, 0), (0, 0)]):
        for h in range(2):
            np.testing.assert_array_equal(f64(vo[b, h, :m]), ref.values(1, b, h, at, at + m))
        assert torch.all(ko[b, :, m:] == 7.0)



@pytest.mark.parametrize("dtype", [BF16, F32])
def test_read_without_out_is_zero_outside(dtype):
    """Rows at n_valid and behind, outside the cache, and of sequences with a negative row."""
    ref, c = pair(4, 2, 150, 96, 32, "e4m3")
    x = randn((4, 2, 150, 96), 8, BF16)
    ref.append(f64(x), f64(-x), [0] * 4)
    c.append(x.cuda(), -x.cuda(), i32([0] * 4))
    torch.full((4, 2, 70, 96), 7.0, device="cuda", dtype=dtype)  # (memory that the outputs may get again)
    got = c.read(i32([-1, 100, 31, 2 ** 31 - 1]), 70, n_valid=i32([70, 70, 33, 70]), dtype=dtype)
    for w, y in enumerate(got):
        for b, (at, m) in enumerate([(0, 0), (100, 50), (31, 33), (0, 0)]):
            for h in range(2):
                want = torch.from_numpy(ref.values(w, b, h, at, at + m)).float().to(dtype)
                assert torch.equal(y[b, h, :m].cpu(), want) and torch.all(y[b, h, m:] == 0)


# ------------------------------------------------------------------------ attention

CASES = [  # d, block, H, G, n, ctx, q_lens
    (128, 64, 2, 8, 1, [1, 16, 17, 1000], None), (128, 64, 2, 1, 1, [0, 64, 65, 333], None),
    (128, 16, 1, 3, 1, [15, 31, 160, 2049], None), (128, 128, 1, 16, 1, [129, 5, 700], None),
    (64, 32, 3, 5, 1, [3, 100, 513], None), (96, 16, 2, 1, 1, [1, 47, 400], None),
    (96, 64, 1, 9, 1, [200, 2], None), (256, 64, 2, 2, 1, [77, 600], None), (256, 16, 1, 12, 1, [300], None),
    (128, 64, 2, 8, 5, [5, 300, 3, 77], [5, 1, 4, 0]), (128, 16, 1, 1, 7, [7, 8, 100], None),
    (128, 32, 1, 4, 70, [70, 200, 33, 0], [70, 33, 50, 9]), (64, 64, 1, 2, 40, [40, 300], None),
    (96, 32, 1, 3, 19, [19, 150], [19, 2]), (256, 32, 1, 2, 33, [33, 90], None),
]


def build(d, block, H, ctx, fmt, seed=0, capacity=None):
    cap = capacity or max(ctx) + 9
    ref, c = pair(len(ctx), H, cap, d, block, fmt)
    k, v = randn((len(ctx), H, cap, d), seed + 1), randn((len(ctx), H, cap, d), seed + 2)
    k[..., :2] *= 8  # channels that stand out
    v[:, :, ::5] *= 6
    k, v = k.to(BF16), v.to(BF16)
    ref.append(f64(k), f64(v), [0] * len(ctx))
    ref.upload(c)
    spoil(c, ctx)
    return ref, c


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,block,H,G,n,ctx,q_lens", CASES)
def test_attend_matches_definition(fmt, dtype, d, block, H, G, n, ctx, q_lens):
    ref, c = build(d, block, H, ctx, fmt)
    q = randn((len(ctx), H * G, n, d), 9, dtype)
    scale = 1 / math.sqrt(d)
    want, want_lse = ref.attend(f64(q), ctx, q_lens, scale)
    lse = torch.full((len(ctx), H * G, n, 2), 5.0, device="cuda")
    got = c.attend(q.cuda(), i32(ctx), max(max(ctx), 1), q_lens=None if q_lens is None else i32(q_lens), lse=lse)
    assert got.dtype == dtype
    check(got, want, ref, ctx, q_lens)
    lse = f64(lse)
    for b in range(len(ctx)):
        m = n if q_lens is None else q_lens[b]
        L = lse[b, :, :m]
        with np.errstate(divide="ignore"):
            have = L[..., 0] + np.log2(L[..., 1])
        np.testing.assert_allclose(have, want_lse[b, :, :m], atol=1e-3 if dtype == F32 else 4e-3)
        assert np.all(lse[b, :, m:] == 5.0) and torch.all(got[b, :, m:] == 0)  # rows of no query
    if n == 1:  # decode is the same call
        out = c.decode(q[:, :, 0].contiguous().cuda(), i32(ctx), max(max(ctx), 1))
        assert out.dtype == F32
        check(out[:, :, None], want, ref, ctx, None, "decode")


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_decode_over_many_chunks_and_lengths(fmt):
    """Split over the whole GPU, lengths on both sides of chunk ends, one empty sequence."""
    ctx = [0, 1, 63, 64, 65, 2047, 2048, 2049, 5000]
    ref, c = build(128, 64, 1, ctx, fmt)
    q = randn((len(ctx), 8, 128), 11)
    out = c.decode(q.cuda(), i32(ctx), 5000)
    want, _ = ref.attend(f64(q[:, :, None]), ctx, None, 1 / math.sqrt(128))
    check(out[:, :, None], want, ref, ctx, None)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("n", [1, 64])
def test_attend_with_scales_far_apart(fmt, n):
    """Blocks of V from 1e-30 to 1e10, all-zero blocks of K and V, tiny and huge queries."""
    ctx, d = [400], 128
    ref, c = pair(1, 1, 400, d, 16, fmt)
    k, v = randn((1, 1, 400, d), 12), randn((1, 1, 400, d), 13)
    k[:, :, 32:64] = 0
    v[:, :, 96:128] = 0
    for j, s in enumerate([1e-30, 1e3, 1e-10, 1e10, 1e-3]):
        v[:, :, 160 + 16 * j:176 + 16 * j] *= s
    ref.append(f64(k), f64(v), [0])
    ref.upload(c)
    for size in (1.0, 1e-30, 1e-44, 1e4):
        q = randn((1, 4, n, d), 14) * size
        scale = 1e-4 if size == 1e4 else 0.09
        want, _ = ref.attend(f64(q), ctx, None, scale)
        check(c.attend(q.cuda(), i32(ctx), 400, attn_scale=scale), want, ref, ctx, None, f"{size}")
        # bf16 output of the same queries
        qb = q.to(BF16)
        want, _ = ref.attend(f64(qb), ctx, None, scale)
        check(c.attend(qb.cuda(), i32(ctx), 400, attn_scale=scale), want, ref, ctx, None, f"bf16 {size}")


@pytest.mark.parametrize("d,G,n", [(128, 2, 160), (128, 4, 20), (256, 2, 60)])
def test_rows_before_a_huge_block_keep_their_precision(d, G, n):
    """A prompt whose last block of V is 1e7 or 1e20 times the others: the queries before it are exact
    to their own values (weights of 11 bits and the output's rounding, as in check)."""
    ctx = [n + 100]
    for size in (1e7, 1e20):
        ref, c = pair(1, 1, ctx[0], d, 16, "int8")
        k, v = randn((1, 1, ctx[0], d), 80), randn((1, 1, ctx[0], d), 81)
        last = (ctx[0] - 1) // 16 * 16
        v[:, :, last:] *= size
        ref.append(f64(k), f64(v), [0])
        ref.upload(c)
        q = randn((1, G, n, d), 82, BF16)
        want, _ = ref.attend(f64(q), ctx, None, d ** -0.5)
        got = f64(c.attend(q.cuda(), i32(ctx), ctx[0]))
        vmax = ref.absmax_v(0, 0, last)
        m = last - 100  # queries at positions below the block
        assert np.all(np.abs(got - want)[:, :, :m] <= 2.0 ** -8 * np.abs(want[:, :, :m]) + 2.0 ** -10 * vmax)


@pytest.mark.parametrize("n", [1, 40])
def test_a_sharp_softmax_picks_its_row(n):
    """Scores hundreds apart: the weights of all rows but one vanish, and the reference moves many times."""
    ref, c = pair(1, 1, 300, 64, 32, "int8")
    k = torch.ones(1, 1, 300, 64) * torch.linspace(0.1, 5, 300).view(1, 1, 300, 1)
    v = randn((1, 1, 300, 64), 15)
    ref.append(f64(k), f64(v), [0])
    ref.upload(c)
    for sign in (1.0, -1.0):
        q = torch.full((1, 2, n, 64), sign)
        want, _ = ref.attend(f64(q), [300], None, 2.0)
        check(c.attend(q.cuda(), i32([300]), 300, attn_scale=2.0), want, ref, [300], None)
        check(c.attend(q.to(BF16).cuda(), i32([300]), 300, attn_scale=2.0), want, ref, [300], None)


def test_nan_and_infinite_queries_stay_in_their_row():
    for n, dtype in ((1, F32), (64, F32), (64, BF16)):
        ref, c = build(128, 64, 1, [200], "int8")
        q = randn((1, 8, n, 128), 16, dtype)
        good = c.attend(q.cuda(), i32([200]), 200)
        q[0, 3, 0, 5], q[0, 4, 0, 7] = float("nan"), float("inf")
        got = c.attend(q.cuda(), i32([200]), 200)
        bad = torch.zeros(8, n, dtype=torch.bool)
        bad[3, 0] = bad[4, 0] = True
        assert torch.isnan(got[0].cpu()[bad]).all()
        assert torch.equal(got[0].cpu()[~bad], good[0].cpu()[~bad])


def test_lengths_out_of_range_are_clamped_and_flagged():
    ref, c = build(128, 64, 2, [50, 50, 50, 50], "int8")
    q = randn((4, 4, 3, 128), 17).cuda()
    ws = torch.empty(_lib.sdpa_q8_workspace_bytes(4, 4, 2, 128, 3, 50), dtype=torch.uint8, device="cuda")
    got = c.attend(q, i32([51, 50, -1, 50]), 50, q_lens=i32([3, 2, 3, 4]), workspace=ws)
    assert ws[:16].view(torch.int32).tolist() == [1, 0, 1, 1]
    want = c.attend(q, i32([50, 50, 0, 50]), 50, q_lens=i32([3, 2, 3, 3]), workspace=ws)
    assert ws[:16].view(torch.int32).tolist() == [0, 0, 0, 0]
    assert torch.equal(got, want) and torch.all(got[2] == 0)


def test_merge_of_context_parts_is_the_whole():
    ref, c = build(128, 64, 2, [300, 129], "int8")
    _, a = pair(2, 2, 192, 128, 64, "int8")
    _, b = pair(2, 2, 192, 128, 64, "int8")
    for part, lo in ((a, 0), (b, 128)):
        rows = min(192, c.capacity - lo)
        part.k_codes[:, :, :rows], part.v_codes[:, :, :rows] = c.k_codes[:, :, lo:lo + rows], c.v_codes[:, :, lo:lo + rows]
        for s, t in ((part.k_scales, c.k_scales), (part.v_scales, c.v_scales)):
            m = min(3, t.shape[2] - lo // 64)
            s[:, :, :m] = t[:, :, lo // 64:lo // 64 + m]
    q = randn((2, 8, 128), 18).cuda()
    outs, lses = torch.empty(2, 2, 8, 128, device="cuda"), torch.empty(2, 2, 8, 2, device="cuda")
    for i, (part, lens) in enumerate(((a, [128, 128]), (b, [172, 1]))):
        part.decode_lse(q, i32(lens), 192, 0.09, outs[i], lses[i])
    out = torch.empty(2, 8, 128, device="cuda")
    _lib.merge_lse(outs, lses, out)
    want, _ = ref.attend(f64(q[:, :, None]), [300, 129], None, 0.09)
    check(out[:, :, None], want, ref, [300, 129], None)


LONG = [  # d, block, H, G, n, ctx, q_lens: many token tiles, row tiles with a rest, prompts from position 0
    (128, 64, 1, 8, 37, [1100, 37, 300], [37, 37, 1]), (128, 16, 1, 1, 300, [300, 911], [300, 257]),
    (64, 32, 2, 3, 100, [1500, 100], None), (96, 128, 1, 4, 129, [129, 1025], [64, 129]),
    (256, 64, 1, 6, 45, [45, 700], [45, 33]), (128, 64, 1, 8, 5, [2000, 5, 129, 0], [5, 4, 1, 5]),
    (64, 16, 1, 16, 3, [1111, 128], None), (96, 16, 2, 8, 4, [777, 130], [3, 4]),
    (256, 128, 1, 16, 2, [1500, 64], None), (128, 128, 2, 1, 17, [640, 16], [17, 16]),
]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("d,block,H,G,n,ctx,q_lens", LONG)
def test_attend_bf16_over_many_tiles(fmt, d, block, H, G, n, ctx, q_lens):
    ref, c = build(d, block, H, ctx, fmt, seed=60)
    q = randn((len(ctx), H * G, n, d), 61, BF16, 1.5)
    want, want_lse = ref.attend(f64(q), ctx, q_lens, 1 / math.sqrt(d))
    marks = torch.full((len(ctx), H * G, n, d), 7.0, device="cuda", dtype=BF16)
    lse = torch.full((len(ctx), H * G, n, 2), 5.0, device="cuda")
    got = c.attend(q.cuda(), i32(ctx), max(ctx), q_lens=None if q_lens is None else i32(q_lens), out=marks, lse=lse)
    check(got, want, ref, ctx, q_lens)
    lse = f64(lse)
    for b in range(len(ctx)):
        m = n if q_lens is None else q_lens[b]
        with np.errstate(divide="ignore"):
            np.testing.assert_allclose(lse[b, :, :m, 0] + np.log2(lse[b, :, :m, 1]), want_lse[b, :, :m], atol=4e-3)
        assert np.all(lse[b, :, m:] == 5.0) and torch.all(got[b, :, m:] == 7.0)


def test_bf16_outputs_of_fp32_queries():
    """The workspace asked for by output type serves queries of either type."""
    ref, c = build(128, 64, 2, [500, 90], "int8")
    q = randn((2, 8, 30, 128), 62)
    want, _ = ref.attend(f64(q), [500, 90], None, 0.1)
    for dtype in (F32, BF16):
        x = q.to(dtype)
        if dtype == BF16:
            want, _ = ref.attend(f64(x), [500, 90], None, 0.1)
        out = torch.empty(2, 8, 30, 128, device="cuda", dtype=BF16)
        ws = torch.empty(_lib.sdpa_q8_workspace_bytes(2, 8, 2, 128, 30, 500, BF16), dtype=torch.uint8, device="cuda")
        check(c.attend(x.cuda(), i32([500, 90]), 500, attn_scale=0.1, out=out, workspace=ws), want, ref, [500, 90], None)


@pytest.mark.parametrize("B", [2, 5, 32, 40])
@pytest.mark.parametrize("n,G,dtype", [(1, 4, F32), (3, 8, BF16), (40, 8, BF16)])
def test_ragged_batches_of_any_size(B, n, G, dtype):
    """Batches split by their lengths (up to 32 sequences) and by the longest one (more)."""
    rng = np.random.RandomState(B)
    ctx = [int(x) for x in rng.randint(0, 1500, B)]
    ctx[B // 2], ctx[-1] = 1500, 0
    q_lens = None if n == 1 else [int(x) for x in rng.randint(0, n + 1, B)]
    ref, c = build(64, 32, 1, ctx, "int8", seed=70, capacity=1500)
    q = randn((B, G, n, 64), 71, dtype)
    want, _ = ref.attend(f64(q), ctx, q_lens, 0.125)
    got = c.attend(q.cuda(), i32(ctx), 1500, q_lens=None if q_lens is None else i32(q_lens))
    check(got, want, ref, ctx, q_lens)
    none = c.attend(q.cuda(), i32([0] * B), 1500)
    assert torch.all(none == 0)


@pytest.mark.parametrize("d,G", [(64, 24), (128, 64), (256, 17), (96, 32)])
def test_decode_of_many_heads_in_bf16(d, G):
    ctx = [700, 1, 257]
    ref, c = build(d, 64, 1, ctx, "e4m3", seed=72)
    q = randn((3, G, d), 73, BF16)
    out = torch.empty(3, G, d, device="cuda", dtype=BF16)
    want, _ = ref.attend(f64(q[:, :, None]), ctx, None, d ** -0.5)
    check(c.decode(q.cuda(), i32(ctx), 700, out=out)[:, :, None], want, ref, ctx, None)
    check(c.decode(q.cuda(), i32(ctx), 700)[:, :, None], want, ref, ctx, None)


def test_a_captured_call_follows_the_lengths():
    """Lengths are read on the device: a replay with others is the call with them."""
    ref, c = build(128, 64, 2, [1800, 1800, 1800], "int8")
    q1, qn = randn((3, 16, 128), 74, BF16).cuda(), randn((3, 16, 6, 128), 75, BF16).cuda()
    ctx, lens = i32([1800, 1800, 1800]), i32([6, 6, 6])
    one, many = torch.empty(3, 16, 128, device="cuda"), torch.empty_like(qn)
    call = lambda: (c.decode(q1, ctx, 1800, out=one), c.attend(qn, ctx, 1800, q_lens=lens, out=many))  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for new, m in (([5, 1800, 64], [5, 6, 1]), ([0, 3, 1799], [0, 3, 6]), ([700, 640, 1000], [6, 6, 6])):
        ctx.copy_(i32(new))
        lens.copy_(i32(m))
        many.fill_(7.0)
        g.replay()
        want_one, want_many = c.decode(q1, i32(new), 1800), c.attend(qn, i32(new), 1800, q_lens=i32(m))
        torch.cuda.synchronize()
        assert torch.equal(one, want_one)
        for b in range(3):
            assert torch.equal(many[b, :, :m[b]], want_many[b, :, :m[b]]) and torch.all(many[b, :, m[b]:] == 7.0)


def test_a_pipeline_that_starves_ends_with_nan():
    """The first tile never arrives: the bounded waits run out and the outputs are NaN."""
    for n, d in ((64, 128), (8, 128), (64, 256)):
        ref, c = build(d, 64, 1, [300], "int8")
        q = randn((1, 4, n, d), 63, BF16).cuda()
        good = c.attend(q, i32([300]), 300)
        tq.load().tq_set_test_hooks(2)
        try:
            assert torch.isnan(c.attend(q, i32([300]), 300)).all()
        finally:
            tq.load().tq_set_test_hooks(0)
        assert torch.equal(c.attend(q, i32([300]), 300), good)


# ------------------------------------------------------------------ used together

@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype,d,G", [(BF16, 128, 4), (F32, 64, 2)])
def test_a_conversation(fmt, dtype, d, G):
    """Prompt in ragged chunks, decode steps, drafted tokens of which some are rejected, and a read back."""
    B, H, cap = 2, 2, 260
    ref, c = pair(B, H, cap, d, 32, fmt)
    ctx, seed = [0, 0], 20
    scale = 1 / math.sqrt(d)
    for n, lens in ((100, [100, 37]), (64, [9, 64]), (1, [1, 1]), (1, [1, 1]), (5, [5, 3]), (1, [1, 1])):
        k, v, q = (randn((B, h, n, d), seed + j, dtype) for j, h in enumerate((H, H, H * G)))
        seed += 3
        ref.append(f64(k), f64(v), ctx, lens)
        ctx_new = [a + b for a, b in zip(ctx, lens)]
        if n == 1:
            out = c.decode_append(q[:, :, 0].contiguous().cuda(), k.cuda(), v.cuda(), i32(ctx_new), cap)[:, :, None]
        else:
            c.append(k.cuda(), v.cuda(), i32(ctx), n_valid=i32(lens))
            out = c.attend(q.cuda(), i32(ctx_new), cap, q_lens=i32(lens))
        assert_same_cache(ref, c)
        want, _ = ref.attend(f64(q), ctx_new, lens, scale)
        check(out, want, ref, ctx_new, lens, f"n={n}")
        ctx = ctx_new
        if n == 5:
            ctx = [ctx[0] - 3, ctx[1] - 1]  # rejected drafts: the next step overwrites them
    got = c.read(i32([3, 0]), 50, n_valid=i32([50, 20]), dtype=F32)[1]
    np.testing.assert_array_equal(f64(got[0, 1]), ref.values(1, 0, 1, 3, 53))


def test_decode_append_is_append_then_decode():
    for fmt in ("int8", "e4m3"):
        ctx = [1, 64, 65, 500, 0]
        ref, c = build(128, 64, 2, ctx, fmt)
        other = BlockKVCache(5, 2, 128, c.capacity, dtype=TORCH[fmt])
        for a, b in zip(other.buffers[:4], c.buffers[:4]):
            a.view(torch.uint8).copy_(b.view(torch.uint8))
        q, k, v = (randn((5, h, *x, 128), 30 + h, BF16).cuda() for h, x in ((16, ()), (2, (1,)), (2, (1,))))
        out = c.decode_append(q, k, v, i32(ctx), 500)
        other.append(k, v, i32([x - 1 for x in ctx]))
        want = other.decode(q, i32(ctx), 500)
        assert torch.equal(out, want) and torch.all(out[4] == 0)
        for a, b in zip(other.buffers[:4], c.buffers[:4]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_repeats_streams_and_graphs_give_the_same_bits():
    ref, c = build(128, 64, 2, [900, 333], "int8")
    q1, qn = randn((2, 16, 128), 40, BF16).cuda(), randn((2, 16, 130, 128), 41, BF16).cuda()
    ctx = i32([900, 333])
    first, chunk = c.decode(q1, ctx, 900), c.attend(qn, ctx, 900)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    on_side = c.decode(q1, ctx, 900, stream=side), c.attend(qn, ctx, 900, stream=side)
    at_once = c.decode(q1, ctx, 900), c.attend(qn, ctx, 900)
    side.synchronize()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):  # two graphs, replayed in turn on refilled inputs
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, c.decode(q1, ctx, 900), c.attend(qn, ctx, 900)))
    keep = q1.clone()
    q1.zero_()
    graphs[0][0].replay()
    mean = graphs[0][1].clone()
    q1.copy_(keep)
    for g, _, _ in graphs + graphs[:1]:
        g.replay()
    torch.cuda.synchronize()
    assert not torch.equal(mean, first)
    for a, b in (on_side, at_once, graphs[0][1:], graphs[1][1:]):
        assert torch.equal(a, first) and torch.equal(b, chunk)


def test_rows_past_four_gigabytes():
    """A cache whose second head begins, and whose last rows lie, past 2^32 bytes."""
    require_cuda()
    cap, d = (1 << 32) // 256 + 200, 256
    c = BlockKVCache(1, 2, d, cap, block=128)
    pos = cap - 101
    k, v = randn((1, 2, 100, d), 50, BF16), randn((1, 2, 100, d), 51, BF16)
    c.append(k.cuda(), v.cuda(), i32([pos]))
    ref = Cache(1, 2, 512, d, 128, "int8")  # the same places in their blocks
    at = pos % 128
    ref.append(f64(k), f64(v), [at])
    got = c.read(i32([pos]), 100, dtype=F32)
    for w in (0, 1):
        for h in (0, 1):
            np.testing.assert_array_equal(f64(got[w][0, h]), ref.values(w, 0, h, at, at + 100))
    # rows in front are zeros: weight 1 each against exp(s) of the last 100
    q = randn((1, 2, 1, d), 52)
    out = f64(c.attend((q * 2).cuda(), i32([pos + 100]), cap, attn_scale=0.5))
    for h in (0, 1):
        kk, vv = ref.values(0, 0, h, at, at + 100), ref.values(1, 0, h, at, at + 100)
        p = np.exp(kk @ f64(q)[0, h, 0])
        want = p @ vv / (p.sum() + pos)
        assert np.linalg.norm(out[0, h, 0] - want) <= REL_L2_GATE * np.linalg.norm(want)
    # two tokens of nine heads each in bf16: rows 0 .. pos + 98 and .. pos + 99
    q = randn((1, 18, 2, d), 53, BF16)
    out = f64(c.attend((q * 2).cuda(), i32([pos + 100]), cap, attn_scale=0.5))
    for h in range(18):
        kk, vv = ref.values(0, 0, h // 9, at, at + 100), ref.values(1, 0, h // 9, at, at + 100)
        for i in range(2):
            m = 99 + i
            p = np.exp(kk[:m] @ f64(q)[0, h, i])
            want = p @ vv[:m] / (p.sum() + pos)
            assert np.all(np.abs(out[0, h, i] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * np.abs(vv).max())


def test_python_calls_refuse():
    require_cuda()
    c = BlockKVCache(2, 2, 64, 40, block=16)
    x, q, n = torch.zeros(2, 2, 3, 64, device="cuda"), torch.zeros(2, 4, 64, device="cuda"), i32([1, 2])
    wide = torch.zeros(2, 2, 3, 128, device="cuda")
    for f in (lambda: c.append(wide[..., ::2], x, n), lambda: c.append(x, x[:, :, :2].contiguous(), n),
              lambda: c.append(x, x, n.long()), lambda: c.append(x, x, n[:1]), lambda: c.append(x[:1], x[:1], n[:1]),
              lambda: c.append(x.cpu(), x, n), lambda: c.append(x, x, n, n_valid=n.float()),
              lambda: c.read(n, 3, out=(x, wide)), lambda: c.read(n.float(), 3), lambda: c.decode(q[:1], n, 40),
              lambda: c.decode(q, n, 40, out=torch.zeros(2, 4, 32, device="cuda")), lambda: c.attend(q, n, 40),
              lambda: c.attend(x, n, 40, lse=torch.zeros(2, 2, 3, device="cuda")),
              lambda: c.decode_append(q, x, x, n, 40),
              lambda: tq.sdpa_q8(x, c.k_codes, c.k_scales, c.v_codes, c.v_scales, 32, n, 40)):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: c.append(x, x.to(BF16), n), lambda: c.append(x.half(), x.half(), n),
              lambda: c.decode(q.half(), n, 40), lambda: c.read(n, 3, dtype=torch.float16),
              lambda: tq.sdpa_q8(x, c.k_codes.view(torch.uint8), c.k_scales, c.v_codes, c.v_scales, 16, n, 40)):
        with pytest.raises(TypeError):
            f()
    for f in (lambda: c.decode(q, n, 41), lambda: c.decode(q, n, 40, attn_scale=0.0), lambda: c.read(n, 0),
              lambda: c.attend(x, n, 40, workspace=torch.empty(4, dtype=torch.uint8, device="cuda"))):
        with pytest.raises((tq.TQError, RuntimeError)):
            f()
