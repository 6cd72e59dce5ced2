"""The 8-bit block-scaled cache without a GPU: calls that have to be refused
are, before any launch, and the reference the GPU tests use is itself right."""
import ctypes

import numpy as np
import pytest
import torch

from compressed_domain_attention_tq_b200 import BlockKVCache, _lib
from q8_reference import Cache, QMAX, TORCH, nearest
from test_boundary_host import FakeBuffers, lib  # noqa: F401

INVALID, UNSUPPORTED, WORKSPACE = _lib.TQ_ERR_INVALID_ARG, _lib.TQ_ERR_UNSUPPORTED, _lib.TQ_ERR_WORKSPACE


def call(lib, what, **kw):
    fb = FakeBuffers()
    a = dict(q=fb.p(0), k=fb.p(256), v=fb.p(512), dtype=1, kv_dtype=1, B=1, Hq=8, Hkv=2, n=1, d=128, fmt=0,
             block=64, pos=fb.p(768), valid=None, kc=fb.p(1024), ks=fb.p(2048), vc=fb.p(3072), vs=fb.p(4096),
             cap=64, max_ctx=64, scale=0.125, out=fb.p(8192), out_dtype=0, lse=None, ws=fb.p(16384),
             ws_bytes=1 << 15)
    for key, val in kw.items():
        a[key] = fb.p(val[1]) if isinstance(val, tuple) else val
    cache = (a["kc"], a["ks"], a["vc"], a["vs"])
    if what == "append":
        return lib.tq_quantize_append_q8(a["k"], a["v"], a["dtype"], a["B"], a["Hkv"], a["n"], a["d"], a["fmt"],
                                         a["block"], a["pos"], a["valid"], *cache, a["cap"], None)
    if what == "read":
        return lib.tq_read_q8(*cache, a["cap"], a["B"], a["Hkv"], a["d"], a["fmt"], a["block"], a["pos"],
                              a["valid"], a["n"], a["k"], a["v"], a["out_dtype"], 0, None)
    if what == "attend":
        return lib.tq_sdpa_q8(a["q"], a["dtype"], a["B"], a["Hq"], a["Hkv"], a["n"], a["d"], a["fmt"],
                              a["block"], *cache, a["cap"], a["pos"], a["valid"], a["max_ctx"], a["scale"],
                              a["out"], a["out_dtype"], a["lse"], a["ws"], a["ws_bytes"], None)
    return lib.tq_sdpa_q8_decode_append(a["q"], a["dtype"], a["k"], a["v"], a["kv_dtype"], a["B"], a["Hq"],
                                        a["Hkv"], a["d"], a["fmt"], a["block"], *cache, a["cap"], a["pos"],
                                        a["max_ctx"], a["scale"], a["out"], a["out_dtype"], a["lse"], a["ws"],
                                        a["ws_bytes"], None)


@pytest.mark.parametrize("what", ["append", "read", "attend", "step"])
@pytest.mark.parametrize("kw,code", [
    (dict(kc=None), INVALID), (dict(ks=None), INVALID), (dict(vc=None), INVALID), (dict(vs=None), INVALID),
    (dict(kc=("off", 1032)), INVALID), (dict(vc=("off", 3073)), INVALID), (dict(vs=("off", 4098)), INVALID),
    (dict(B=0), INVALID), (dict(Hkv=0), INVALID), (dict(cap=0), INVALID), (dict(fmt=2), INVALID),
    (dict(fmt=-1), INVALID), (dict(B=1 << 16, Hkv=1 << 16), INVALID), (dict(k=None), INVALID),
    (dict(d=32), UNSUPPORTED), (dict(d=160), UNSUPPORTED), (dict(d=512), UNSUPPORTED),
    (dict(block=0), UNSUPPORTED), (dict(block=8), UNSUPPORTED), (dict(block=48), UNSUPPORTED),
    (dict(block=256), UNSUPPORTED)])
def test_every_call_checks_its_cache(lib, what, kw, code):
    if what == "attend" and "k" in kw:
        kw = dict(q=None)
    assert call(lib, what, **kw) == code


@pytest.mark.parametrize("what,kw,code", [
    ("append", dict(v=None), INVALID), ("append", dict(pos=None), INVALID), ("append", dict(n=0), INVALID),
    ("append", dict(dtype=2), INVALID), ("append", dict(k=("off", 264)), INVALID),
    ("append", dict(pos=("off", 770)), INVALID), ("append", dict(valid=("off", 770)), INVALID),
    ("append", dict(n=(1 << 31) - 1, B=64), INVALID),
    ("read", dict(v=None), INVALID), ("read", dict(n=0), INVALID), ("read", dict(out_dtype=3), INVALID),
    ("read", dict(k=("off", 264)), INVALID), ("read", dict(n=(1 << 31) - 1, B=64), INVALID),
    ("attend", dict(pos=None), INVALID), ("attend", dict(out=None), INVALID), ("attend", dict(dtype=2), INVALID),
    ("attend", dict(out_dtype=2), INVALID), ("attend", dict(Hq=7), INVALID), ("attend", dict(Hq=1), INVALID),
    ("attend", dict(n=0), INVALID), ("attend", dict(max_ctx=0), INVALID), ("attend", dict(max_ctx=65), INVALID),
    ("attend", dict(scale=0.0), INVALID), ("attend", dict(scale=-1.0), INVALID),
    ("attend", dict(scale=float("inf")), INVALID), ("attend", dict(scale=float("nan")), INVALID),
    ("attend", dict(q=("off", 8)), INVALID), ("attend", dict(out=("off", 8200)), INVALID),
    ("attend", dict(lse=("off", 8196)), INVALID), ("attend", dict(ws=None), WORKSPACE),
    ("attend", dict(ws=("off", 16392)), WORKSPACE), ("attend", dict(ws_bytes=255), WORKSPACE),
    ("attend", dict(n=1 << 30, Hq=16), INVALID),
    ("step", dict(v=None), INVALID), ("step", dict(kv_dtype=2), INVALID), ("step", dict(k=("off", 264)), INVALID),
    ("step", dict(max_ctx=65), INVALID), ("step", dict(ws_bytes=0), WORKSPACE)])
def test_refusals(lib, what, kw, code):
    assert call(lib, what, **kw) == code


@pytest.mark.parametrize("args", [(0, 8, 8, 128, 1, 10), (1, 6, 4, 128, 1, 10), (1, 8, 8, 160, 1, 10),
                                  (1, 8, 8, 128, 0, 10), (1, 8, 8, 128, 1, 0)])
def test_workspace_of_invalid_sizes_is_zero(lib, args):
    assert _lib.sdpa_q8_workspace_bytes(*args) == 0


@pytest.mark.parametrize("B,Hq,Hkv,d,n,T", [(1, 4, 4, 128, 1, 4096), (1, 64, 8, 128, 1, 131073),
                                            (16, 64, 8, 128, 1, 65536), (8, 64, 8, 64, 5, 16384),
                                            (1, 64, 8, 128, 2048, 16384), (2, 32, 32, 96, 33, 100),
                                            (1, 8, 8, 256, 1, (1 << 31) - 1)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_workspace_is_deterministic_and_bounded(lib, B, Hq, Hkv, d, n, T, dtype):
    ws = _lib.sdpa_q8_workspace_bytes(B, Hq, Hkv, d, n, T, dtype)
    assert ws == _lib.sdpa_q8_workspace_bytes(B, Hq, Hkv, d, n, T, dtype)
    # a call is split only until its work items fill the GPU a few times
    assert 4 * B <= ws <= 4 * B + 256 + max(64 << 20, 8 * 4 * B * Hq * n * (d + 4))


@pytest.mark.parametrize("kw", [dict(head_dim=80), dict(head_dim=512), dict(block=8), dict(block=100),
                                dict(dtype=torch.uint8), dict(dtype=torch.float8_e5m2)])
def test_cache_class_refuses(kw):
    a = dict(batch=1, num_kv_heads=2, head_dim=128, capacity=70, device="cpu") | kw
    with pytest.raises(ValueError):
        BlockKVCache(**a)


def test_python_calls_refuse_host_tensors():
    c = BlockKVCache(1, 2, 64, 40, block=16, device="cpu")
    assert c.k_scales.shape == (1, 2, 3) and c.nbytes() == 2 * (2 * 40 * 64 + 2 * 3 * 4)
    pos = torch.zeros(1, dtype=torch.int32)
    x = torch.zeros(1, 2, 1, 64)
    for f in (lambda: c.append(x, x, pos), lambda: c.read(pos, 1), lambda: c.decode(x[:, :, 0], pos, 40),
              lambda: c.attend(x, pos, 40), lambda: c.decode_append(x[:, :, 0], x, x, pos, 40)):
        with pytest.raises(ValueError):
            f()


# ------------------------------------------------------------- the reference itself

def test_reference_e4m3_is_the_format():
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    every = every[~every.isnan()].double().numpy()
    assert np.array_equal(nearest(every, "e4m3"), every)
    grid = np.unique(every)
    mid = (grid[1:] + grid[:-1]) / 2  # halfway values, and values just beside them
    x = np.concatenate([mid, mid * (1 + 1e-6), mid * (1 - 1e-6), [1e-9, -500.0, 500.0, np.inf, -np.inf]])
    want = torch.from_numpy(np.clip(x, -448, 448)).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(nearest(np.float32(x).astype(np.float64), "e4m3"), want)
    assert nearest(np.array([np.nan]), "e4m3")[0] == 0


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_reference_append_bounds(fmt):
    """One write: every value is within half a step of its input; a block's largest is Q s."""
    rng = np.random.default_rng(1)
    x = rng.standard_normal((1, 1, 40, 64)).astype(np.float32).astype(np.float64)
    c = Cache(1, 1, 48, 64, 16, fmt)
    c.append(x, 2 * x, [5])
    s = c.scales[0][0, 0].copy()
    got = c.values(0, 0, 0, 5, 45)
    half = s[np.arange(5, 45) // 16][:, None] * 0.5
    err = np.abs(got - x[0, 0])
    if fmt == "int8":
        assert np.all(err <= half * (1 + 1e-5))
    else:  # 3 bits behind the leading one: half a step is 2^-4 of the value, 2^-10 s near 0
        assert np.all(err <= np.maximum(np.abs(x[0, 0]) * 2.0 ** -4, half * 2.0 ** -9) * (1 + 1e-5))
    assert np.abs(c.codes[0][0, 0]).max() == QMAX[fmt]
    # a larger row in the same block raises the scale and moves the kept codes
    before = c.values(0, 0, 0, 32, 45).copy()
    c.append(100 * x[:, :, :1], x[:, :, :1], [45])
    assert c.scales[0][0, 0, 2] > s[2] and c.scales[0][0, 0, 1] == s[1]
    after = c.values(0, 0, 0, 32, 45)
    assert np.all(np.abs(after - before) <= c.scales[0][0, 0, 2] * (0.5 if fmt == "int8" else 1e9))


def test_reference_attention_of_equal_keys_is_the_mean():
    c = Cache(1, 1, 32, 64, 16, "int8")
    rng = np.random.default_rng(2)
    k = np.ones((1, 1, 20, 64))
    v = rng.integers(-127, 128, (1, 1, 20, 64)).astype(np.float64)
    v[..., 0] = 127  # scale 1: codes are the values
    c.append(k, v, [0])
    out, lse = c.attend(np.ones((1, 1, 3, 64)), [20], None, 0.5)
    assert np.allclose(out[0, 0, 2], v[0, 0, :20].mean(0)) and np.allclose(out[0, 0, 0], v[0, 0, :18].mean(0))
    assert np.allclose(lse[0, 0], np.log2([18, 19, 20]) + 32 / np.log(2))
    out, lse = c.attend(np.ones((1, 1, 3, 64)), [1], None, 0.5)  # two of the three sit in front of row 0
    assert np.all(out[0, 0, :2] == 0) and np.all(lse[0, 0, :2] == -np.inf) and np.allclose(out[0, 0, 2], v[0, 0, 0])
