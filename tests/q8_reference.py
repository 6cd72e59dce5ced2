"""The 8-bit block-scaled cache in plain numpy, 64 bits, one sequence and head at
a time: what the q8 calls of include/tq.h are compared with.  Written from the
definitions there; shares no code with the package."""
import numpy as np
import torch

QMAX = {"int8": 127.0, "e4m3": 448.0}
TORCH = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


def _fl32(x):
    return np.asarray(x, np.float64).astype(np.float32).astype(np.float64)


def nearest(y, fmt):
    """Nearest code of y, halves to even, ends saturate, NaN is 0."""
    y = np.where(np.isnan(y), 0.0, y)
    y = np.clip(y, -QMAX[fmt], QMAX[fmt])
    if fmt == "int8":
        return np.round(y)
    _, e = np.frexp(np.maximum(np.abs(y), 2.0 ** -6))  # |y| = m 2^e, m in [1/2, 1)
    step = 2.0 ** (e - 4)
    return np.round(y / step) * step


def _divide(x, s):
    """fl32(x / s), 0 where s is 0."""
    with np.errstate(all="ignore"):
        return np.zeros_like(x) if s == 0 else _fl32(x / s)


class Cache:
    """codes[b][h] as float64 [capacity][d], scales[b][h] as float64 [blocks]; which = K, V."""

    def __init__(self, B, H, capacity, d, block, fmt):
        self.B, self.H, self.capacity, self.d, self.block, self.fmt = B, H, capacity, d, block, fmt
        blocks = -(-capacity // block)
        self.codes = [np.zeros((B, H, capacity, d)) for _ in range(2)]
        self.scales = [np.zeros((B, H, blocks)) for _ in range(2)]

    def append(self, k, v, pos, n_valid=None):
        """k, v [B][H][n][d] (any float type, as float64)."""
        for w, x in enumerate((k, v)):
            for b in range(self.B):
                valid = x.shape[2] if n_valid is None else min(max(int(n_valid[b]), 0), x.shape[2])
                if pos[b] < 0:
                    continue
                for h in range(self.H):
                    self._append(self.codes[w][b, h], self.scales[w][b, h], x[b, h, :valid], int(pos[b]))

    def _append(self, codes, scales, x, pos):
        x = x[: max(0, self.capacity - pos)]
        T, at = self.block, 0
        while at < len(x):
            j, r = divmod(pos + at, T)
            new = x[at:at + T - r]
            mag = np.abs(new)
            a = np.max(mag[np.isfinite(mag)], initial=0.0)
            s = float(_fl32(a / QMAX[self.fmt]))
            if r > 0:
                old = scales[j]
                s = max(s, old)
                if s > old:
                    kept = codes[j * T:j * T + r]
                    codes[j * T:j * T + r] = nearest(_divide(_fl32(kept * old), s), self.fmt)
            codes[pos + at:pos + at + len(new)] = nearest(_divide(new, s), self.fmt)
            scales[j] = s
            at += len(new)

    def values(self, w, b, h, lo, hi):
        rows = np.arange(lo, hi)
        return _fl32(self.codes[w][b, h, lo:hi] * self.scales[w][b, h, rows // self.block][:, None])

    def attend(self, q, ctx, q_lens, scale):
        """q [B][Hq][n][d] -> (out [B][Hq][n][d], log2 of the sums of weights [B][Hq][n])."""
        B, Hq, n, d = q.shape
        out, lse = np.zeros(q.shape), np.full(q.shape[:3], -np.inf)
        for b in range(B):
            m = n if q_lens is None else int(q_lens[b])
            for hq in range(Hq):
                h = hq // (Hq // self.H)
                k, v = (self.values(w, b, h, 0, int(ctx[b])) for w in (0, 1))
                for i in range(m):
                    last = int(ctx[b]) - m + i + 1
                    if last <= 0:
                        continue
                    s = scale * (k[:last] @ q[b, hq, i])
                    p = np.exp(s - s.max())
                    out[b, hq, i] = p @ v[:last] / p.sum()
                    lse[b, hq, i] = np.log2(p.sum()) + s.max() / np.log(2)
        return out, lse

    def absmax_v(self, b, h, ctx):
        return np.max(np.abs(self.values(1, b, h, 0, ctx)), initial=0.0)

    def upload(self, cache):
        """Copies this cache's content into a BlockKVCache."""
        for mine, theirs in zip(self.codes, (cache.k_codes, cache.v_codes)):
            theirs.copy_(torch.from_numpy(mine).float().to(TORCH[self.fmt]))
        for mine, theirs in zip(self.scales, (cache.k_scales, cache.v_scales)):
            theirs.copy_(torch.from_numpy(mine).float())


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)
