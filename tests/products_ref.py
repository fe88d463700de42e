"""Plain 64-bit forms of the 8-bit quantiser and of the dense and grouped products, for the tests.

Written from the definitions in include/nvfp4moe.h with numpy on the CPU; nothing here calls the
library.
"""
import numpy as np
import torch


def _decode_all():
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        if e == 15 and m == 7:
            a = np.nan
        else:
            a = (m / 8.0) * 2.0 ** -6 if e == 0 else (1.0 + m / 8.0) * 2.0 ** (e - 7)
        v[c] = -a if c & 128 else a
    return v


E4M3 = _decode_all()
GRID = E4M3[:127]                     # the non-negative numbers, ascending; code = index


def f64(t):
    """Any tensor the tests use -> float64 numpy."""
    t = t.detach().cpu()
    if t.dtype == torch.float8_e4m3fn:
        return E4M3[t.contiguous().view(torch.uint8).numpy()]
    return t.double().numpy()


def nearest_code(v):
    """Code of the E4M3 number nearest to v (|v| <= 448), ties to the even code; the sign is kept."""
    a = np.abs(v)
    hi = np.minimum(np.searchsorted(GRID, a), 126)
    lo = np.maximum(hi - 1, 0)
    up, down = GRID[hi] - a, a - GRID[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (code | np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def quantize(x, block_rows):
    """(codes uint8, scales float32) of a bf16 tensor [B, R, K], block by block."""
    d = f64(x)
    B, R, K = d.shape
    rb, kb = -(-R // block_rows), -(-K // 128)
    q = np.empty(d.shape, np.uint8)
    s = np.empty((B, rb, kb), np.float32)
    with np.errstate(all="ignore"):
        for b in range(B):
            for i in range(rb):
                for j in range(kb):
                    at = (b, slice(i * block_rows, (i + 1) * block_rows), slice(j * 128, (j + 1) * 128))
                    p = d[at]
                    a = np.nan if np.isnan(p).any() else np.abs(p).max()
                    s[b, i, j] = 1.0 if a == 0 else a / 448.0
                    v = p * 448.0 / (448.0 if a == 0 else a)
                    q[at] = np.where(np.isnan(v), 0x7F, nearest_code(np.nan_to_num(v)))
    return q, s


def spread(s, block_rows, R, K):
    """Block scales [.., rb, kb] -> one of each element."""
    s = np.repeat(s, 128, axis=-1)[..., :K]
    return s if block_rows == 1 else np.repeat(s, block_rows, axis=-2)[..., :R, :]


def rows_of(offsets, token_list, R, k, gather, scatter):
    """(x row or -1, y row, expert) of every list position that belongs to an expert and writes a row."""
    off = np.clip(np.asarray(offsets, np.int64), 0, R)
    out = []
    for e in range(len(off) - 1):
        for r in range(off[e], off[e + 1]):
            src = dst = r
            if gather or scatter:
                entry = int(token_list[r])
                bad = not 0 <= entry < R
                if gather:
                    src = -1 if bad else entry // k
                if scatter:
                    if bad:
                        continue
                    dst = entry
            out.append((src, dst, e))
    return out


def grouped(x, w, offsets, token_list, R, k, gather, scatter):
    """(y, S, written): float64 [R, N] rows, the sums of |x w| behind them, and which rows are written."""
    N = w.shape[1]
    y, S, written = np.zeros((R, N)), np.zeros((R, N)), np.zeros(R, bool)
    for src, dst, e in rows_of(offsets, token_list, R, k, gather, scatter):
        v = np.zeros(x.shape[1]) if src < 0 else x[src]
        y[dst], S[dst], written[dst] = w[e] @ v, np.abs(w[e]) @ np.abs(v), True
    return y, S, written


def bound(y, S, K, bf16, fp8):
    """How far an fp32 sum of K products may be from the exact one. The products of two 8-bit
    significands are exact in fp32. The tensor cores add at least 8 products to the running sum at a
    time, each time off by at most one unit of 2^-23 of a partial sum that is at most S (they may cut
    off instead of rounding); joining up to 16 partial sums adds as many roundings of 2^-24. With block
    scales, every block of 128 adds the rounding of the scales' product and of the addition, 2 * 2^-24.
    An output in bf16 adds half a step, 2^-8 of its value."""
    steps = (K / 8 + 1) * 2 + 16 + (2 * (K / 128 + 1) if fp8 else 0)
    fp32 = steps * 2.0 ** -24 * S
    return fp32 + (2.0 ** -8 * (np.abs(y) + fp32) if bf16 else 0.0)
