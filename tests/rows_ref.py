"""Plain 64-bit forms of NVFP4 rows, the norm, the SwiGLU and of rows sorted by expert, for the tests.

Written from the definitions in include/nvfp4moe.h with numpy on the CPU; nothing here calls the library.
"""
import numpy as np

from products_ref import E4M3, GRID, f64, nearest_code  # noqa: F401  (shared with the 8-bit tests)

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def nearest_e2m1(v):
    """Code of the E2M1 number nearest to v, ties to the even code, saturating; the sign is kept."""
    a = np.minimum(np.abs(v), 6.0)
    hi = np.minimum(np.searchsorted(E2M1, a), 7)
    lo = np.maximum(hi - 1, 0)
    up, down = E2M1[hi] - a, a - E2M1[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (code | np.where(np.signbit(v), 8, 0)).astype(np.uint8)


def row_scale(amax):
    """The smallest power of two >= amax / 2688, at least 2^-126; 1 for zeros, NaN where amax is not finite."""
    out = np.full(amax.shape, np.nan, np.float64)
    for i, a in enumerate(amax):
        if a == 0:
            out[i] = 1.0
        elif np.isfinite(a):
            s = 2.0 ** -126
            while s < a / 2688.0:
                s *= 2.0
            out[i] = s
    return out


def quantize_rows(x):
    """(codes uint8 [R, K], one a byte, block scale codes uint8 [R, K/16], row scales float32 [R])."""
    R, K = x.shape
    with np.errstate(all="ignore"):
        bad = ~np.isfinite(x).all(axis=1)
        d = np.where(bad[:, None], 0.0, x)
        s = row_scale(np.abs(d).max(axis=1) if K else np.zeros(R))
        b = np.abs(d).reshape(R, K // 16, 16).max(axis=2)
        e = nearest_code(b / (6.0 * s[:, None]))
        unit = np.repeat(E4M3[e], 16, axis=1) * s[:, None]
        codes = np.where(unit == 0, 0, nearest_e2m1(d / np.where(unit == 0, 1.0, unit)))
        s[bad] = np.nan
    return codes.astype(np.uint8), e, s.astype(np.float32)


def pack_codes(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack_codes(packed):
    out = np.empty(packed.shape[:-1] + (2 * packed.shape[-1],), np.uint8)
    out[..., 0::2], out[..., 1::2] = packed & 15, packed >> 4
    return out


def code_values(codes):
    return np.where(codes & 8, -1.0, 1.0) * E2M1[codes & 7]


def values(packed, scales):
    """code x block scale of packed rows [..., K/2] and E4M3 scale codes [..., K/16]."""
    return code_values(unpack_codes(packed)) * np.repeat(E4M3[scales], 16, axis=-1)


def norm(h, delta, w, eps):
    """(h_out, x): h_out rounded to bf16 as float64, x unrounded."""
    import torch
    if delta is not None:
        h = torch.from_numpy(h + delta).to(torch.bfloat16).double().numpy()      # exact in 64 bits, one rounding
    return h, h / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps) * (1.0 + w)


def silu_up(gu):
    I = gu.shape[1] // 2
    g, u = gu[:, :I], gu[:, I:]
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def within(got, lo_hi):
    """Every code is the nearest to the lower or the upper of two values that are a tolerance apart (both codes are
    neighbours, or the same, for tolerances far below a step)."""
    lo, hi = lo_hi
    return (got == lo) | (got == hi)


def check_fp8(q, s, x, delta):
    """E4M3 rows q, s against 64-bit x whose fp32 values are off by at most `delta` of them (an array or a number)."""
    R, K = x.shape
    delta = np.broadcast_to(delta, x.shape)
    for j in range((K + 127) // 128):
        at = slice(j * 128, min(K, (j + 1) * 128))
        p, d = x[:, at], delta[:, at].max(axis=1, keepdims=True)
        a = np.abs(p).max(axis=1, keepdims=True)
        want = np.where(a == 0, 1.0, a / 448.0)
        assert np.all(np.abs(s[:, j:j + 1] - want) <= (d + 2.0 ** -23) * want), "scales"
        v = np.where(a == 0, 0.0, 448.0 * p / np.where(a == 0, 1.0, a))
        # both the value and the largest one are off by delta, and three roundings of 2^-24
        t = 2 * d + 4 * 2.0 ** -24
        lim = lambda f: nearest_code(np.clip(v * f, -448.0, 448.0))  # noqa: E731
        assert within(q[:, at] & 0x7F, (lim(1 - t) & 0x7F, lim(1 + t) & 0x7F)).all(), "codes"


def check_nvfp4(packed, scales, row_scales, x, delta):
    """NVFP4 rows against 64-bit x whose fp32 values are off by at most `delta` of them."""
    R, K = x.shape
    delta = np.broadcast_to(delta, x.shape)
    d = delta.max(axis=1, keepdims=True) + 4 * 2.0 ** -24
    a = np.abs(x).max(axis=1)
    s = row_scales.astype(np.float64)
    assert within(s, (row_scale(a * (1 - d[:, 0])), row_scale(a * (1 + d[:, 0])))).all(), "row scales"
    b = np.abs(x).reshape(R, K // 16, 16).max(axis=2) / (6.0 * s[:, None])
    assert within(scales, (nearest_code(np.minimum(b * (1 - d), 448)), nearest_code(np.minimum(b * (1 + d), 448)))).all(), "block scales"
    unit = np.repeat(E4M3[scales], 16, axis=1) * s[:, None]
    v = x / np.where(unit == 0, 1.0, unit)
    codes = unpack_codes(packed)
    lo, hi = (np.where(unit == 0, 0, nearest_e2m1(v * f) & 7) for f in (1 - d, 1 + d))
    assert within(codes & 7, (lo, hi)).all(), "codes"
    signs = (codes & 8 != 0) == np.signbit(x)
    assert (signs | (x == 0) | (unit == 0)).all(), "signs"


def permute(x, token_list, k, positions):
    """rows; positions is changed in place."""
    R = len(token_list)
    rows = np.zeros((R, x.shape[1]))
    for r, entry in enumerate(token_list):
        if 0 <= entry < R:
            rows[r], positions[entry] = x[entry // k], r
    return rows


def combine(rows, w, positions, add, T, k):
    """(y, sum of magnitudes)."""
    R = T * k
    y, S = np.zeros((T, rows.shape[1])), np.zeros((T, rows.shape[1]))
    for t in range(T):
        for j in range(k):
            p = positions[t * k + j] if positions is not None else t * k + j
            if 0 <= p < R:
                c = 1.0 if w is None else w[t, j]
                y[t] += c * rows[p]
                S[t] += abs(c) * np.abs(rows[p])
    if add is not None:
        y, S = y + add, S + np.abs(add)
    return y, S


def combine_backward(dy, rows, w, positions, T, k, d_rows):
    """(d_w, sums of magnitudes); d_rows is changed in place."""
    R = T * k
    d_w, S = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            p = positions[t * k + j] if positions is not None else t * k + j
            if 0 <= p < R:
                d_rows[p] = (1.0 if w is None else w[t, j]) * dy[t]
                d_w[t, j], S[t, j] = dy[t] @ rows[p], np.abs(dy[t]) @ np.abs(rows[p])
    return d_w, S
