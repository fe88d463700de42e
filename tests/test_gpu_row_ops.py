"""nvfp4_quantize_rows, nvfp4_dequantize_rows, rmsnorm_residual and moe_swiglu on the GPU, against plain 64-bit forms
(rows_ref).

Codes of bf16 rows are equal bit for bit. The norm's and the SwiGLU's values are fp32 before they are rounded: a code
may be the other one only where the exact quotient lies within the derived fp32 error of the point between the two.
"""
import numpy as np
import pytest
import torch

import rows_ref as ref

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _np(t):
    return t.detach().cpu().numpy()


def _norm_error(K):
    """fp32 error of a normed element, relative: at most K / 8 / 32 + 16 + 5 + 32 additions in a chain of the sum of
    squares (2^-24 each, halved by the root; 64 elements a thread at most), and the roundings of each square, of the
    mean, eps, root, reciprocal, 1 + w and two products."""
    return ((64 + 37) / 2 + 8) * 2.0 ** -24


# ---------------------------------------------------------------- quantiser

def _rows(K, seed):
    g = _gen(seed)
    x = torch.randn(9, K, generator=g) * torch.pow(2.0, torch.randint(-30, 30, (9, 1), generator=g).float())
    x[1] = 0
    x[2, : K // 2] = 0
    x[3, 0] = 3e38
    x[4] = 2.0 ** -133                     # subnormal bf16
    x[5] *= 2.0 ** -20
    x[5, 7] = 1e30                         # blocks whose scale underflows
    x[6] = -0.0
    return x.to(BF16)


@pytest.mark.parametrize("K", [32, 64, 96, 1000 // 32 * 32, 1024, 1056, 2048, 4096, 4128, 16384, 32768])
def test_quantize_rows(nv, K):
    x = _rows(K, K)
    packed, scales, rs = nv.nvfp4_quantize_rows(x.cuda())
    codes, e, s = ref.quantize_rows(ref.f64(x))
    assert np.array_equal(_np(rs), s)
    assert np.array_equal(_np(scales), e)
    assert np.array_equal(_np(packed), ref.pack_codes(codes))
    # and back: what the rows stand for, exactly where bf16 can hold it
    want = ref.code_values(codes) * np.repeat(ref.E4M3[e], 16, axis=1) * s[:, None].astype(np.float64)
    back = nv.nvfp4_dequantize_rows(packed, scales, rs, out_dtype=torch.float32)
    normal = np.abs(want) >= 2.0 ** -126
    assert np.array_equal(_np(back)[normal], want.astype(np.float32)[normal])
    back = nv.nvfp4_dequantize_rows(packed, scales, rs)
    assert np.array_equal(ref.f64(back)[normal], want[normal])


def test_quantize_rows_every_tie(nv):
    """Every midpoint of E2M1 under every block scale that a row of largest 2688 can have, both signs, and the values
    next to it; every midpoint of the block scales."""
    mid = (ref.E2M1[1:] + ref.E2M1[:-1]) / 2
    rows = []
    for e in ref.GRID[1:]:
        vals = np.concatenate([mid, -mid]) * e
        v = np.zeros(32)
        v[0], v[1:15], v[15] = 6 * e, vals, 0.0          # block scale e exactly
        v[16] = 2688.0                                    # row scale 1
        rows += [v, np.where(np.arange(32) == 16, v, v * (1 + 2.0 ** -8)), np.where(np.arange(32) == 16, v, v * (1 - 2.0 ** -8))]
    for b in (ref.GRID[1:] + ref.GRID[:-1]) / 2 * 6:
        v = np.zeros(32)
        v[0], v[1], v[16] = b, -b / 2, 2688.0
        rows.append(v)
    x = torch.from_numpy(np.stack(rows)).to(BF16)
    for scale in (1.0, 2.0 ** -100, 2.0 ** 110):
        y = x * scale
        packed, scales, rs = nv.nvfp4_quantize_rows(y.cuda())
        codes, e, s = ref.quantize_rows(ref.f64(y))
        assert np.array_equal(_np(rs), s) and np.array_equal(_np(scales), e)
        assert np.array_equal(_np(packed), ref.pack_codes(codes))


def test_quantize_rows_that_are_not_finite(nv):
    x = torch.randn(5, 96, generator=_gen(1)).to(BF16)
    x[0, 3], x[2, 95], x[3, 0] = float("nan"), float("inf"), float("-inf")
    packed, scales, rs = (_np(t) for t in nv.nvfp4_quantize_rows(x.cuda()))
    codes, e, s = ref.quantize_rows(ref.f64(x))
    assert np.array_equal(rs, s, equal_nan=True) and np.isnan(rs[[0, 2, 3]]).all()
    for r in (0, 2, 3):
        assert not packed[r].any() and not scales[r].any()
    for r in (1, 4):
        assert np.array_equal(scales[r], e[r]) and np.array_equal(packed[r], ref.pack_codes(codes[r]))


def test_quantize_rows_agrees_with_the_packer(nv):
    """A row whose largest value makes the packer's tensor scale a power of two packs to the same bytes."""
    x = torch.randn(3, 2048, generator=_gen(2)).to(BF16)
    x = torch.clamp(x, -3, 3)
    x[:, 5] = 5.25                               # 5.25 / 2688 = 2^-9
    packed, scales, rs = nv.nvfp4_quantize_rows(x.cuda())
    for r in range(3):
        w = nv.nvfp4_pack(x[r:r + 1].float().cuda())
        assert float(w.tensor_scale[0]) == float(rs[r]) == 2.0 ** -9
        assert torch.equal(w.packed[0], packed[r]) and torch.equal(w.scales[0], scales[r])


def test_dequantize_a_packed_matrix_and_a_layers_expert(nv):
    g = _gen(3)
    N, K = 70, 96
    w = nv.nvfp4_pack((torch.randn(N, K, generator=g) * 0.02).cuda())
    t = float(w.tensor_scale[0])
    want = ref.values(_np(w.packed), _np(w.scales)) * t
    got = nv.nvfp4_dequantize_rows(w.packed, w.scales, w.tensor_scale, out_dtype=torch.float32)
    assert np.all(np.abs(ref.f64(got) - want) <= 2.0 ** -24 * np.abs(want))
    got = nv.nvfp4_dequantize_rows(w.packed, w.scales, w.tensor_scale)
    assert np.all(np.abs(ref.f64(got) - want) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(want))
    L = nv.MoELayer.allocate(96, 2, 1, 64, 0, device="cuda")
    for e in range(2):
        L.pack_expert(e, *(torch.randn(*s, generator=g).cuda() for s in ((64, 96), (64, 96), (96, 64))))
    for e in range(2):
        got = nv.nvfp4_dequantize_rows(L.gu_packed[e], L.gu_scales[e], L.gu_tscale[e], out_dtype=torch.float32)
        want = ref.values(_np(L.gu_packed[e]), _np(L.gu_scales[e])) * np.repeat(_np(L.gu_tscale[e]).astype(np.float64), 64)[:, None]
        assert np.all(np.abs(ref.f64(got) - want) <= 2.0 ** -24 * np.abs(want))


# ---------------------------------------------------------------- norm

def _check_rows(nv, kind, rows, x, err):
    if kind == nv.ROWS_BF16:
        assert np.all(np.abs(ref.f64(rows) - x) <= (2.0 ** -8 * (1 + err) + err) * np.abs(x))
    elif kind == nv.ROWS_FP8:
        ref.check_fp8(_np(rows[0].view(torch.uint8)), _np(rows[1]).astype(np.float64), x, err)
    else:
        ref.check_nvfp4(*(_np(t) for t in rows), x, err)


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("T,H", [(1, 32), (1, 2048), (5, 1024 + 32), (3, 96), (7, 4096), (2, 4160), (300, 544),
                                 (2, 20480), (1, 32768)])
@pytest.mark.parametrize("delta", [False, True])
def test_norm(nv, kind, T, H, delta):
    g = _gen(H + T)
    h = (torch.randn(T, H, generator=g) * torch.pow(2.0, torch.randint(-6, 6, (T, 1), generator=g).float())).to(BF16)
    d = torch.randn(T, H, generator=g).to(BF16) if delta else None
    w = (torch.randn(H, generator=g) * 0.3).to(BF16)
    want_h, x = ref.norm(ref.f64(h), ref.f64(d) if delta else None, ref.f64(w), 1e-6)
    hc = h.cuda()
    h_out, rows = nv.rmsnorm_residual(hc, w.cuda(), 1e-6, delta=d.cuda() if delta else None, kind=kind)
    assert np.array_equal(ref.f64(h_out), want_h)
    assert delta or h_out is hc
    _check_rows(nv, kind, rows, x, _norm_error(H))


@pytest.mark.parametrize("kind,H", [(0, 8), (0, 1000), (1, 16), (1, 1008), (1, 144)])
def test_norm_of_widths_that_only_some_kinds_take(nv, kind, H):
    g = _gen(H)
    h, w = torch.randn(6, H, generator=g).to(BF16), torch.randn(H, generator=g).to(BF16)
    _, x = ref.norm(ref.f64(h), None, ref.f64(w), 1e-5)
    _, rows = nv.rmsnorm_residual(h.cuda(), w.cuda(), 1e-5, kind=kind)
    _check_rows(nv, kind, rows, x, _norm_error(H))


@pytest.mark.parametrize("H", [16, 128, 1008, 2048, 5120, 20480])
def test_e4m3_scales_of_rows_known_to_the_bit(nv, H):
    """Rows whose mean square is a power of four and gates whose sigmoid is 1 give fp32 values without a rounding: the
    scales are a / 448 rounded once, as fp8_quantize_block128's, and the codes off by the roundings of 448 / a and of one
    product at most."""
    T = 12
    g = _gen(H)
    sign = torch.randint(0, 2, (T, H), generator=g) * 2.0 - 1.0
    power = torch.pow(2.0, torch.randint(-12, 13, (T, 1), generator=g).float())
    w = (torch.randn(H, generator=g) * 0.5).to(BF16).float()
    w = torch.where((w.abs() < 2.0 ** -14) | (w < -0.99), torch.zeros(()), w)       # 1 + w is exact
    x = ref.f64(sign) * (1.0 + ref.f64(w))
    _, (q, s) = nv.rmsnorm_residual((sign * power).to(BF16).cuda(), w.to(BF16).cuda(), 0.0, kind=nv.ROWS_FP8)
    gates = torch.pow(2.0, torch.randint(7, 10, (T, H), generator=g).float())       # exp(-128) is no part of 1 + exp(-128)
    up = torch.randn(T, H, generator=g).to(BF16).float() * power
    x2 = ref.f64(gates) * ref.f64(up)
    q2, s2 = nv.moe_swiglu(torch.cat([gates, up], dim=1).to(BF16).cuda(), nv.ROWS_FP8)
    for codes, scales, want in ((q, s, x), (q2, s2, x2)):
        for j in range(scales.shape[1]):
            a = np.abs(want[:, j * 128:(j + 1) * 128]).max(axis=1).astype(np.float32)
            assert np.array_equal(_np(scales)[:, j], a / np.float32(448.0))
        ref.check_fp8(_np(codes.view(torch.uint8)), _np(scales).astype(np.float64), want, 0.0)
    back, sb = nv.fp8_quantize_block128(torch.from_numpy(x2).to(BF16).cuda())
    assert torch.equal(sb, s2)


def test_norm_in_place_and_copies(nv):
    g = _gen(8)
    h, d = (torch.randn(33, 2048, generator=g).to(BF16).cuda() for _ in range(2))
    w = torch.randn(2048, generator=g).to(BF16).cuda()
    want_h, want = nv.rmsnorm_residual(h, w, delta=d)
    for into in (0, 1):
        hh, dd = h.clone(), d.clone()
        got_h, got = nv.rmsnorm_residual(hh, w, delta=dd, h_out=(hh, dd)[into])
        assert torch.equal(got_h, want_h) and torch.equal(got, want)
        assert torch.equal((dd, hh)[into], (d, h)[into])
    copy = torch.empty_like(h)
    got_h, got = nv.rmsnorm_residual(h, w, h_out=copy)
    assert got_h is copy and torch.equal(copy, h)
    same = h.clone()
    nv.rmsnorm_residual(same, w, h_out=same)
    assert torch.equal(same, h)
    # the rows do not depend on how many there are
    for kind in (0, 1, 2):
        _, many = nv.rmsnorm_residual(h, w, delta=d, kind=kind)
        _, one = nv.rmsnorm_residual(h[20:21].contiguous(), w, delta=d[20:21].contiguous(), kind=kind)
        for a, b in zip((many,) if kind == 0 else many, (one,) if kind == 0 else one):
            assert torch.equal(a[20:21].view(torch.uint8), b.view(torch.uint8))


def test_norm_of_zeros_and_of_values_that_are_not_finite(nv):
    h = torch.randn(5, 256, generator=_gen(4)).to(BF16)
    h[0] = 0
    h[2, 3], h[3, 9] = float("nan"), float("inf")
    w = torch.zeros(256, dtype=BF16)
    for kind in (0, 1, 2):
        _, rows = nv.rmsnorm_residual(h.cuda(), w.cuda(), 1e-6, kind=kind)
        if kind == 0:
            x = ref.f64(rows)
            assert not x[0].any() and np.isnan(x[2]).all() and np.isnan(x[3, 9]) and not x[3, :9].any()
            assert np.isfinite(x[[1, 4]]).all()
        elif kind == 1:
            s = _np(rows[1])
            assert (s[0] == 1).all() and np.isnan(s[2]).all() and np.isfinite(s[[1, 4]]).all() and np.isnan(s[3, 0])
        else:
            s = _np(rows[2])
            assert s[0] == 1 and np.isnan(s[2:4]).all() and np.isfinite(s[[1, 4]]).all()
            assert not _np(rows[0])[[0, 2, 3]].any()


# ---------------------------------------------------------------- SwiGLU

@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("dtype", [BF16, torch.float32])
@pytest.mark.parametrize("R,I", [(1, 32), (7, 512), (65, 544), (3, 2048), (2, 5120), (1, 32768)])
def test_swiglu(nv, kind, dtype, R, I):
    g = _gen(R + I)
    gu = (torch.randn(R, 2 * I, generator=g) * 3).to(dtype)
    gu[0, :4] = torch.tensor([-80.0, 80.0, 0.0, -0.0])
    d = ref.f64(gu)
    # the fast exponential is off by 2 + 1.173 |g| units of 2^-23 at most; the sum, the quotient and the product round
    err = (4 + 1.2 * np.abs(d[:, :I])) * 2.0 ** -23 + 3 * 2.0 ** -24
    rows = nv.moe_swiglu(gu.cuda(), kind)
    _check_rows(nv, kind, rows, ref.silu_up(d), err)


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("dtype", [BF16, torch.float32])
def test_swiglu_of_gates_far_below_zero(nv, kind, dtype):
    """exp(-g) passes fp32 at g = -88.7, silu(g) does not: with a large up the product is an ordinary number."""
    I = 128
    g = _gen(kind)
    gate = torch.empty(9, I)
    for r, (lo, hi) in enumerate(((-87, -80), (-88.7, -88), (-89.5, -88.7), (-91, -88.5), (-92, -90), (-92, -80), (-92, 5), (-60, -50),
                                  (60, 90))):
        gate[r] = lo + (hi - lo) * torch.rand(I, generator=g)
    gate = gate.to(dtype)
    silu = gate.double() * torch.sigmoid(gate.double())
    up = (torch.randn(9, I, generator=g).double() / silu.abs()).clamp(-1e38, 1e38).to(dtype)
    gu = torch.cat([gate, up], dim=1)
    d = ref.f64(gu)
    # the fast exponential is off by 2 + 1.173 |g| units of exp(-|g|), which are those of subnormals from |g| = 87.4 on;
    # the division by 2 units of 2^-23; the sum and two products round (g exp(g) is a subnormal below -91.9)
    unit = np.maximum(2.0 ** -23, 2.0 ** -149 * np.exp(np.abs(d[:, :I])))
    err = (2 + 1.2 * np.abs(d[:, :I])) * unit + 2 * 2.0 ** -23 + 3 * 2.0 ** -24 + unit / 64
    x = ref.silu_up(d)
    assert (np.abs(x) > 2.0 ** -20).mean() > 0.99 and (d[:, :I] < -88.8).mean() > 0.3
    _check_rows(nv, kind, nv.moe_swiglu(gu.cuda(), kind), x, err)


def test_swiglu_of_gates_without_a_finite_value(nv):
    inf, nan = float("inf"), float("nan")
    gate, up = [inf, -inf, nan, 1e38, -1e38, -0.0, 0.0, 3.0], [2.0, 2.0, 2.0, 2.0, 2.0, 2.0, 2.0, inf]
    got = nv.moe_swiglu(torch.tensor([gate + up], device="cuda"))[0].tolist()
    assert got[0] == inf and np.isnan(got[1:3]).all() and got[3] == float(torch.tensor(2e38).to(BF16))
    assert got[4:7] == [0.0, 0.0, 0.0] and got[7] == inf


def test_swiglu_of_widths_that_only_some_kinds_take(nv):
    for kind, I in ((0, 8), (0, 1000), (1, 16), (1, 1136)):
        gu = torch.randn(5, 2 * I, generator=_gen(I)).to(BF16)
        err = (4 + 1.2 * 6) * 2.0 ** -23 + 3 * 2.0 ** -24
        _check_rows(nv, kind, nv.moe_swiglu(gu.cuda(), kind), ref.silu_up(ref.f64(gu)), err)


def test_row_ops_outputs_streams_and_graphs(nv):
    """Given outputs, another stream, no rows at all, and a captured call replayed on changed inputs."""
    g = _gen(6)
    gu = torch.randn(40, 1024, generator=g).to(BF16).cuda()
    h = torch.randn(40, 512, generator=g).to(BF16).cuda()
    w = torch.randn(512, generator=g).to(BF16).cuda()
    calls = [lambda **kw: nv.moe_swiglu(gu, nv.ROWS_NVFP4, **kw), lambda **kw: nv.moe_swiglu(gu, nv.ROWS_FP8, **kw),
             lambda **kw: nv.rmsnorm_residual(h, w, kind=nv.ROWS_NVFP4, **kw)[1], lambda **kw: nv.nvfp4_quantize_rows(h, **kw)]
    st = torch.cuda.Stream()
    for call in calls:
        want = call()
        out = tuple(torch.zeros_like(t) for t in want)
        st.wait_stream(torch.cuda.current_stream())
        got = call(out=out, stream=st)
        st.synchronize()
        assert all(a is b for a, b in zip(got, out))
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(want, out))
        graph = torch.cuda.CUDAGraph()
        for t in out:
            t.view(torch.uint8).zero_()
        with torch.cuda.graph(graph):
            call(out=out)
        keep = gu.clone(), h.clone()
        gu.copy_(gu.flip(0)), h.copy_(h.flip(0))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, out):
            assert torch.equal(a.flip(0).view(torch.uint8), b.view(torch.uint8))
        gu.copy_(keep[0]), h.copy_(keep[1])
    e = lambda *s, dtype=BF16: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
    assert nv.nvfp4_quantize_rows(e(0, 64))[0].shape == (0, 32)
    assert nv.moe_swiglu(e(0, 64)).shape == (0, 32)
    assert nv.rmsnorm_residual(e(0, 64), e(64))[1].shape == (0, 64)
    assert nv.nvfp4_dequantize_rows(e(0, 32, dtype=torch.uint8), e(0, 4, dtype=torch.uint8), e(0, dtype=torch.float32)).shape == (0, 64)


def test_rows_past_32_bits(nv):
    """2.3e9 elements: the last rows are where they should be."""
    R, K = 70001, 32768
    x = torch.zeros(R, K, dtype=BF16, device="cuda")
    tail = torch.randn(3, K, generator=_gen(1)).to(BF16).cuda()
    x[-3:] = tail
    packed, scales, rs = nv.nvfp4_quantize_rows(x)
    for a, b in zip((packed, scales, rs), nv.nvfp4_quantize_rows(tail)):
        assert torch.equal(a[-3:], b) and not a[1000].any() or a.dtype == torch.float32
    back = nv.nvfp4_dequantize_rows(packed, scales, rs)
    assert torch.equal(back[-3:], nv.nvfp4_dequantize_rows(*nv.nvfp4_quantize_rows(tail)))
    del back, packed, scales
    w = torch.zeros(K, dtype=BF16, device="cuda")
    _, (q, s) = nv.rmsnorm_residual(x, w, kind=nv.ROWS_FP8)
    _, (qt, st) = nv.rmsnorm_residual(tail, w, kind=nv.ROWS_FP8)
    assert torch.equal(q[-3:].view(torch.uint8), qt.view(torch.uint8)) and torch.equal(s[-3:], st)
    del q, s
    assert torch.equal(nv.moe_swiglu(x)[-3:], nv.moe_swiglu(tail))


def test_all_three_arrays_of_rows_past_32_bits(nv):
    """2.3e9 elements, rows of zeros but for the last three: codes, block scales and row scales of each are where they should
    be, and 1 and zeros everywhere else."""
    R, K = 70001, 32768
    x = torch.zeros(R, K, dtype=BF16, device="cuda")
    tail = (torch.randn(3, K, generator=_gen(1)) * 8).to(BF16).cuda()
    x[-3:] = tail
    packed, scales, rs = nv.nvfp4_quantize_rows(x)
    want = nv.nvfp4_quantize_rows(tail)
    assert torch.equal(packed[-3:], want[0]) and torch.equal(scales[-3:], want[1]) and torch.equal(rs[-3:], want[2])
    assert (want[2] < 0.1).all() and (rs[:-3] == 1).all() and not packed[:-3].any() and not scales[:-3].any()
