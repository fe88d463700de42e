"""fp8_quantize_block128, fp8_gemm_block128 and the products grouped by expert on the GPU, against
plain 64-bit forms (products_ref).

Most cases use operands whose sums are exact in fp32 in any order (small integers, block scales that
are powers of two), so every output is known to the bit: fp32 outputs are equal, bf16 outputs are the
one rounding of the exact sum. Cases with real values use the bound that products_ref derives.
"""
import numpy as np
import pytest
import torch

import products_ref as ref

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _small(gen, *shape, most=4):
    return torch.randint(-most, most + 1, shape, generator=gen).float()


def _pow2(gen, *shape):
    """Scales 1/4 .. 4: with |x|, |w| <= 4 and K <= 4096 every product is a multiple of 2^-4 and every
    sum stays below 2^20: 24 bits hold it."""
    return torch.pow(2.0, torch.randint(-2, 3, shape, generator=gen).float())


def _check_exact(y, want, what=""):
    got = y.detach().cpu()
    w = torch.from_numpy(np.ascontiguousarray(want)).to(got.dtype if got.dtype == torch.float32 else torch.float32)
    w = w.to(got.dtype)
    bad = ~((got == w) | (got.isnan() & w.isnan()))
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:5].tolist())


# ---------------------------------------------------------------- quantiser

@pytest.mark.parametrize("B,R,K", [(1, 1, 16), (1, 1, 128), (1, 3, 144), (1, 129, 2048), (2, 130, 272), (3, 1, 1040),
                                   (1, 1000, 64), (1, 1100, 2048), (2, 1050, 1040)])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize(nv, B, R, K, block_rows):
    g = _gen(R * K + block_rows)
    x = (torch.randn(B, R, K, generator=g) * torch.pow(2.0, torch.randint(-20, 20, (B, R, 1), generator=g).float()))
    x = x.to(torch.bfloat16)
    x[0, 0, : K // 2] = 0                       # a block of zeros where K >= 256, else zeros in a block
    q, s = nv.fp8_quantize_block128(x.cuda(), block_rows)
    torch.cuda.synchronize()
    qw, sw = ref.quantize(x, block_rows)
    assert np.array_equal(s.cpu().numpy(), sw)
    assert np.array_equal(q.cpu().view(torch.uint8).numpy(), qw)


def test_quantize_every_tie(nv):
    """Blocks whose largest value is 448, 1.75 and 7 times powers of two meet every midpoint of E4M3
    exactly; every bf16 significand against every other covers the quotients next to them."""
    mid = (ref.GRID[1:] + ref.GRID[:-1]) / 2
    rows = []
    for scale in (1.0, 2.0 ** -20, 2.0 ** 30):
        v = np.concatenate([mid, -mid])
        for i in range(0, len(v), 127):
            part = v[i:i + 127] * scale
            rows.append(np.concatenate([[448.0 * scale], part, np.zeros(127 - len(part))]))
    m = np.arange(128, 256) / 128.0
    for a in m:                                  # largest 255-ish significands over one binade and below
        for d in (0, 1, 5, 8, 9, 10):
            v = m * 2.0 ** -d
            v[v > a] /= 2
            v[0] = a
            rows.append(v)
    x = torch.from_numpy(np.stack(rows)).to(torch.bfloat16)[None]
    q, s = nv.fp8_quantize_block128(x.cuda(), 1)
    qw, sw = ref.quantize(x, 1)
    assert np.array_equal(s.cpu().numpy(), sw)
    assert np.array_equal(q.cpu().view(torch.uint8).numpy(), qw)


def test_quantize_extremes(nv):
    """Zeros of both signs, the smallest and largest bf16, infinities and NaN."""
    tiny, big = 2.0 ** -133, float(torch.finfo(torch.bfloat16).max)
    x = torch.zeros(1, 8, 128)
    x[0, 0, 1] = -0.0
    x[0, 1, :3] = torch.tensor([tiny, -tiny, 0.0])
    x[0, 2, :3] = torch.tensor([big, -big, tiny])
    x[0, 3, :4] = torch.tensor([2.0 ** -126, 2.0 ** -130, 2.0 ** -64, 2.0 ** -65])
    x[0, 4, :3] = torch.tensor([float("inf"), 1.0, -1.0])
    x[0, 5, :2] = torch.tensor([float("nan"), 1.0])
    x[0, 6, :3] = torch.tensor([float("nan"), float("-inf"), 3.0])
    x[0, 7] = 5.0
    x = x.to(torch.bfloat16)
    for br, times in ((1, 1), (1, 2500), (128, 1), (128, 40)):      # few blocks and many
        q, s = nv.fp8_quantize_block128(x.repeat(times, 1, 1).cuda(), br)
        qw, sw = (np.repeat(v, times, axis=0) for v in ref.quantize(x, br))
        assert np.array_equal(s.cpu().numpy(), sw, equal_nan=True)
        got = q.cpu().view(torch.uint8).numpy()
        nan = (qw & 0x7F) == 0x7F
        assert np.array_equal((got & 0x7F) == 0x7F, nan)
        assert np.array_equal(got[~nan], qw[~nan])


def test_quantize_two_dimensions_outputs_and_streams(nv):
    x = torch.randn(300, 272, generator=_gen(5)).to(torch.bfloat16).cuda()
    q, s = nv.fp8_quantize_block128(x)
    assert q.shape == (300, 272) and s.shape == (300, 3)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    q2, s2 = torch.empty_like(q), torch.empty_like(s)
    out = nv.fp8_quantize_block128(x, q=q2, scales=s2, stream=st)
    q3, s3 = nv.fp8_quantize_block128(x, stream=st)
    st.synchronize()
    assert out[0] is q2 and out[1] is s2
    for a, b in ((q, q2), (q, q3)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert torch.equal(s, s2) and torch.equal(s, s3)
    for shape in ((0, 64), (2, 0, 64)):
        q0, _ = nv.fp8_quantize_block128(torch.empty(shape, dtype=torch.bfloat16, device="cuda"))
        assert q0.shape == shape


# ---------------------------------------------------------------- dense

def _dense_case(T, N, K, seed):
    g = _gen(seed)
    x, w = _small(g, T, K), _small(g, N, K)
    xs, ws = _pow2(g, T, -(-K // 128)), _pow2(g, -(-N // 128), -(-K // 128))
    want = (x.double() * torch.from_numpy(ref.spread(xs.numpy(), 1, T, K)).double()) @ \
        (w.double() * torch.from_numpy(ref.spread(ws.numpy(), 128, N, K)).double()).t()
    return x.to(F8).cuda(), xs.cuda(), w.to(F8).cuda(), ws.cuda(), want.numpy()


@pytest.mark.parametrize("T,N,K", [(1, 1, 16), (1, 128, 128), (1, 130, 144), (2, 129, 2048), (7, 300, 1040), (8, 64, 256),
                                   (9, 1000, 400), (16, 128, 4096), (17, 257, 272), (33, 136, 640), (64, 2048, 512),
                                   (65, 131, 384), (129, 260, 1296), (255, 127, 128), (257, 384, 2000), (700, 513, 1024)])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_dense_exact(nv, T, N, K, dt):
    x, xs, w, ws, want = _dense_case(T, N, K, T + N + K)
    wk = nv.Workspace(256)
    y = nv.fp8_gemm_block128(x, xs, w, ws, out_dtype=dt, ws=wk)
    assert wk.status() == nv.NVFP4_OK
    assert y.shape == (T, N) and y.dtype == dt
    _check_exact(y, want)


@pytest.mark.parametrize("T,N,K", [(1, 8192, 2048), (5, 500, 2000), (40, 300, 1040), (300, 520, 2048), (600, 1111, 1296)])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_dense_real_values(nv, T, N, K, dt):
    g = _gen(T * 7 + N)
    x = torch.randn(T, K, generator=g).to(torch.bfloat16).cuda()
    x[:, 3] *= 30
    w = (torch.randn(N, K, generator=g) * 0.02).to(torch.bfloat16).cuda()
    xq, xs = nv.fp8_quantize_block128(x)
    wq, ws = nv.fp8_quantize_block128(w, 128)
    y = nv.fp8_gemm_block128(xq, xs, wq, ws, out_dtype=dt)
    xd = ref.f64(xq) * ref.spread(ref.f64(xs), 1, T, K)
    wd = ref.f64(wq) * ref.spread(ref.f64(ws), 128, N, K)
    want, S = xd @ wd.T, np.abs(xd) @ np.abs(wd).T
    err = np.abs(ref.f64(y) - want)
    assert np.all(err <= ref.bound(want, S, K, dt == torch.bfloat16, True)), float((err / S).max())


@pytest.mark.parametrize("T", [1, 40, 300])
def test_dense_special_values_stay_in_their_row_and_column(nv, T):
    """NaN codes and infinite scales reach the outputs of their row or column and no other."""
    x, xs, w, ws, want = _dense_case(T, 300, 400, 11 + T)
    xq = x.clone()
    xq.view(torch.uint8)[T - 1, 399] = 0x7F
    w.view(torch.uint8)[299, 5] = 0xFF
    y = nv.fp8_gemm_block128(xq, xs, w, ws, out_dtype=torch.float32)
    bad = np.zeros((T, 300), bool)
    bad[T - 1], bad[:, 299] = True, True
    assert np.array_equal(np.isnan(ref.f64(y)), bad)
    assert np.array_equal(ref.f64(y)[~bad], want[~bad])
    xs2 = xs.clone()
    xs2[T - 1, 0] = float("inf")
    y = ref.f64(nv.fp8_gemm_block128(x, xs2, w, ws, out_dtype=torch.float32))
    assert not np.isfinite(y[T - 1]).any()
    assert np.array_equal(y[:T - 1, :299], want[:T - 1, :299])


def test_dense_empty_and_alignment_and_refusals(nv):
    x, xs, w, ws, want = _dense_case(4, 130, 256, 1)
    y = nv.fp8_gemm_block128(x[:0], xs[:0], w, ws)
    assert y.shape == (0, 130)
    # scale tensors need 4-byte alignment only: a view one row in
    xs5 = torch.cat([xs[:1], xs])
    _check_exact(nv.fp8_gemm_block128(x, xs5[1:], w, ws, out_dtype=torch.float32), want)
    with pytest.raises(nv.NVFP4Error):
        nv.fp8_gemm_block128(x, xs, w.t(), ws)
    with pytest.raises(nv.NVFP4Error):
        nv.fp8_gemm_block128(x, xs[:, :1], w, ws)
    with pytest.raises(nv.NVFP4Error):
        nv.fp8_gemm_block128(x, xs, w, ws, out_dtype=torch.float16)
    with pytest.raises(nv.NVFP4Error):
        nv.fp8_gemm_block128(x, xs, w, ws, y=torch.empty(4, 131, device="cuda"))
    flat = torch.zeros(4 * 256 + 8, dtype=torch.uint8, device="cuda").view(F8)
    with pytest.raises(nv.NVFP4Error):
        nv.fp8_gemm_block128(flat[8:].view(4, 256), xs, w, ws)


# ---------------------------------------------------------------- grouped

def _counts(kind, R, E, g):
    if kind == "one":                            # every row in one expert
        c = [0] * E
        c[E // 2] = R
    elif kind == "even":
        c = [R // E + (1 if e < R % E else 0) for e in range(E)]
    elif kind == "holes":                        # only every third expert
        on = list(range(0, E, 3))
        c = [0] * E
        for i in range(R):
            c[on[i % len(on)]] += 1
    else:                                        # skewed
        p = torch.softmax(torch.randn(E, generator=g) * 2, 0)
        c = torch.bincount(torch.multinomial(p, R, True, generator=g), minlength=E).tolist()
    return torch.tensor([0] + list(np.cumsum(c)), dtype=torch.int32)


def _grouped_case(T, k, E, N, K, kind, rows, fp8, seed):
    g = _gen(seed)
    R = T * k
    off = _counts(kind, R, E, g)
    lst = torch.randperm(R, generator=g).to(torch.int32)
    x, w = _small(g, T if rows == "gather" else R, K), _small(g, E, N, K)
    a = dict(x=x.to(F8 if fp8 else torch.bfloat16).cuda(), w=w.to(F8 if fp8 else torch.bfloat16).cuda())
    xd, wd = x.double().numpy(), w.double().numpy()
    if fp8:
        KB = -(-K // 128)
        xs, ws = _pow2(g, x.shape[0], KB), _pow2(g, E, -(-N // 128), KB)
        a.update(x_scales=xs.cuda(), w_scales=ws.cuda())
        xd, wd = xd * ref.spread(xs.numpy(), 1, 0, K), wd * ref.spread(ws.numpy(), 128, N, K)
    a.update(offsets=off.cuda(), k=k, gather=rows == "gather", scatter=rows == "scatter",
             token_list=lst.cuda() if rows != "list" else None)
    return a, xd, wd, off, lst, R


def _call(nv, a, **kw):
    return (nv.moe_grouped_gemm_fp8 if "x_scales" in a else nv.moe_grouped_gemm_bf16)(**a, **kw)


def _want(a, xd, wd, off, lst, R):
    return ref.grouped(xd, wd, off.numpy(), lst.numpy(), R, a["k"], a["gather"], a["scatter"])


CASES = [  # T, k, E, N, K, kind
    (1, 1, 1, 1, 16, "one"), (1, 8, 256, 128, 256, "even"), (1, 8, 40, 130, 2048, "skew"), (3, 2, 5, 17, 48, "holes"),
    (5, 8, 64, 300, 272, "skew"), (64, 4, 30, 129, 512, "skew"), (40, 8, 3, 200, 144, "even"),
    (300, 2, 4, 260, 400, "one"), (257, 1, 2, 127, 640, "even"), (200, 8, 17, 385, 1040, "skew"),
    (1024, 1, 256, 64, 128, "skew"), (33, 1, 33, 136, 4096, "even"),
]


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("rows", ["gather", "scatter", "list"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_grouped_exact(nv, case, rows, fp8):
    a, xd, wd, off, lst, R = _grouped_case(*case, rows, fp8, sum(case[:5]))
    want, _, written = _want(a, xd, wd, off, lst, R)
    assert written.all()
    wk = nv.Workspace(256)
    for dt in (torch.float32, torch.bfloat16):
        y = _call(nv, a, out_dtype=dt, ws=wk)
        _check_exact(y, want, dt)
    assert wk.status() == nv.NVFP4_OK


@pytest.mark.parametrize("K", [8, 24, 72, 120, 136])
@pytest.mark.parametrize("T", [2, 200])
def test_grouped_bf16_widths_of_8(nv, T, K):
    a, xd, wd, off, lst, R = _grouped_case(T, 3, 7, 50, K, "skew", "gather", False, K)
    _check_exact(_call(nv, a, out_dtype=torch.float32), _want(a, xd, wd, off, lst, R)[0])


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("T", [2, 150])
def test_grouped_both_maps_and_unwritten_rows(nv, T, fp8):
    """gather and scatter at once; a list that stops early and starts late leaves the other rows of y."""
    a, xd, wd, off, lst, R = _grouped_case(T, 4, 6, 140, 272, "even", "gather", fp8, 9)
    a["scatter"] = True
    off = off.clone()
    off[0], off[-1] = 1, R - 2                  # the first expert's first and the last one's last rows belong to none
    a["offsets"] = off.cuda()
    want, _, written = _want(a, xd, wd, off, lst, R)
    assert 0 < written.sum() < R - 1
    y = torch.full((R, 140), -77.0, device="cuda")
    assert _call(nv, a, y=y) is y
    want[~written] = -77.0
    _check_exact(y, want)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("T,K", [(3, 144), (180, 144), (180, 2048)])
def test_grouped_bad_offsets_and_entries_stay_in_bounds(nv, T, K, fp8):
    """Offsets outside [0, R] and groups that run backwards, entries outside [0, R): as documented. (The
    last case has few tiles and a long K, which several pairs of CTAs share.)"""
    for rows in ("gather", "scatter"):
        a, xd, wd, off, lst, R = _grouped_case(T, 2, 5, 130, K, "even", rows, fp8, 21)
        off = torch.tensor([-5, 2, 1, 3, R, R + 100], dtype=torch.int32)
        lst[2], lst[0], lst[R - 1] = -1, R, 2 ** 31 - 1
        a["offsets"], a["token_list"] = off.cuda(), lst.cuda()
        # group 1 (2 to 1) is empty and group 2 (1 to 3) overlaps group 0 in position 1: both are in
        # bounds, and what they write is undefined
        y = torch.full((R, 130), -77.0, device="cuda")
        _call(nv, a, y=y)
        torch.cuda.synchronize()
        want, _, written = ref.grouped(xd, wd, np.array([3, 3, 3, 3, R, R]), lst.numpy(), R, 2, rows == "gather",
                                       rows == "scatter")
        got = ref.f64(y)
        assert np.array_equal(got[written], want[written])
        if rows == "scatter":
            touched = {int(v) for v in lst if 0 <= int(v) < R}
            for r in set(range(R)) - touched:
                assert (got[r] == -77.0).all()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("K", [144, 1024])
def test_grouped_groups_that_all_overlap(nv, K, fp8):
    """Every group is the whole list: far more tiles than the host counts. The call stays in bounds and
    returns, and the next one is right."""
    a, xd, wd, off, lst, R = _grouped_case(130, 2, 40, 130, K, "even", "list", fp8, 3)
    good = a["offsets"]
    bad = torch.tensor([0, R] * 20 + [0], dtype=torch.int32).cuda()
    y = torch.full((R + 1, 130), -77.0, device="cuda")
    _call(nv, dict(a, offsets=bad), y=y[:R])
    assert (y[R] == -77.0).all()
    _check_exact(_call(nv, dict(a, offsets=good), out_dtype=torch.float32), _want(a, xd, wd, off, lst, R)[0])


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("N,K", [(260, 2048), (1030, 1040), (5000, 528), (300, 144)])
@pytest.mark.parametrize("rows", [64, 65, 127, 128, 129, 192, 257, 400])
def test_tile_heights_and_shared_sums(nv, rows, N, K, fp8):
    """Few and many tiles just below and above every height of a tile, with K in one, two and four parts."""
    for E, kind, order in ((1, "even", "list"), (2, "skew", "gather")):
        a, xd, wd, off, lst, R = _grouped_case(rows * E, 1, E, N, K, kind, order, fp8, rows + N)
        wk = nv.Workspace(256)
        y = _call(nv, a, out_dtype=torch.float32, ws=wk)
        assert wk.status() == nv.NVFP4_OK
        _check_exact(y, _want(a, xd, wd, off, lst, R)[0], (E, kind, order))


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("N", [1, 3, 33, 250, 255, 257, 1022])
def test_grouped_output_widths(nv, N, fp8):
    """Rows of y that start at every alignment, ends inside a 32-output piece and a 128-row half; the
    element after the last row is left alone."""
    a, xd, wd, off, lst, R = _grouped_case(60, 2, 3, N, 160, "skew", "scatter", fp8, N)
    want = _want(a, xd, wd, off, lst, R)[0]
    for dt in (torch.bfloat16, torch.float32):
        buf = torch.full((R * N + 64,), -77.0, dtype=dt, device="cuda")
        _call(nv, a, y=buf[:R * N].view(R, N))
        _check_exact(buf[:R * N].view(R, N), want, dt)
        assert (buf[R * N:] == -77.0).all()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("case", [(1, 8, 64, 256, 1024), (90, 4, 12, 200, 1000), (700, 2, 6, 300, 512)], ids=str)
def test_grouped_real_values(nv, case, fp8):
    T, k, E, N, K = case
    K = K // 16 * 16
    g = _gen(T)
    off = _counts("skew", T * k, E, g)
    lst = torch.randperm(T * k, generator=g).to(torch.int32)
    x = torch.randn(T, K, generator=g).to(torch.bfloat16).cuda()
    w = (torch.randn(E, N, K, generator=g) * 0.02).to(torch.bfloat16).cuda()
    a = dict(x=x, w=w)
    xd, wd = ref.f64(x), ref.f64(w)
    if fp8:
        xq, xs = nv.fp8_quantize_block128(x)
        wq, ws = nv.fp8_quantize_block128(w, 128)
        a = dict(x=xq, x_scales=xs, w=wq, w_scales=ws)
        xd, wd = ref.f64(xq) * ref.spread(ref.f64(xs), 1, T, K), ref.f64(wq) * ref.spread(ref.f64(ws), 128, N, K)
    a.update(offsets=off.cuda(), token_list=lst.cuda(), k=k, gather=True)
    want, S, _ = ref.grouped(xd, wd, off.numpy(), lst.numpy(), T * k, k, True, False)
    for dt in (torch.float32, torch.bfloat16):
        y = _call(nv, a, out_dtype=dt)
        err = np.abs(ref.f64(y) - want)
        assert np.all(err <= ref.bound(want, S, K, dt == torch.bfloat16, fp8)), float((err / S).max())


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("T", [1, 100])
def test_grouped_graph_streams_and_repeats(nv, T, fp8):
    """The same bits from eager calls, another stream and a captured graph that is replayed on new rows."""
    a, xd, wd, off, lst, R = _grouped_case(T, 8, 20, 260, 528, "skew", "gather", fp8, 33)
    want = _want(a, xd, wd, off, lst, R)[0]
    y = _call(nv, a, out_dtype=torch.float32)
    _check_exact(y, want)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    y2 = _call(nv, a, out_dtype=torch.float32, stream=st)
    st.synchronize()
    assert torch.equal(y, y2)
    y3 = torch.zeros_like(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _call(nv, a, y=y3)
    # new routing in the same buffers: all rows to the last expert, the list reversed
    off2 = torch.zeros_like(off)
    off2[-1] = R
    a["offsets"].copy_(off2)
    a["token_list"].copy_(lst.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    _check_exact(y3, _want(a, xd, wd, off2, lst.flip(0), R)[0])


_FIRST_IN_CAPTURE = """
import sys
sys.path[:0] = [%r, %r]
import torch
import nvfp4_w4a16_moe_gb300 as nv
T, N, K = %d, 300, 2048
x = torch.ones(T, K, dtype=torch.bfloat16, device="cuda")
w = torch.ones(1, N, K, dtype=torch.bfloat16, device="cuda")
off = torch.tensor([0, T], dtype=torch.int32, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    y = nv.moe_grouped_gemm_bf16(x, w, off)
    q, s = nv.fp8_quantize_block128(x)
    v, t = nv.fp8_quantize_block128(w[0], 128)
    z = nv.fp8_gemm_block128(q, s, v, t, out_dtype=torch.float32)
g.replay()
torch.cuda.synchronize()
# 1 = 448 / 448: codes 448, scales fl(1 / 448), so every product is 1 within four roundings
assert (y == K).all() and ((z - K).abs() <= K * 2.0 ** -20).all()
"""


@pytest.mark.parametrize("T", [4, 300])
def test_first_calls_of_a_process_inside_a_capture(nv, T):
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = _FIRST_IN_CAPTURE % (root, os.path.join(root, "tests"), T)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_two_streams_at_once(nv):
    """Large and small calls on two streams, interleaved, each with its own outputs."""
    cases = [_grouped_case(T, 4, 20, 520, 1040, "skew", "gather", fp8, T) for T in (2, 200) for fp8 in (False, True)]
    wants = [_want(*c) for c in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    torch.cuda.synchronize()
    for i in range(12):
        c = cases[i % 4]
        outs.append(_call(nv, c[0], out_dtype=torch.float32, stream=streams[(i // 2) % 2]))
    torch.cuda.synchronize()
    for i, y in enumerate(outs):
        _check_exact(y, wants[i % 4][0])


def test_grouped_empty_and_refusals(nv):
    a, xd, wd, off, lst, R = _grouped_case(4, 2, 3, 20, 64, "even", "gather", False, 2)
    e = dict(a, x=a["x"][:0], token_list=a["token_list"][:0], offsets=torch.zeros(4, dtype=torch.int32, device="cuda"))
    assert _call(nv, e).shape == (0, 20)
    for kw in (dict(token_list=None), dict(token_list=a["token_list"][:3]), dict(offsets=a["offsets"][:3]), dict(k=0),
               dict(offsets=a["offsets"].long()), dict(w=a["w"].float()), dict(w=a["w"].transpose(1, 2)),
               dict(out_dtype=torch.float16), dict(x=a["x"][:, :32])):
        with pytest.raises(nv.NVFP4Error):
            _call(nv, dict(a, **kw))


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("rows", ["gather", "scatter", "list"])
@pytest.mark.parametrize("T", [2, 90])
def test_grouped_neighbours_do_not_leak(nv, T, rows, fp8):
    """Tiles reach past an expert's weight rows and list positions: NaN in the matrices of experts without
    rows, and in rows of x that no position reads, stays there."""
    E, N, K = 9, 130, 272
    a, xd, wd, off, lst, R = _grouped_case(T, 4, E, N, K, "holes", rows, fp8, 44)
    off = off.clone()
    last = int(off[-1]) - 3                      # the last three positions belong to no expert
    off = torch.minimum(off, torch.tensor(last, dtype=torch.int32))
    a["offsets"] = off.cuda()
    bits = lambda t: t.view(torch.uint8 if fp8 else torch.int16)
    nan = 0x7F if fp8 else 0x7FC0
    empty = (off[1:] == off[:-1]).nonzero().flatten()
    bits(a["w"])[empty.cuda()] = nan
    if rows == "gather":
        used = {int(e) // 4 for e in lst[:last]}
    else:
        used = set(range(last))
    idle = [r for r in range(a["x"].shape[0]) if r not in used]
    if idle:
        bits(a["x"])[torch.tensor(idle).cuda()] = nan
    want, _, written = _want(a, np.nan_to_num(xd), wd, off, lst, R)
    y = torch.full((R, N), -77.0, device="cuda")
    _call(nv, a, y=y)
    want[~written] = -77.0
    _check_exact(y, want)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_grouped_outputs_and_weights_past_32_bits(nv, fp8):
    """2.3e9 outputs, and 2^33 weight elements: the last rows and the last expert are where they should be."""
    g = torch.Generator(device="cuda").manual_seed(6)
    dt = F8 if fp8 else torch.bfloat16

    def small(*shape):
        return torch.randint(-2, 3, shape, generator=g, device="cuda", dtype=torch.int8).to(torch.bfloat16).to(dt)

    def check(x, w, off, rows, R, N):
        kw = {}
        if fp8:
            kw = dict(x_scales=torch.ones(x.shape[0], -(-x.shape[1] // 128), device="cuda"),
                      w_scales=torch.ones(w.shape[0], -(-N // 128), -(-x.shape[1] // 128), device="cuda"))
        y = _call(nv, dict(x=x, w=w, offsets=off, **kw))
        for r in rows:
            e = int((off[1:] <= r).sum())
            want = (w[e].float() @ x[r].float()).to(torch.bfloat16)
            assert torch.equal(y[r], want), r

    R, N, K = 280000, 8200, 64
    off = torch.tensor([0, 100, R], dtype=torch.int32, device="cuda")
    check(small(R, K), small(2, N, K), off, (0, 99, 100, 262143, R - 1), R, N)
    E, N, K = 128, 8192, 8192
    w = torch.empty(E, N, K, dtype=dt, device="cuda")
    for e in range(E):
        w[e] = small(N, K)
    for R in (4, 70):
        off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        off[1:] = R // 2
        off[-1] = R
        check(small(R, K), w, off, (0, R // 2 - 1, R // 2, R - 1), R, N)


def _run_twice(step, n):
    """The outputs of n steps in a row, and of the same steps with the device idle between all calls."""
    outs = []
    for wait in (False, True):
        torch.cuda.synchronize()
        outs.append([[o.clone() for o in step(i, torch.cuda.synchronize if wait else (lambda: None))] for i in range(n)])
    torch.cuda.synchronize()
    return outs


def test_chains_over_reused_buffers(nv):
    """Quantise, multiply, round, quantise again in the same buffers, few and many rows in turn: a call that
    started before the one ahead of it was done, or read a stale line, would differ from the slow run."""
    g = _gen(8)
    E, N = 4, 512
    w = (torch.randn(E, N, N, generator=g) * 0.06).to(torch.bfloat16).cuda()
    wq, ws = nv.fp8_quantize_block128(w, 128)
    xs = [torch.randn(r, N, generator=g).to(torch.bfloat16).cuda() for r in (6, 700)]
    offs = [torch.tensor([0, r // 4, r // 2, r // 2, r], dtype=torch.int32, device="cuda") for r in (6, 700)]
    bufs = [(torch.empty_like(x), torch.empty(x.shape, dtype=F8, device="cuda"),
             torch.empty(x.shape[0], N // 128, device="cuda")) for x in xs]

    def step(i, wait):
        b = i % 2
        (y, q, s), off = bufs[b], offs[b]
        y.copy_(xs[b] * (1 + i % 3))
        for _ in range(4):
            wait()
            nv.fp8_quantize_block128(y, q=q, scales=s)
            wait()
            nv.moe_grouped_gemm_fp8(q, s, wq, ws, off, y=y)
            wait()
            nv.fp8_quantize_block128(y, q=q, scales=s)
            wait()
            nv.fp8_gemm_block128(q, s, wq[1], ws[1], y=y)
        wait()
        return y, q.view(torch.uint8), s

    fast, slow = _run_twice(step, 30)
    for a, b in zip(fast, slow):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_chains_with_the_nvfp4_kernels(nv):
    """The NVFP4 packer, GEMV and single-token layer read weights before they wait for the kernel ahead of
    them: with the new kernels in between, freshly written weights and workspaces are still seen."""
    import workload as wl
    from harness import gpu_layer
    layer = gpu_layer(wl.LayerInputs(wl.SMALL256, seed=3))
    H = wl.SMALL256.H
    g = _gen(12)
    masters = [torch.randn(512, H, generator=g).cuda() * 0.1 for _ in range(3)]
    x = torch.randn(1, H, generator=g).to(torch.bfloat16).cuda()
    w = (torch.randn(1, H, H, generator=g) * 0.1).to(torch.bfloat16).cuda()
    off = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    W = nv.nvfp4_pack(masters[0])
    wk = nv.Workspace(nv.moe_layer_workspace_size(layer, 1))
    q, s = nv.fp8_quantize_block128(x)

    def step(i, wait):
        wait()
        nv.nvfp4_pack(masters[i % 3], out=W)
        wait()
        nv.fp8_quantize_block128(x, q=q, scales=s)
        wait()
        a = nv.nvfp4_gemv_w4a16(W, x)
        wait()
        b = nv.moe_layer_forward(layer, x, ws=wk)
        wait()
        c = nv.moe_grouped_gemm_bf16(b, w, off)
        wait()
        d = nv.moe_layer_forward(layer, c, ws=wk)
        wait()
        return a, b, c, d

    fast, slow = _run_twice(step, 40)
    assert wk.status() == nv.NVFP4_OK
    for a, b in zip(fast, slow):
        assert all(torch.equal(p.view(torch.int16), r.view(torch.int16)) for p, r in zip(a, b))


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("T", [1, 50, 300])
def test_experts_of_a_layer_from_the_routers_lists(nv, T, fp8):
    """Route, gate/up gathered from the tokens, SwiGLU, down scattered to the entries, weighted sum: the
    experts of one layer in bf16 or 8 bits, against the same steps in 64 bits on the GPU's routing."""
    E, k, H, I = 24, 4, 256, 144
    g = _gen(T + 5)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    gu = (torch.randn(E, 2 * I, H, generator=g) * 0.1).to(torch.bfloat16).cuda()
    dn = (torch.randn(E, H, I, generator=g) * 0.1).to(torch.bfloat16).cuda()
    ids, wts, off, lst = nv.moe_route_topk(torch.randn(T, E, generator=g).cuda(), k)
    if fp8:
        gq, gs = nv.fp8_quantize_block128(gu, 128)
        dq, ds = nv.fp8_quantize_block128(dn, 128)
        xq, xs = nv.fp8_quantize_block128(x)
        ab = nv.moe_grouped_gemm_fp8(xq, xs, gq, gs, off, lst, k, gather=True, out_dtype=torch.float32)
    else:
        ab = nv.moe_grouped_gemm_bf16(x, gu, off, lst, k, gather=True, out_dtype=torch.float32)
    h = (torch.nn.functional.silu(ab[:, :I]) * ab[:, I:]).to(torch.bfloat16)
    if fp8:
        hq, hs = nv.fp8_quantize_block128(h)
        rows = nv.moe_grouped_gemm_fp8(hq, hs, dq, ds, off, lst, k, scatter=True, out_dtype=torch.float32)
    else:
        rows = nv.moe_grouped_gemm_bf16(h, dn, off, lst, k, scatter=True, out_dtype=torch.float32)
    y = (rows.view(T, k, H) * wts[:, :, None]).sum(1)

    xd, gd, dd = ref.f64(x), ref.f64(gu), ref.f64(dn)
    if fp8:
        xd = ref.f64(xq) * ref.spread(ref.f64(xs), 1, T, H)
        gd = ref.f64(gq) * ref.spread(ref.f64(gs), 128, 2 * I, H)
        dd = ref.f64(dq) * ref.spread(ref.f64(ds), 128, H, I)
    idn, wn = ids.cpu().numpy(), ref.f64(wts)
    hg = ref.f64(h)
    hd = ref.f64(hq) * ref.spread(ref.f64(hs), 1, 0, I) if fp8 else hg
    place = np.argsort(lst.cpu().numpy())        # list position of every entry
    for t in range(T):
        total, slack = np.zeros(H), np.zeros(H)
        for j in range(k):
            e = idn[t, j]
            p = place[t * k + j]
            ab_w, S = gd[e] @ xd[t], np.abs(gd[e]) @ np.abs(xd[t])
            b = ref.bound(ab_w, S, H, False, fp8)
            z, u = ab_w[:I], ab_w[I:]
            sig = 1 / (1 + np.exp(-z))
            # |d silu| <= 1.1 |dz|; fp32 silu and product within 2^-20; one rounding of h to bf16
            want_h = z * sig * u
            tol = 1.1 * b[:I] * (np.abs(u) + b[I:]) + np.abs(z * sig) * b[I:] + (2.0 ** -8 + 2.0 ** -20) * np.abs(want_h)
            assert np.all(np.abs(hg[p] - want_h) <= 1.01 * tol + 1e-30)
            r, Sr = dd[e] @ hd[p], np.abs(dd[e]) @ np.abs(hd[p])
            total += wn[t, j] * r
            slack += wn[t, j] * (ref.bound(r, Sr, I, False, fp8) + 2.0 ** -20 * Sr)
        assert np.all(np.abs(ref.f64(y)[t] - total) <= slack + 1e-30)


@pytest.mark.parametrize("T", [1, 8, 40, 300])
def test_scales_at_the_ends_of_their_range(nv, T):
    """The contract beyond the normal range of the scales' product: y = fl(fl(xs ws) * sum) for one block."""
    g = _gen(T)
    N, K = 200, 128
    x, w = _small(g, T, K), _small(g, N, K)
    x[:, 64:] = 0
    w[5, :64] = 0                                                # sums of zero, the operands are not
    part = (x.double() @ w.double().t()).numpy().astype(np.float32)
    assert (part == 0).any()
    for ex, ew in ((-60, -66), (-70, -70), (60, 67), (60, 90), (100, -100)):
        xs = torch.full((T, 1), (1 + 2.0 ** -9) * 2.0 ** ex)
        ws = torch.full((2, 1), (1 + 2.0 ** -20) * 2.0 ** ew)
        y = nv.fp8_gemm_block128(x.to(F8).cuda(), xs.cuda(), w.to(F8).cuda(), ws.cuda(), out_dtype=torch.float32)
        with np.errstate(all="ignore"):
            want = part * (np.float32(xs[0, 0].item()) * np.float32(ws[0, 0].item()))
        assert want.dtype == np.float32
        assert np.array_equal(y.cpu().numpy(), want, equal_nan=True), (ex, ew)


@pytest.mark.parametrize("K", [16, 32, 48, 64, 80, 96, 112])
@pytest.mark.parametrize("rows", ["gather", "scatter", "list"])
@pytest.mark.parametrize("T", [2, 200])
def test_grouped_fp8_widths_below_a_block(nv, T, rows, K):
    """Rows of 16 to 112 bytes: one partial block, narrower than a step of the tiles."""
    a, xd, wd, off, lst, R = _grouped_case(T, 2, 5, 150, K, "skew", rows, True, K + T)
    want, _, written = _want(a, xd, wd, off, lst, R)
    assert written.all()
    _check_exact(_call(nv, a, out_dtype=torch.float32), want)
