"""nvfp4_gemm_w4a4 and moe_grouped_gemm_nvfp4 on the GPU, against plain 64-bit forms (rows_ref, products_ref).

Most cases use codes up to 2 and scales that are powers of two: with K <= 4096 every product is a multiple of 2^-4 and
every sum is below 2^17, so fp32 outputs are known to the bit and bf16 outputs are their one rounding.
"""
import numpy as np
import pytest
import torch

import products_ref as pref
import rows_ref as ref
from test_gpu_products import _check_exact, _counts, _run_twice

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _small_codes(g, *shape):
    """Packed codes 0, .5, 1, 1.5, 2 of both signs, two a byte."""
    c = torch.randint(0, 5, shape, generator=g) | (torch.randint(0, 2, shape, generator=g) << 3)
    return (c[..., 0::2] | (c[..., 1::2] << 4)).to(torch.uint8)


def _small_scales(g, *shape):
    """E4M3 codes of 1/2, 1 and 2."""
    return (torch.randint(6, 9, shape, generator=g) << 3).to(torch.uint8)


def _pow2(g, *shape):
    return torch.pow(2.0, torch.randint(-8, 9, shape, generator=g).float())


def _dense(T, N, K, seed):
    g = _gen(seed)
    x, xs, xr = _small_codes(g, T, K), _small_scales(g, T, K // 16), _pow2(g, T)
    w, ws, wt = _small_codes(g, N, K), _small_scales(g, N, K // 16), _pow2(g, 1)
    xd = ref.values(x.numpy(), xs.numpy()) * ref.f64(xr)[:, None]
    wd = ref.values(w.numpy(), ws.numpy()) * float(wt)
    return (x.cuda(), xs.cuda(), xr.cuda()), (w.cuda(), ws.cuda(), wt.cuda()), xd, wd


def _weight(nv, w, N, K):
    return nv.NVFP4Weight(*w, N, K, nv.SCALE_E4M3)


DENSE = [(1, 1, 32), (1, 130, 32), (1, 128, 2048), (2, 513, 2016), (3, 8192, 2048), (7, 300, 1056), (8, 256, 4096),
         (9, 40, 64), (16, 1000, 96), (17, 2048, 512), (64, 5003, 2048), (65, 129, 288), (128, 512, 1024), (129, 257, 544),
         (200, 2600, 512), (256, 256, 256), (257, 255, 224), (300, 513, 4096), (700, 1030, 160), (2000, 2600, 512),
         (64, 8192, 4096), (500, 2048, 8192), (256, 1500, 16384), (40, 8000, 4064), (250, 1500, 16352)]   # pairs share K


@pytest.mark.parametrize("T,N,K", DENSE)
def test_dense_exact(nv, T, N, K):
    x, w, xd, wd = _dense(T, N, K, T + N + K)
    want = xd @ wd.T
    wk = nv.Workspace(256)
    for dt in (F32, BF16):
        _check_exact(nv.nvfp4_gemm_w4a4(*x, _weight(nv, w, N, K), out_dtype=dt, ws=wk), want, dt)
    assert wk.status() == nv.NVFP4_OK


@pytest.mark.parametrize("rows", [1, 63, 64, 65, 127, 128, 129, 192, 193, 255, 256, 257, 400])
@pytest.mark.parametrize("N,K", [(260, 2048), (1030, 1056), (5000, 512), (300, 160)])
def test_dense_rows_around_every_tile(nv, rows, N, K):
    x, w, xd, wd = _dense(rows, N, K, rows + N)
    _check_exact(nv.nvfp4_gemm_w4a4(*x, _weight(nv, w, N, K), out_dtype=F32), xd @ wd.T)


@pytest.mark.parametrize("K", [32, 64, 96, 128, 160, 192, 224, 256, 288, 320, 480, 512, 544, 768, 800, 1024, 1280])
@pytest.mark.parametrize("T", [2, 90])
def test_dense_every_end_of_k(nv, T, K):
    """Block scales whose rows start at every alignment that K allows, and a last step that K fills in part: what lies
    behind the end of K is neither operand (the bytes there are the next row's, and NaN behind the last one)."""
    N = 150
    x, w, xd, wd = _dense(T, N, K, K)

    def guarded(t):         # the same values in front of NaN scales and codes of 6
        buf = torch.full((t.numel() + 4096,), 0x7F, dtype=torch.uint8, device="cuda")
        buf[:t.numel()] = t.reshape(-1)
        return buf[:t.numel()].view(t.shape)

    x = (guarded(x[0]), guarded(x[1]), x[2])
    w = (guarded(w[0]), guarded(w[1]), w[2])
    _check_exact(nv.nvfp4_gemm_w4a4(*x, _weight(nv, w, N, K), out_dtype=F32), xd @ wd.T)


def test_every_code_and_scale(nv):
    """One product at a time: all 16 codes of x against all of w, and every block scale of either."""
    K = 32
    codes = torch.arange(16, dtype=torch.uint8)
    x = torch.zeros(16, K // 2, dtype=torch.uint8)
    x[:, 0] = codes                                  # element 0
    x[:, 8] = codes << 4                             # element 17
    w = x.clone()
    one = torch.full((16, 2), 0x38, dtype=torch.uint8)
    r, t = torch.ones(16).cuda(), torch.ones(1).cuda()
    v = ref.code_values(codes.numpy())
    y = nv.nvfp4_gemm_w4a4(x.cuda(), one.cuda(), r, _weight(nv, (w.cuda(), one.cuda(), t), 16, K), out_dtype=F32)
    _check_exact(y, 2 * np.outer(v, v))
    s = torch.arange(127, dtype=torch.uint8)
    x = torch.full((127, K // 2), 0x22, dtype=torch.uint8)       # all 1
    xs = torch.stack([s, torch.zeros_like(s)], 1)
    ws = torch.stack([s.flip(0), torch.full_like(s, 0x38)], 1)
    y = nv.nvfp4_gemm_w4a4(x.cuda(), xs.cuda(), torch.ones(127).cuda(), _weight(nv, (x.cuda(), ws.cuda(), t), 127, K), out_dtype=F32)
    _check_exact(y, 16 * np.outer(ref.E4M3[s.numpy()], ref.E4M3[s.numpy()[::-1]]))


def test_fp32_scales_and_rows_that_are_not_finite(nv):
    """Row scales over the whole range times the tensor scale; a NaN row scale stays in its row, a NaN block scale of
    x in its row, of W in its column."""
    T, N, K = 70, 140, 288
    x, w, xd, wd = _dense(T, N, K, 5)
    part = ref.values(x[0].cpu().numpy(), x[1].cpu().numpy()) @ ref.values(w[0].cpu().numpy(), w[1].cpu().numpy()).T
    for er, et in ((-60, -60), (60, 60), (-120, 20), (100, -100)):
        xr = torch.full((T,), (1 + 2.0 ** -9) * 2.0 ** er)
        wt = torch.full((1,), (1 + 2.0 ** -20) * 2.0 ** et)
        y = nv.nvfp4_gemm_w4a4(x[0], x[1], xr.cuda(), _weight(nv, (w[0], w[1], wt.cuda()), N, K), out_dtype=F32)
        with np.errstate(all="ignore"):
            want = part.astype(np.float32) * (np.float32(xr[0].item()) * np.float32(wt[0].item()))
        assert np.array_equal(y.cpu().numpy(), want), (er, et)
    xr, xs, ws = x[2].clone(), x[1].clone(), w[1].clone()
    xr[3], xs[66, 17], ws[131, 0] = float("nan"), 0x7F, 0x7F
    y = nv.nvfp4_gemm_w4a4(x[0], xs, xr, _weight(nv, (w[0], ws, w[2]), N, K), out_dtype=F32)
    want = xd @ wd.T
    want[[3, 66]], want[:, 131] = np.nan, np.nan
    _check_exact(y, want)


def _real(g, nv, E, N, K, parts):
    L = []
    for _ in range(E * parts):
        L.append(nv.nvfp4_pack((torch.randn(N // parts, K, generator=g) * 0.02 * (1 + len(L) % 3)).cuda()))
    w = torch.stack([p.packed for p in L]).view(E, N, K // 2)
    ws = torch.stack([p.scales for p in L]).view(E, N, K // 16)
    return w, ws, torch.cat([p.tensor_scale for p in L]).view(E, parts)


@pytest.mark.parametrize("T,N,K", [(1, 512, 2048), (50, 300, 2016), (300, 1030, 1024), (1, 2000, 4096)])
def test_dense_real_values(nv, T, N, K):
    g = _gen(T + N)
    x = nv.nvfp4_quantize_rows(torch.randn(T, K, generator=g).to(BF16).cuda())
    w, ws, wt = (t[0] for t in _real(g, nv, 1, N, K, 1))
    xd = ref.values(x[0].cpu().numpy(), x[1].cpu().numpy()) * ref.f64(x[2])[:, None]
    wd = ref.values(w.cpu().numpy(), ws.cpu().numpy()) * float(wt)
    want, S = xd @ wd.T, np.abs(xd) @ np.abs(wd).T
    for dt in (F32, BF16):
        y = nv.nvfp4_gemm_w4a4(*x, nv.NVFP4Weight(w, ws, wt, N, K, nv.SCALE_E4M3), out_dtype=dt)
        err = np.abs(ref.f64(y) - want)
        # products_ref.bound, and the roundings of the two scales' product and of its use
        assert np.all(err <= pref.bound(want, S, K, dt == BF16, False) + 3 * 2.0 ** -24 * S), float((err / S).max())


# ---------------------------------------------------------------- grouped

def _case(T, k, E, N, K, kind, rows, parts, seed):
    g = _gen(seed)
    R = T * k
    off = _counts(kind, R, E, g)
    lst = torch.randperm(R, generator=g).to(torch.int32)
    xrows = T if rows == "gather" else R
    x, xs, xr = _small_codes(g, xrows, K), _small_scales(g, xrows, K // 16), _pow2(g, xrows)
    w, ws, wt = _small_codes(g, E, N, K), _small_scales(g, E, N, K // 16), _pow2(g, E, parts)
    xd = ref.values(x.numpy(), xs.numpy()) * ref.f64(xr)[:, None]
    wd = ref.values(w.numpy(), ws.numpy()) * np.repeat(ref.f64(wt), N // parts, axis=1)[:, :, None]
    a = dict(x=x.cuda(), x_scales=xs.cuda(), x_row_scales=xr.cuda(), w=w.cuda(), w_scales=ws.cuda(), w_tscale=wt.cuda(),
             offsets=off.cuda(), k=k, gather=rows == "gather", scatter=rows == "scatter",
             token_list=lst.cuda() if rows != "list" else None)
    return a, xd, wd, off, lst, R


def _want(a, xd, wd, off, lst, R):
    return pref.grouped(xd, wd, off.numpy(), lst.numpy(), R, a["k"], a["gather"], a["scatter"])


CASES = [  # T, k, E, N, K, kind, parts
    (1, 1, 1, 1, 32, "one", 1), (1, 8, 256, 128, 256, "even", 2), (1, 8, 40, 130, 2048, "skew", 2), (3, 2, 5, 17, 64, "holes", 1),
    (5, 8, 64, 300, 288, "skew", 3), (64, 4, 30, 129, 512, "skew", 1), (40, 8, 3, 200, 160, "even", 2),
    (300, 2, 4, 260, 416, "one", 2), (257, 1, 2, 127, 640, "even", 1), (200, 8, 17, 386, 1056, "skew", 2),
    (1024, 1, 256, 64, 128, "skew", 2), (33, 1, 33, 136, 4096, "even", 136), (90, 8, 6, 1024, 2048, "skew", 2),
    (700, 1, 2, 261, 1984, "one", 1), (450, 2, 3, 130, 1920, "even", 1), (600, 1, 2, 135, 2016, "skew", 1),
    (300, 2, 4, 130, 256, "skew", 1), (40, 4, 9, 70, 768, "skew", 1), (900, 1, 2, 200, 512, "skew", 1),
]


@pytest.mark.parametrize("rows", ["gather", "scatter", "list"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_grouped_exact(nv, case, rows):
    T, k, E, N, K, kind, parts = case
    a, xd, wd, off, lst, R = _case(T, k, E, N, K, kind, rows, parts, sum(case[:5]))
    want, _, written = _want(a, xd, wd, off, lst, R)
    assert written.all()
    wk = nv.Workspace(256)
    for dt in (F32, BF16):
        _check_exact(nv.moe_grouped_gemm_nvfp4(**a, out_dtype=dt, ws=wk), want, dt)
    assert wk.status() == nv.NVFP4_OK
    if parts == 1:
        a["w_tscale"] = a["w_tscale"][:, 0].contiguous()
        _check_exact(nv.moe_grouped_gemm_nvfp4(**a, out_dtype=F32), want)


@pytest.mark.parametrize("T", [2, 150])
def test_grouped_both_maps_and_unwritten_rows(nv, T):
    a, xd, wd, off, lst, R = _case(T, 4, 6, 140, 288, "even", "gather", 2, 9)
    a["scatter"] = True
    off = off.clone()
    off[0], off[-1] = 1, R - 2
    a["offsets"] = off.cuda()
    want, _, written = _want(a, xd, wd, off, lst, R)
    assert 0 < written.sum() < R - 1
    y = torch.full((R, 140), -77.0, device="cuda")
    assert nv.moe_grouped_gemm_nvfp4(**a, y=y) is y
    want[~written] = -77.0
    _check_exact(y, want)


@pytest.mark.parametrize("T,K", [(3, 160), (180, 160), (180, 2048)])
def test_grouped_bad_offsets_and_entries_stay_in_bounds(nv, T, K):
    for rows in ("gather", "scatter"):
        a, xd, wd, off, lst, R = _case(T, 2, 5, 130, K, "even", rows, 1, 21)
        off = torch.tensor([-5, 2, 1, 3, R, R + 100], dtype=torch.int32)
        lst[2], lst[0], lst[R - 1] = -1, R, 2 ** 31 - 1
        a["offsets"], a["token_list"] = off.cuda(), lst.cuda()
        y = torch.full((R, 130), -77.0, device="cuda")
        nv.moe_grouped_gemm_nvfp4(**a, y=y)
        torch.cuda.synchronize()
        want, _, written = pref.grouped(xd, wd, np.array([3, 3, 3, 3, R, R]), lst.numpy(), R, 2, rows == "gather", rows == "scatter")
        got = ref.f64(y)
        assert np.array_equal(got[written], want[written])
        if rows == "scatter":
            touched = {int(v) for v in lst if 0 <= int(v) < R}
            for r in set(range(R)) - touched:
                assert (got[r] == -77.0).all()


@pytest.mark.parametrize("K", [160, 1024])
def test_grouped_groups_that_all_overlap(nv, K):
    a, xd, wd, off, lst, R = _case(130, 2, 40, 130, K, "even", "list", 2, 3)
    bad = torch.tensor([0, R] * 20 + [0], dtype=torch.int32).cuda()
    y = torch.full((R + 1, 130), -77.0, device="cuda")
    nv.moe_grouped_gemm_nvfp4(**dict(a, offsets=bad), y=y[:R])
    assert (y[R] == -77.0).all()
    _check_exact(nv.moe_grouped_gemm_nvfp4(**a, out_dtype=F32), _want(a, xd, wd, off, lst, R)[0])


@pytest.mark.parametrize("N", [1, 3, 33, 250, 255, 257, 1022])
def test_grouped_output_widths(nv, N):
    a, xd, wd, off, lst, R = _case(60, 2, 3, N, 160, "skew", "scatter", 1, N)
    want = _want(a, xd, wd, off, lst, R)[0]
    for dt in (BF16, F32):
        buf = torch.full((R * N + 64,), -77.0, dtype=dt, device="cuda")
        nv.moe_grouped_gemm_nvfp4(**a, y=buf[:R * N].view(R, N))
        _check_exact(buf[:R * N].view(R, N), want, dt)
        assert (buf[R * N:] == -77.0).all()


@pytest.mark.parametrize("rows", ["gather", "scatter", "list"])
@pytest.mark.parametrize("T", [2, 90])
def test_grouped_neighbours_do_not_leak(nv, T, rows):
    """NaN block scales of experts without rows, and of rows of x that no position reads, stay there."""
    E, N, K = 9, 130, 288
    a, xd, wd, off, lst, R = _case(T, 4, E, N, K, "holes", rows, 2, 44)
    last = int(off[-1]) - 3
    off = torch.minimum(off, torch.tensor(last, dtype=torch.int32))
    a["offsets"] = off.cuda()
    empty = (off[1:] == off[:-1]).nonzero().flatten()
    a["w_scales"][empty.cuda()] = 0x7F
    a["w_tscale"][empty.cuda()] = float("nan")
    used = {int(e) // 4 for e in lst[:last]} if rows == "gather" else set(range(last))
    idle = torch.tensor([r for r in range(a["x"].shape[0]) if r not in used], dtype=torch.long).cuda()
    a["x_scales"][idle] = 0x7F
    a["x_row_scales"][idle] = float("nan")
    want, _, written = _want(a, xd, wd, off, lst, R)
    y = torch.full((R, N), -77.0, device="cuda")
    nv.moe_grouped_gemm_nvfp4(**a, y=y)
    want[~written] = -77.0
    _check_exact(y, want)


@pytest.mark.parametrize("T", [1, 100])
def test_grouped_graph_streams_and_repeats(nv, T):
    a, xd, wd, off, lst, R = _case(T, 8, 20, 260, 544, "skew", "gather", 2, 33)
    want = _want(a, xd, wd, off, lst, R)[0]
    y = nv.moe_grouped_gemm_nvfp4(**a, out_dtype=F32)
    _check_exact(y, want)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    y2 = nv.moe_grouped_gemm_nvfp4(**a, out_dtype=F32, stream=st)
    st.synchronize()
    assert torch.equal(y, y2)
    y3 = torch.zeros_like(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nv.moe_grouped_gemm_nvfp4(**a, y=y3)
    off2 = torch.zeros_like(off)
    off2[-1] = R
    a["offsets"].copy_(off2)
    a["token_list"].copy_(lst.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    _check_exact(y3, _want(a, xd, wd, off2, lst.flip(0), R)[0])


def test_two_streams_at_once(nv):
    cases = [_case(T, 4, 20, 520, 1056, "skew", rows, 2, T) for T in (2, 200) for rows in ("gather", "list")]
    wants = [_want(*c) for c in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = [nv.moe_grouped_gemm_nvfp4(**cases[i % 4][0], out_dtype=F32, stream=streams[(i // 2) % 2]) for i in range(12)]
    torch.cuda.synchronize()
    for i, y in enumerate(outs):
        _check_exact(y, wants[i % 4][0])


def test_past_32_bits(nv):
    """2.3e9 outputs, and 2^33 weight elements: the last rows and the last expert are where they should be."""
    g = torch.Generator(device="cuda").manual_seed(6)

    def codes(*shape):
        b = torch.randint(0, 3, shape, generator=g, device="cuda", dtype=torch.uint8)
        return b | (torch.randint(0, 3, shape, generator=g, device="cuda", dtype=torch.uint8) << 4)

    def val(p):
        return torch.stack([p & 15, p >> 4], -1).flatten(-2).float() * 0.5

    def check(x, w, off, rows):
        (R, half), (E, N, _) = x.shape, w.shape
        K = 2 * half
        s = lambda *shape: torch.full(shape, 0x38, dtype=torch.uint8, device="cuda")  # noqa: E731
        y = nv.moe_grouped_gemm_nvfp4(x, s(R, K // 16), torch.ones(R, device="cuda"), w, s(E, N, K // 16),
                                      torch.ones(E, device="cuda"), off)
        for r in rows:
            e = int((off[1:] <= r).sum())
            assert torch.equal(y[r], (val(w[e]) @ val(x[r])).to(BF16)), r

    R = 280000
    off = torch.tensor([0, 100, R], dtype=torch.int32, device="cuda")
    check(codes(R, 32), codes(2, 8200, 32), off, (0, 99, 100, 262143, R - 1))
    E, N, K = 128, 8192, 8192
    w = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda")
    for e in range(E):
        w[e] = codes(N, K // 2)
    for R in (4, 70):
        off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        off[1:] = R // 2
        off[-1] = R
        check(codes(R, K // 2), w, off, (0, R // 2 - 1, R // 2, R - 1))


def test_empty_and_refusals(nv):
    x, w, xd, wd = _dense(4, 64, 96, 1)
    W = _weight(nv, w, 64, 96)
    assert nv.nvfp4_gemm_w4a4(x[0][:0], x[1][:0], x[2][:0], W).shape == (0, 64)
    # fp32 scales need 4-byte alignment only
    xr = torch.cat([x[2][:1], x[2]])
    _check_exact(nv.nvfp4_gemm_w4a4(x[0], x[1], xr[1:], W, out_dtype=F32), xd @ wd.T)
    for bad in (dict(x_scales=x[1][:, :5]), dict(x_row_scales=x[2][:3]), dict(x=x[0].view(torch.int8)),
                dict(out_dtype=torch.float16), dict(W=nv.NVFP4Weight(*w, 64, 96, nv.SCALE_UE8M0)),
                dict(W=nv.NVFP4Weight(w[0], w[1], w[2], 64, 64, nv.SCALE_E4M3)), dict(x_scales=x[1].t().contiguous().t())):
        with pytest.raises(nv.NVFP4Error):
            nv.nvfp4_gemm_w4a4(**dict(dict(x=x[0], x_scales=x[1], x_row_scales=x[2], W=W), **bad))
    a = _case(4, 2, 3, 20, 64, "even", "gather", 2, 2)[0]
    for bad in (dict(w_tscale=a["w_tscale"][:, :1]), dict(w_tscale=torch.ones(3, 3, device="cuda")), dict(token_list=None),
                dict(offsets=a["offsets"].long()), dict(w=a["w"][:2]), dict(k=0)):
        with pytest.raises(nv.NVFP4Error):
            nv.moe_grouped_gemm_nvfp4(**dict(a, **bad))


# ---------------------------------------------------------------- waits

@pytest.mark.parametrize("rows", ["list", "gather", "scatter"])
@pytest.mark.parametrize("T,N,K", [(2000, 2600, 512), (2000, 2600, 544), (64, 6000, 2048), (128, 513, 4096), (300, 300, 1056),
                                   (64, 8192, 4096), (40, 8000, 4064), (128, 513, 4064)],
                         ids=["one_pair", "one_pair_odd", "few_tiles", "four_pairs", "odd", "two_pairs", "two_pairs_odd",
                              "four_pairs_odd"])
def test_a_wait_that_runs_out_is_reported(nv, T, N, K, rows):
    """A limit of 1 ns is over at the first poll that fails, and the first operands take a round trip to memory: the
    status and the NaN are always there, and the next call is exact again."""
    a, xd, wd, off, lst, R = _case(T, 1, 1, N, K, "one", rows, 1, T)
    want = _want(a, xd, wd, off, lst, R)[0]
    ws = nv.Workspace(256)
    for dtype in (F32, BF16):
        buf = torch.zeros(R * N + 64, dtype=dtype, device="cuda")
        y = buf[:R * N].view(R, N)
        try:
            nv.set_device_wait_limit(1)
            nv.moe_grouped_gemm_nvfp4(**a, y=y, ws=ws)
            torch.cuda.synchronize()
            assert ws.status(clear=True) == nv.NVFP4_ERR_DEVICE_TIMEOUT
            assert torch.isnan(y).any() and not buf[R * N:].any()
        finally:
            nv.set_device_wait_limit(0)
        nv.moe_grouped_gemm_nvfp4(**a, y=y, ws=ws)
        assert ws.status() == nv.NVFP4_OK
        _check_exact(y, want, dtype)


@pytest.mark.parametrize("T,N,K,rows", [(300, 1030, 4096, "list"), (300, 1030, 4064, "list"), (700, 600, 2048, "gather"),
                                        (700, 600, 2080, "gather"), (100, 513, 8192, "list")])
def test_scales_that_change_from_call_to_call(nv, T, N, K, rows):
    """The same buffers with other block scales, call behind call: both CTAs of a pair multiply by this call's."""
    a, xd, wd, off, lst, R = _case(T, 1, 1, N, K, "one", rows, 1, T)
    want = torch.from_numpy(_want(a, xd, wd, off, lst, R)[0]).float().cuda()
    xs, ws = a["x_scales"].clone(), a["w_scales"].clone()
    ys = [torch.zeros(R, N, device="cuda") for _ in range(12)]
    for i, y in enumerate(ys):
        for t, s, step in ((a["x_scales"], xs, 8 * (i % 4)), (a["w_scales"], ws, 8 * (i // 4))):      # codes of twice the scale
            t.copy_(s)
            t.add_(step)
        nv.moe_grouped_gemm_nvfp4(**a, y=y)
    for i, y in enumerate(ys):
        assert torch.equal(y, want * 2.0 ** (i % 4 + i // 4))


@pytest.mark.parametrize("limit", [200, 2000, 20000])
def test_waits_that_may_run_out(nv, limit):
    """Limits around what the waits take: the status and the NaN go together, whatever has finished is right, and
    the next call is exact."""
    for T, N, K, rows in ((700, 1030, 2048, "gather"), (64, 6000, 2048, "list"), (100, 513, 4096, "scatter")):
        a, xd, wd, off, lst, R = _case(T, 1, 3, N, K, "skew", rows, 1, T)
        want = torch.from_numpy(_want(a, xd, wd, off, lst, R)[0]).float().cuda()
        ws = nv.Workspace(256)
        y = torch.zeros(R, N, device="cuda")
        try:
            nv.set_device_wait_limit(limit)
            for _ in range(3):
                nv.moe_grouped_gemm_nvfp4(**a, y=y, ws=ws)
                torch.cuda.synchronize()
                code = ws.status(clear=True)
                bad = y.isnan()
                assert code == (nv.NVFP4_ERR_DEVICE_TIMEOUT if bad.any() else nv.NVFP4_OK) or code == nv.NVFP4_ERR_DEVICE_TIMEOUT
                assert torch.equal(y[~bad], want[~bad])
        finally:
            nv.set_device_wait_limit(0)
        nv.moe_grouped_gemm_nvfp4(**a, y=y, ws=ws)
        assert ws.status() == nv.NVFP4_OK and torch.equal(y, want)


_FIRST_IN_CAPTURE = """
import sys
sys.path[:0] = [%r, %r]
import torch
import nvfp4_w4a16_moe_gb300 as nv
T, N, K = %d, 300, 2048
x = torch.ones(T, K, dtype=torch.bfloat16, device="cuda")
w = torch.zeros(K, dtype=torch.bfloat16, device="cuda")
W = nv.nvfp4_pack(torch.ones(N, K, device="cuda"))
gu = torch.ones(T, 2 * K, dtype=torch.bfloat16, device="cuda")
lst = torch.arange(T, dtype=torch.int32, device="cuda").flip(0).contiguous()
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    h, q = nv.rmsnorm_residual(x, w, 0.0, kind=nv.ROWS_NVFP4)
    y = nv.nvfp4_gemm_w4a4(*q, W)
    z = nv.nvfp4_gemm_w4a4(*nv.nvfp4_quantize_rows(x), W, out_dtype=torch.float32)
    s = nv.moe_swiglu(gu)
    r, p = nv.moe_permute(z, lst, 1)
    c = nv.moe_combine(r, 1, None, p, out_dtype=torch.float32)
g.replay()
torch.cuda.synchronize()
# W is 6 * 448 * fl(1 / 2688): 1 within its roundings. A row of ones has row scale 2^-11 (the power of two above 1 / 2688),
# block scale 352 (of 320 and 352 the nearer to 2^11 / 6 = 341.3) and codes 6 (2^11 / 352 = 5.8): 6 * 352 / 2^11 = 33 / 32.
want = K * 33 / 32
assert (y.float() - want).abs().max() <= want * 2.0 ** -8 and (z - want).abs().max() <= want * 2.0 ** -20
assert torch.equal(c, z) and torch.equal(r, z.flip(0))
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


# ---------------------------------------------------------------- together

def test_chains_over_reused_buffers(nv):
    """Norm, quantise, multiply, SwiGLU, multiply, combine in the same buffers, few and many rows in turn: a call that
    started before the one ahead of it was done, or read a stale line, would differ from the slow run."""
    g = _gen(8)
    E, H, I, k = 6, 256, 160, 2
    gu, dn = _real(g, nv, E, 2 * I, H, 2), _real(g, nv, E, H, I, 1)
    nw = (torch.randn(H, generator=g) * 0.2).to(BF16).cuda()
    sizes = (5, 400)
    hs = [torch.randn(T, H, generator=g).to(BF16).cuda() for T in sizes]
    routes = [nv.moe_route_topk(torch.randn(T, E, generator=g).cuda(), k) for T in sizes]
    e = lambda *s, dtype=BF16: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    rows4 = lambda R, K: (e(R, K // 2, dtype=torch.uint8), e(R, K // 16, dtype=torch.uint8), e(R, dtype=F32))  # noqa: E731
    bufs = [(e(T, H), rows4(T, H), e(T * k, 2 * I), rows4(T * k, I), e(T * k, H)) for T in sizes]

    def step(i, wait):
        b = i % 2
        (h, xq, ab, aq, back), (ids, w, off, lst) = bufs[b], routes[b]
        h.copy_(hs[b] * (1 + i % 3))
        for _ in range(3):
            wait()
            nv.rmsnorm_residual(h, nw, kind=nv.ROWS_NVFP4, out=xq)
            wait()
            nv.moe_grouped_gemm_nvfp4(*xq, *gu, off, lst, k, gather=True, y=ab)
            wait()
            nv.moe_swiglu(ab, nv.ROWS_NVFP4, out=aq)
            wait()
            nv.moe_grouped_gemm_nvfp4(*aq, *dn, off, lst, k, scatter=True, y=back)
            wait()
            nv.moe_combine(back, k, w, add=h, y=h)
        wait()
        return h, xq[0], ab, aq[0], back

    fast, slow = _run_twice(step, 24)
    for p, q in zip(fast, slow):
        assert all(torch.equal(s, t) for s, t in zip(p, q))


@pytest.mark.parametrize("T", [1, 50, 300])
def test_a_layers_experts_on_4_bit_rows(nv, T):
    """The whole run on a MoELayer's own weights: norm into NVFP4 rows, gate/up, SwiGLU into NVFP4 rows, down,
    weighted sum with the residual. Each product is checked against 64 bits on the rows it was given, the sum on
    the rows that down wrote; the rows themselves by their own tests' rules."""
    E, k, H, I = 24, 4, 256, 160
    g = _gen(T + 5)
    L = nv.MoELayer.allocate(H, E, k, I, 0, device="cuda")
    for e in range(E):
        L.pack_expert(e, *((torch.randn(*s, generator=g) * 0.1).cuda() for s in ((I, H), (I, H), (H, I))))
    h, d = (torch.randn(T, H, generator=g).to(BF16) for _ in range(2))
    nw = (torch.randn(H, generator=g) * 0.2).to(BF16)
    ids, wts, off, lst = nv.moe_route_topk(torch.randn(T, E, generator=g).cuda(), k)
    h1, xq = nv.rmsnorm_residual(h.cuda(), nw.cuda(), 1e-6, delta=d.cuda(), kind=nv.ROWS_NVFP4)
    ab = nv.moe_grouped_gemm_nvfp4(*xq, L.gu_packed, L.gu_scales, L.gu_tscale, off, lst, k, gather=True, out_dtype=F32)
    aq = nv.moe_swiglu(ab, nv.ROWS_NVFP4)
    back = nv.moe_grouped_gemm_nvfp4(*aq, L.dn_packed, L.dn_scales, L.dn_tscale, off, lst, k, scatter=True, out_dtype=F32)
    out = nv.moe_combine(back, k, wts, add=h1)
    # the same through permuted rows and list order
    rows, pos = nv.moe_permute(torch.empty(T, 8, dtype=BF16, device="cuda").zero_(), lst, k)
    listed = nv.moe_grouped_gemm_nvfp4(*aq, L.dn_packed, L.dn_scales, L.dn_tscale, off, out_dtype=F32)
    assert torch.equal(nv.moe_combine(listed, k, wts, pos, add=h1), out)

    n = lambda t: t.cpu().numpy()  # noqa: E731
    want_h, x = ref.norm(ref.f64(h), ref.f64(d), ref.f64(nw), 1e-6)
    assert np.array_equal(ref.f64(h1), want_h)
    ref.check_nvfp4(*(n(t) for t in xq), x, ((64 + 37) / 2 + 8) * 2.0 ** -24)
    wd = ref.values(n(L.gu_packed), n(L.gu_scales)) * np.repeat(ref.f64(L.gu_tscale), I, axis=1)[:, :, None]
    want, S, _ = pref.grouped(ref.values(n(xq[0]), n(xq[1])) * ref.f64(xq[2])[:, None], wd, n(off), n(lst), T * k, k, True, False)
    got = ref.f64(ab)
    assert np.all(np.abs(got - want) <= pref.bound(want, S, H, False, False) + 3 * 2.0 ** -24 * S)
    err = (4 + 1.2 * np.abs(got[:, :I])) * 2.0 ** -23 + 3 * 2.0 ** -24
    ref.check_nvfp4(*(n(t) for t in aq), ref.silu_up(got), err)
    wd = ref.values(n(L.dn_packed), n(L.dn_scales)) * ref.f64(L.dn_tscale)[:, None, None]
    want, S, _ = pref.grouped(ref.values(n(aq[0]), n(aq[1])) * ref.f64(aq[2])[:, None], wd, n(off), n(lst), T * k, k, False, True)
    assert np.all(np.abs(ref.f64(back) - want) <= pref.bound(want, S, I, False, False) + 3 * 2.0 ** -24 * S)
    y, S = ref.combine(ref.f64(back), ref.f64(wts), None, want_h, T, k)
    err = (k + 2) * 2.0 ** -24 * S
    assert np.all(np.abs(ref.f64(out) - y) <= err + 2.0 ** -8 * (np.abs(y) + err))
