"""Checks of NVFP4 rows, their products, the norm, the SwiGLU and the sorted rows that need no GPU: the 64-bit forms
that the GPU tests compare with, the arithmetic that the kernels rest on, and the refusals of the C entry points and
of the Python calls (all before CUDA is touched)."""
import ctypes

import numpy as np
import pytest
import torch

import rows_ref as ref
from test_products_cpu import FAKE, Groups, Operand, _status, nv  # noqa: F401

U8, F32, BF16, I32, F8 = torch.uint8, torch.float32, torch.bfloat16, torch.int32, torch.float8_e4m3fn


class Rows(ctypes.Structure):           # nvfp4_rows of the C header
    _fields_ = [("kind", ctypes.c_int32), ("data", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("row_scales", ctypes.c_void_p)]


def test_python_packs_the_structures_like_c(nv):  # noqa: F811
    assert bytes(Rows(1, 2, 3, 4)) == nv._ROWS.pack(1, 2, 3, 4)
    assert bytes(nv.NVFP4WeightC(1, 2, 3, 4, 5, 0)) == nv._WEIGHT.pack(1, 2, 3, 4, 5, 0)


def test_reference_codes_are_the_oracles(orc):
    """The packer's definition with a row's power-of-two scale as the tensor scale gives the same codes."""
    g = torch.Generator().manual_seed(1)
    x = torch.randn(4, 64, generator=g).clamp(-3, 3).to(BF16)
    x[:, 3] = 5.25                                   # 5.25 / 2688 = 2^-9
    codes, e, s = ref.quantize_rows(ref.f64(x))
    for r in range(4):
        m = orc.pack(x[r:r + 1].float())
        assert float(s[r]) == float(np.asarray(m.tensor_scale).ravel()[0]) == 2.0 ** -9
        assert np.array_equal(np.asarray(m.packed).ravel(), ref.pack_codes(codes)[r])
        assert np.array_equal(np.asarray(m.scales).ravel(), e[r])


def test_reference_checks_accept_the_nearest_and_refuse_neighbours():
    x = np.random.default_rng(0).standard_normal((3, 64))
    codes, e, s = ref.quantize_rows(x)
    ref.check_nvfp4(ref.pack_codes(codes), e, s, x, 0.0)
    bad = codes.copy()
    bad[1, 5] ^= 1
    with pytest.raises(AssertionError):
        ref.check_nvfp4(ref.pack_codes(bad), e, s, x, 1e-6)
    with pytest.raises(AssertionError):
        ref.check_nvfp4(ref.pack_codes(codes), e, s * 2, x, 1e-6)


def test_quotients_of_bf16_stay_off_the_rounding_points():
    """What the quantiser's fp32 arithmetic rests on, for 8-bit significands m: v / e with an E4M3 e (significand 1 to
    15) is on a rounding point of E2M1 (odd numerator 1, 3, 5 or 7) or off it by 2^-8; b / 6 on one of E4M3 (odd, below
    32) or off it by 2^-13; a / 2688 a power of two or off it by 1 / 168."""
    m = np.arange(128, 256).astype(np.float64)
    near = lambda q, p: min((np.abs(q - p * 2.0 ** d) / (p * 2.0 ** d))[np.abs(q - p * 2.0 ** d) > 0].min() for d in range(-12, 13))  # noqa: E731
    assert min(near(m[:, None] / np.arange(1, 16)[None, :], p) for p in (1, 3, 5, 7)) >= 2.0 ** -8
    assert min(near(m / 6, p) for p in range(1, 32, 2)) >= 2.0 ** -13
    assert near(m / 2688, 1) >= 1 / 168 - 1e-12


def test_power_of_two_row_scale_by_bits():
    """The kernel's rule on the bits of fl32(a / 2688) is the smallest power of two at or above the real quotient, for
    every bf16 a."""
    bits = np.arange(1, 0x7F80, dtype=np.uint32) << 16
    a = bits.view(np.float32)
    q = (a / np.float32(2688.0)).view(np.uint32)
    s = np.maximum((q + np.uint32(0x7FFFFF)) & np.uint32(0x7F800000), np.uint32(0x00800000)).view(np.float32).astype(np.float64)
    a = a.astype(np.float64)
    assert np.all(s >= a / 2688) and np.all((s / 2 < a / 2688) | (s == 2.0 ** -126))
    assert np.array_equal(ref.row_scale(a[::97]), s[::97])


# ---------------------------------------------------------------- refusals

def test_quantize_and_dequantize_refusals(nv):  # noqa: F811
    call = lambda x=FAKE, R=4, K=64, p=FAKE, s=FAKE, r=FAKE: _status(nv, "nvfp4_quantize_rows", x, R, K, p, s, r, None)  # noqa: E731
    for kw in (dict(x=None), dict(p=None), dict(s=None), dict(r=None)):
        assert call(**kw) == nv.NVFP4_ERR_INVALID_ARG
    for kw in (dict(R=-1), dict(K=0), dict(K=16), dict(K=48), dict(K=32800), dict(K=-32)):
        assert call(**kw) == nv.NVFP4_ERR_UNSUPPORTED_SHAPE
    for kw in (dict(x=FAKE + 8), dict(p=FAKE + 8), dict(s=FAKE + 4), dict(r=FAKE + 2)):
        assert call(**kw) == nv.NVFP4_ERR_MISALIGNED
    back = lambda p=FAKE, s=FAKE, t=FAKE, n=1, R=4, K=64, y=FAKE, yt=0: _status(nv, "nvfp4_dequantize_rows", p, s, t, n, R, K, y, yt, None)  # noqa: E731
    for kw in (dict(p=None), dict(s=None), dict(t=None), dict(y=None), dict(yt=2)):
        assert back(**kw) == nv.NVFP4_ERR_INVALID_ARG
    for kw in (dict(n=0), dict(R=-1), dict(K=16), dict(K=40), dict(K=65568)):
        assert back(**kw) == nv.NVFP4_ERR_UNSUPPORTED_SHAPE
    for kw in (dict(p=FAKE + 8), dict(s=FAKE + 8), dict(t=FAKE + 2), dict(y=FAKE + 4)):
        assert back(**kw) == nv.NVFP4_ERR_MISALIGNED


@pytest.mark.parametrize("fn", ["rmsnorm_residual", "moe_swiglu"])
def test_row_op_refusals(nv, fn):  # noqa: F811
    def call(x=FAKE, delta=None, w=FAKE, eps=1e-6, R=4, K=64, h_out=None, kind=2, data=FAKE, s=FAKE, r=FAKE, null=False, gt=0):
        o = Rows(kind, data, s, r)
        p = None if null else ctypes.addressof(o)
        if fn == "moe_swiglu":
            return _status(nv, fn, x, gt, R, K, p, None)
        return _status(nv, fn, x, delta, w, eps, R, K, h_out, p, None)
    for kw in (dict(x=None), dict(null=True), dict(kind=3), dict(kind=-1), dict(data=None), dict(s=None), dict(r=None),
               dict(kind=1, s=None)):
        assert call(**kw) == nv.NVFP4_ERR_INVALID_ARG, kw
    for kw in (dict(R=-1), dict(K=0), dict(K=48), dict(K=24, kind=1), dict(K=12, kind=0), dict(K=32800), dict(K=32776, kind=0)):
        assert call(**kw) == nv.NVFP4_ERR_UNSUPPORTED_SHAPE, kw
    for kw in (dict(x=FAKE + 8), dict(data=FAKE + 8), dict(s=FAKE + 8), dict(r=FAKE + 1), dict(kind=1, s=FAKE + 2)):
        assert call(**kw) == nv.NVFP4_ERR_MISALIGNED, kw
    if fn == "moe_swiglu":
        assert call(gt=2) == nv.NVFP4_ERR_INVALID_ARG
    else:
        for kw in (dict(w=None), dict(delta=FAKE), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf"))):
            assert call(**kw) == nv.NVFP4_ERR_INVALID_ARG, kw
        for kw in (dict(delta=FAKE + 8, h_out=FAKE), dict(h_out=FAKE + 2), dict(w=FAKE + 4)):
            assert call(**kw) == nv.NVFP4_ERR_MISALIGNED, kw


def test_dense_product_refusals(nv):  # noqa: F811
    def call(x=FAKE, xs=FAKE, xr=FAKE, T=4, w=FAKE, ws=FAKE, wt=FAKE, N=16, K=64, kind=0, y=FAKE, yt=0, wk=None, wb=0, null=False):
        W = nv.NVFP4WeightC(w, ws, wt, N, K, kind)
        return _status(nv, "nvfp4_gemm_w4a4", x, xs, xr, T, None if null else ctypes.addressof(W), y, yt, wk, wb, None)
    for kw in (dict(x=None), dict(xs=None), dict(xr=None), dict(w=None), dict(ws=None), dict(wt=None), dict(y=None),
               dict(yt=2), dict(kind=4), dict(null=True)):
        assert call(**kw) == nv.NVFP4_ERR_INVALID_ARG, kw
    for kw in (dict(T=-1), dict(T=(1 << 20) + 1), dict(N=0), dict(N=(1 << 22) + 1), dict(K=0), dict(K=16), dict(K=48),
               dict(K=65568), dict(kind=1), dict(kind=2), dict(kind=3)):
        assert call(**kw) == nv.NVFP4_ERR_UNSUPPORTED_SHAPE, kw
    for kw in (dict(x=FAKE + 8), dict(w=FAKE + 4), dict(y=FAKE + 2), dict(xs=FAKE + 8), dict(ws=FAKE + 1), dict(xr=FAKE + 2),
               dict(wt=FAKE + 2), dict(wk=FAKE + 8, wb=256)):
        assert call(**kw) == nv.NVFP4_ERR_MISALIGNED, kw
    assert call(wk=FAKE, wb=128) == nv.NVFP4_ERR_WORKSPACE_TOO_SMALL


def test_grouped_product_refusals(nv):  # noqa: F811
    def call(R=8, E=4, k=2, gather=0, scatter=0, off=FAKE, lst=FAKE, x=FAKE, xs=FAKE, xr=FAKE, w=FAKE, ws=FAKE, wt=FAKE,
             parts=1, N=16, K=64, y=FAKE, yt=0, wk=None, wb=0, null=False):
        g = Groups(R, E, k, gather, scatter, off, lst)
        return _status(nv, "moe_grouped_gemm_nvfp4", None if null else ctypes.addressof(g), x, xs, xr, w, ws, wt, parts, N, K, y,
                       yt, wk, wb, None)
    for kw in (dict(null=True), dict(off=None), dict(lst=None, gather=1), dict(lst=None, scatter=1), dict(x=None), dict(xs=None),
               dict(xr=None), dict(w=None), dict(ws=None), dict(wt=None), dict(y=None), dict(yt=-1)):
        assert call(**kw) == nv.NVFP4_ERR_INVALID_ARG, kw
    for kw in (dict(R=-1), dict(R=(1 << 20) + 2), dict(E=0), dict(E=257), dict(k=0), dict(R=7, gather=1), dict(N=0), dict(K=0),
               dict(K=48), dict(parts=0), dict(parts=3), dict(parts=32), dict(E=256, N=1 << 23)):
        assert call(**kw) == nv.NVFP4_ERR_UNSUPPORTED_SHAPE, kw
    for kw in (dict(x=FAKE + 8), dict(w=FAKE + 8), dict(y=FAKE + 4), dict(off=FAKE + 2), dict(lst=FAKE + 1), dict(xs=FAKE + 4),
               dict(ws=FAKE + 8), dict(xr=FAKE + 1), dict(wt=FAKE + 1)):
        assert call(**kw) == nv.NVFP4_ERR_MISALIGNED, kw
    assert call(wk=FAKE, wb=16) == nv.NVFP4_ERR_WORKSPACE_TOO_SMALL


def test_sorted_rows_refusals(nv):  # noqa: F811
    permute = lambda x=FAKE, ty=0, lst=FAKE, T=4, k=2, N=8, rows=FAKE, pos=FAKE: _status(nv, "moe_permute", x, ty, lst, T, k, N, rows, pos, None)  # noqa: E731
    combine = lambda rows=FAKE, ty=0, w=FAKE, pos=FAKE, add=FAKE, T=4, k=2, N=8, y=FAKE, yt=0: _status(  # noqa: E731
        nv, "moe_combine", rows, ty, w, pos, add, T, k, N, y, yt, None)
    back = lambda dy=FAKE, dt=0, rows=FAKE, ty=0, w=FAKE, pos=FAKE, T=4, k=2, N=8, dr=FAKE, dw=FAKE: _status(  # noqa: E731
        nv, "moe_combine_backward", dy, dt, rows, ty, w, pos, T, k, N, dr, dw, None)
    for call in (permute, combine, back):
        for kw in (dict(T=-1), dict(k=0), dict(N=0), dict(N=(1 << 22) + 1), dict(T=1 << 20, k=2), dict(T=1 << 30, k=1 << 30)):
            assert call(**kw) == nv.NVFP4_ERR_UNSUPPORTED_SHAPE, kw
        for kw in (dict(ty=2), dict(ty=-1)):
            assert call(**kw) == nv.NVFP4_ERR_INVALID_ARG
    for call, null, off in ((permute, ("lst", "pos", "x"), ("x", "rows")), (combine, ("rows", "y"), ("rows", "add", "y")),
                            (back, ("dy", "rows"), ("dy", "rows", "dr"))):
        for name in null:
            assert call(**{name: None}) == nv.NVFP4_ERR_INVALID_ARG, name
        for name in off:
            assert call(**{name: FAKE + 8}) == nv.NVFP4_ERR_MISALIGNED, name
    assert combine(yt=2) == back(dt=2) == back(dr=None, dw=None) == nv.NVFP4_ERR_INVALID_ARG
    for bad in (permute(lst=FAKE + 2), permute(pos=FAKE + 2), combine(w=FAKE + 2), combine(pos=FAKE + 1), back(w=FAKE + 2),
                back(pos=FAKE + 2), back(dw=FAKE + 2)):
        assert bad == nv.NVFP4_ERR_MISALIGNED


def _refused(nv, call, status=None):  # noqa: F811
    with pytest.raises(nv.NVFP4Error) as e:
        call()
    assert status is None or e.value.status == status


def test_python_refuses_what_does_not_fit(nv):  # noqa: F811
    host = torch.zeros(4, 64, dtype=BF16)
    for call in (lambda: nv.nvfp4_quantize_rows(host), lambda: nv.rmsnorm_residual(host, host[0]), lambda: nv.moe_swiglu(host),
                 lambda: nv.moe_combine(host, 2), lambda: nv.moe_permute(host, torch.zeros(8, dtype=I32), 2),
                 lambda: nv.moe_combine_backward(host, host)):
        _refused(nv, call)
    x = Operand((4, 64), BF16)
    rows = lambda R, K: (Operand((R, K // 2), U8), Operand((R, K // 16), U8), Operand((R,), F32))  # noqa: E731
    for out in (rows(4, 32), rows(5, 64), rows(4, 64)[:2], Operand((4, 64), BF16)):
        _refused(nv, lambda: nv.nvfp4_quantize_rows(x, out=out), nv.NVFP4_ERR_INVALID_ARG)
    w = Operand((64,), BF16)
    for kw in (dict(kind=3), dict(kind=0, out=Operand((4, 64), F32)), dict(kind=1, out=Operand((4, 64), F8)),
               dict(kind=1, out=(Operand((4, 64), F8), Operand((4, 2), F32))), dict(kind=2, out=rows(4, 96)),
               dict(delta=Operand((4, 32), BF16), h_out=x, out=x), dict(h_out=Operand((4, 64), F32), out=x)):
        _refused(nv, lambda: nv.rmsnorm_residual(x, w, **kw), nv.NVFP4_ERR_INVALID_ARG)
    _refused(nv, lambda: nv.moe_swiglu(Operand((4, 65), BF16), out=Operand((4, 32), BF16)), nv.NVFP4_ERR_UNSUPPORTED_SHAPE)
    _refused(nv, lambda: nv.moe_swiglu(Operand((4, 64), torch.float16)), nv.NVFP4_ERR_INVALID_ARG)
    _refused(nv, lambda: nv.moe_combine(Operand((7, 8), BF16), 2, y=x), nv.NVFP4_ERR_UNSUPPORTED_SHAPE)
    _refused(nv, lambda: nv.moe_combine_backward(Operand((4, 8), BF16), Operand((7, 8), BF16)), nv.NVFP4_ERR_UNSUPPORTED_SHAPE)
    _refused(nv, lambda: nv.moe_permute(x, Operand((7,), I32), 2, rows=Operand((8, 64), BF16), positions=Operand((8,), I32)),
             nv.NVFP4_ERR_INVALID_ARG)


@pytest.mark.parametrize("N", [(1 << 31), (1 << 32) + 5])
def test_sizes_past_32_bits_are_refused(nv, N):  # noqa: F811
    x = (Operand((4, 16), U8), Operand((4, 2), U8), Operand((4,), F32))
    W = nv.NVFP4Weight(Operand((N, 16), U8), Operand((N, 2), U8), Operand((1,), F32), N, 32, nv.SCALE_E4M3)
    y = Operand((4, N), F32)
    for call in (lambda: nv.nvfp4_gemm_w4a4(*x, W, y=y),
                 lambda: nv.moe_grouped_gemm_nvfp4(*x, Operand((2, N, 16), U8), Operand((2, N, 2), U8), Operand((2,), F32),
                                                   Operand((3,), I32), y=y),
                 lambda: nv.moe_grouped_gemm_nvfp4(*x, Operand((N, 8, 16), U8), Operand((N, 8, 2), U8), Operand((N,), F32),
                                                   Operand((N + 1,), I32), y=Operand((4, 8), F32)),
                 lambda: nv.moe_permute(Operand((4, 8), BF16), Operand((4 * N,), I32), N, rows=y, positions=y),
                 lambda: nv.nvfp4_quantize_rows(Operand((N, 64), BF16), out=(x[0], x[1], x[2])),
                 lambda: nv.nvfp4_dequantize_rows(Operand((4, N), U8), Operand((4, N // 8), U8), x[2], y=y),
                 lambda: nv.moe_combine(Operand((4, N), BF16), 2, y=y)):
        _refused(nv, call, nv.NVFP4_ERR_UNSUPPORTED_SHAPE)


def test_scales_cross_a_pair_of_ctas_at_its_scope():
    """The first CTA of a pair reads scales that the second one's warps stored: the arrival that hands them over releases to
    the cluster, and the wait for it acquires from there. (An order that only the source can show.)"""
    import os
    import re
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "nvfp4_w4a16_moe_gb300", "csrc")
    with open(os.path.join(csrc, "pair_tc.cuh")) as f:
        pair = f.read()
    with open(os.path.join(csrc, "rows_fp4.cu")) as f:
        kernel = f.read()
    body = lambda name: re.search(r"\b%s\(.*?\n}" % name, pair, re.S).group(0)  # noqa: E731
    release = body("arrive_cluster_release_smem")
    assert 0 < release.index("fence.release.sync_restrict::shared::cta.cluster") < release.index("mbarrier.arrive.relaxed.cluster.shared::cluster.b64")
    for name in ("test", "try"):
        assert "mbarrier.%s_wait.parity.acquire.cluster.shared::cta.b64" % name in body("mbar_%s_wait_cluster" % name)
    arrivals = re.findall(r"fence_proxy_async_smem\(\);\s*__syncwarp\(\);\s*if \(elect_one\(\)\) (\w+)\(", kernel)
    assert arrivals == ["arrive_cluster_release_smem"] * 2      # rows of scales that are strides, and others
    assert kernel.count("fence_proxy_async_smem()") == 2
    assert re.findall(r"wait\.one(\S*)\(&sf_ready\[", kernel) == ["<true>"]


def test_copies_go_to_one_cta():
    """Ranks of several GPUs load the library, and loads that a cluster's CTAs share are for one GPU's own memory alone: no
    copy from memory names more than one CTA. (What does are the tensor cores' arrivals on barriers.)"""
    import glob
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    sources = glob.glob(os.path.join(root, "nvfp4_w4a16_moe_gb300", "csrc", "*.cu*")) + [os.path.join(root, "include", "nvfp4moe.h")]
    assert len(sources) > 10
    for path in sources:
        with open(path) as f:
            text = re.sub(r'"\s*\n\s*"', "", f.read())       # instructions in several literals
        for literal in re.findall(r'"([^"\n]*multicast[^"\n]*)"', text):
            for instruction in literal.split(";"):
                if "multicast" in instruction:
                    assert instruction.strip().startswith("tcgen05.commit."), (os.path.basename(path), instruction)
