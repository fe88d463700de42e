"""Checks of the 8-bit and grouped products that need no GPU: the 64-bit forms that the GPU tests
compare with, and the refusals of the C entry points (all before CUDA is touched)."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import products_ref as ref


@pytest.fixture(scope="module")
def nv():
    import __graft_entry__
    __graft_entry__.build()
    import nvfp4_w4a16_moe_gb300 as nv
    return nv


def test_reference_decodes_and_rounds_like_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(np.isnan(want), np.isnan(ref.E4M3))
    fin = ~np.isnan(want)
    assert np.array_equal(want[fin], ref.E4M3[fin])
    mid = (ref.GRID[1:] + ref.GRID[:-1]) / 2          # every tie
    v = np.concatenate([ref.GRID, mid, mid * (1 + 1e-6), mid * (1 - 1e-6), np.linspace(0, 448, 1001)])
    v = np.concatenate([v, -v]).astype(np.float32)
    t = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.nearest_code(v.astype(np.float64)), t)


def test_quantised_values_are_within_half_a_step():
    g = torch.Generator().manual_seed(3)
    x = (torch.randn(2, 130, 200, generator=g) * 3).to(torch.bfloat16)
    for br in (1, 128):
        q, s = ref.quantize(x, br)
        back = ref.E4M3[q] * ref.spread(s.astype(np.float64), br, 130, 200)
        d = ref.f64(x)
        amax = ref.spread(s.astype(np.float64), br, 130, 200) * 448
        # half a step of E4M3 is 2^-4 of the value, or 2^-10 of the scale below the smallest normal
        assert np.all(np.abs(back - d) <= np.maximum(np.abs(d) * 2.0 ** -4, amax / 448 * 2.0 ** -10) * (1 + 1e-6))


def test_ratio_of_bf16_significands_stays_off_the_rounding_points():
    """The quantiser rounds 448 x / a from an fp32 value within 2^-22 of it, put on 16 significant
    bits: no quotient of two bf16 significands comes nearer than 2^-13 to a point where the
    rounding changes without being on it."""
    m = np.arange(128, 256)
    nearest = np.inf
    for j in range(1, 32, 2):
        for d in range(-12, 13):
            num = 7 * m[:, None] * 2.0 ** d - j * m[None, :]
            rel = np.abs(num) / (j * m[None, :])
            nearest = min(nearest, rel[rel > 0].min())
    assert nearest >= 2.0 ** -13


class Groups(ctypes.Structure):         # moe_groups of the C header
    _fields_ = [("R", ctypes.c_int32), ("E", ctypes.c_int32), ("k", ctypes.c_int32), ("gather", ctypes.c_int32),
                ("scatter", ctypes.c_int32), ("expert_offsets", ctypes.c_void_p), ("token_list", ctypes.c_void_p)]


def test_python_packs_the_groups_like_c(nv):
    g = Groups(1, 2, 3, 4, 5, 6, 7)
    assert bytes(g) == nv._GROUPS.pack(1, 2, 3, 4, 5, 6, 7)


FAKE = 0x100000        # never dereferenced: the checks fail first


def _status(nv, fn, *args):
    return getattr(nv.lib, fn)(*args)


def test_quantize_refusals(nv):
    call = lambda x=FAKE, B=1, R=4, K=64, br=1, q=FAKE, s=FAKE: _status(nv, "fp8_quantize_block128", x, B, R, K, br,
                                                                        q, s, None)
    assert call(br=64) == nv.NVFP4_ERR_INVALID_ARG
    for kw in (dict(x=None), dict(q=None), dict(s=None)):
        assert call(**kw) == nv.NVFP4_ERR_INVALID_ARG
    for kw in (dict(B=-1), dict(R=-1), dict(K=0), dict(K=8), dict(K=24), dict(K=65552), dict(B=1 << 16, R=1 << 16)):
        assert call(**kw) == nv.NVFP4_ERR_UNSUPPORTED_SHAPE
    for kw in (dict(x=FAKE + 8), dict(q=FAKE + 8), dict(s=FAKE + 2)):
        assert call(**kw) == nv.NVFP4_ERR_MISALIGNED


def test_dense_refusals(nv):
    def call(x=FAKE, xs=FAKE, T=4, w=FAKE, ws=FAKE, N=16, K=64, y=FAKE, yt=0, wk=None, wb=0):
        return _status(nv, "fp8_gemm_block128", x, xs, T, w, ws, N, K, y, yt, wk, wb, None)
    assert call(yt=2) == nv.NVFP4_ERR_INVALID_ARG
    for kw in (dict(x=None), dict(xs=None), dict(w=None), dict(ws=None), dict(y=None)):
        assert call(**kw) == nv.NVFP4_ERR_INVALID_ARG
    for kw in (dict(T=-1), dict(T=(1 << 20) + 1), dict(N=0), dict(N=(1 << 22) + 1), dict(K=0), dict(K=40),
               dict(K=65552)):
        assert call(**kw) == nv.NVFP4_ERR_UNSUPPORTED_SHAPE
    for kw in (dict(x=FAKE + 8), dict(w=FAKE + 4), dict(y=FAKE + 2), dict(xs=FAKE + 2), dict(ws=FAKE + 1),
               dict(wk=FAKE + 8, wb=256)):
        assert call(**kw) == nv.NVFP4_ERR_MISALIGNED
    assert call(wk=FAKE, wb=128) == nv.NVFP4_ERR_WORKSPACE_TOO_SMALL


@pytest.mark.parametrize("fp8", [False, True])
def test_grouped_refusals(nv, fp8):
    def call(R=8, E=4, k=2, gather=0, scatter=0, off=FAKE, lst=FAKE, x=FAKE, w=FAKE, N=16, K=64, y=FAKE, yt=0,
             wk=None, wb=0, xs=FAKE, ws=FAKE, null=False):
        g = Groups(R, E, k, gather, scatter, off, lst)
        p = None if null else ctypes.addressof(g)
        if fp8:
            return _status(nv, "moe_grouped_gemm_fp8", p, x, xs, w, ws, N, K, y, yt, wk, wb, None)
        return _status(nv, "moe_grouped_gemm_bf16", p, x, w, N, K, y, yt, wk, wb, None)
    for kw in (dict(null=True), dict(off=None), dict(lst=None, gather=1), dict(lst=None, scatter=1), dict(x=None),
               dict(w=None), dict(y=None), dict(yt=-1)):
        assert call(**kw) == nv.NVFP4_ERR_INVALID_ARG
    for kw in (dict(R=-1), dict(R=(1 << 20) + 2), dict(E=0), dict(E=257), dict(k=0), dict(R=7, gather=1), dict(N=0),
               dict(K=0), dict(K=20), dict(K=24 if fp8 else 4), dict(E=256, N=1 << 23)):
        assert call(**kw) == nv.NVFP4_ERR_UNSUPPORTED_SHAPE, kw
    assert call(E=256, N=1 << 22, x=None) == nv.NVFP4_ERR_INVALID_ARG    # 2^30 rows of W: the next check is reached
    for kw in (dict(x=FAKE + 8), dict(w=FAKE + 8), dict(y=FAKE + 4), dict(off=FAKE + 2), dict(lst=FAKE + 1)):
        assert call(**kw) == nv.NVFP4_ERR_MISALIGNED
    if fp8:
        assert call(xs=None) == nv.NVFP4_ERR_INVALID_ARG and call(ws=FAKE + 2) == nv.NVFP4_ERR_MISALIGNED
    assert call(wk=FAKE, wb=16) == nv.NVFP4_ERR_WORKSPACE_TOO_SMALL


def test_python_refuses_host_tensors(nv):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(nv.NVFP4Error):
        nv.fp8_quantize_block128(x)
    with pytest.raises(nv.NVFP4Error):
        nv.fp8_quantize_block128(x, block_rows=64)
    with pytest.raises(nv.NVFP4Error):
        nv.moe_grouped_gemm_bf16(x, torch.zeros(2, 8, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32))


class Operand:
    """What the Python calls read of a tensor, at any size: no memory behind it."""

    def __init__(self, shape, dtype):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, "cuda:0"

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return FAKE


F8, F32, BF16, I32 = torch.float8_e4m3fn, torch.float32, torch.bfloat16, torch.int32


@pytest.mark.parametrize("N", [(1 << 31), (1 << 32) + 5])
def test_outputs_past_32_bits_are_refused(nv, N):
    """The C ABI takes int32: 2^32 + 5 weight rows must not arrive there as 5."""
    dense = lambda: nv.fp8_gemm_block128(Operand((4, 16), F8), Operand((4, 1), F32), Operand((N, 16), F8),
                                         Operand(((N + 127) // 128, 1), F32), y=Operand((4, N), F32))
    grouped = lambda: nv.moe_grouped_gemm_bf16(Operand((4, 16), BF16), Operand((2, N, 16), BF16), Operand((3,), I32),
                                               y=Operand((4, N), F32))
    grouped8 = lambda: nv.moe_grouped_gemm_fp8(Operand((4, 16), F8), Operand((4, 1), F32), Operand((2, N, 16), F8),
                                               Operand((2, (N + 127) // 128, 1), F32), Operand((3,), I32),
                                               y=Operand((4, N), F32))
    for call in (dense, grouped, grouped8):
        with pytest.raises(nv.NVFP4Error) as e:
            call()
        assert e.value.status == nv.NVFP4_ERR_UNSUPPORTED_SHAPE


@pytest.mark.parametrize("E", [1 << 31, (1 << 32) + 2])
def test_experts_past_32_bits_are_refused(nv, E):
    with pytest.raises(nv.NVFP4Error) as e:
        nv.moe_grouped_gemm_bf16(Operand((4, 16), BF16), Operand((E, 8, 16), BF16), Operand((E + 1,), I32),
                                 y=Operand((4, 8), F32))
    assert e.value.status == nv.NVFP4_ERR_UNSUPPORTED_SHAPE


@pytest.mark.parametrize("shape", [(), (16,), (1, 8, 16)])
def test_a_dense_weight_has_two_dimensions(nv, shape):
    with pytest.raises(nv.NVFP4Error) as e:
        nv.fp8_gemm_block128(Operand((4, 16), F8), Operand((4, 1), F32), Operand(shape, F8), Operand((1, 1), F32),
                             y=Operand((4, 8), F32))
    assert e.value.status == nv.NVFP4_ERR_INVALID_ARG


def test_imports_on_a_torch_without_cuda(nv):
    """Such a torch lacks the two private names that the product calls use where they are there."""
    code = ("import torch\n"
            "del torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream\n"
            "import nvfp4_w4a16_moe_gb300 as nv\n"
            "assert callable(nv._current_device) and callable(nv._raw_stream)\n"
            "assert nv.lib.nvfp4_version() >= 1\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


PTXAS = """ptxas info    : Compiling entry function '_ZN14rows_tc_kernelILb%dELi64ELi1EEEvx' for 'sm_103a'
ptxas info    : Function properties for _ZN14rows_tc_kernelILb%dELi64ELi1EEEvx
    0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads
ptxas info    : Used %d registers, used 1 barriers
"""


def test_build_refuses_another_register_count_than_the_launch_needs(nv):
    """The 8-bit tile kernels move registers between their warps; compiled to another count they would be refused
    at every launch. bf16 kernels (Lb0) do not."""
    from nvfp4_w4a16_moe_gb300 import build
    source = "constexpr int kLaunchRegs = 80, kEpiRegs = 96;"
    good = PTXAS % (0, 0, 72) + PTXAS % (1, 1, 80)
    build.check_launch_registers("constexpr int kOther = 1;", "")
    build.check_launch_registers(source, good)
    for bad in (PTXAS % (0, 0, 72), good + PTXAS % (1, 1, 72), PTXAS % (1, 1, 88) + good):
        with pytest.raises(RuntimeError, match="register"):
            build.check_launch_registers(source, bad)
