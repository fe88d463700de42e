"""Cases of the operators between and around the experts' products: the norm with the residual, NVFP4 rows and
their products, the SwiGLU, and rows sorted by expert and back.

``run`` computes one pass of an operator: with ``own`` false in elementary torch operations, with ``own`` true
through this package's entry points. The sizes are those of the Qwen3.6-35B-A3B-shaped layer that the tests and the
benchmark use (hidden 2048, 256 experts, 8 per token, intermediate 512) and of its dense 8192 x 2048 projection,
with ragged sizes around them. 4-bit values are returned as what they stand for.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
E2M1_MAX = 6.0
EPS = 1e-6


def listed():
    return [
        # residual add and norm of a prefill call before 8-bit experts
        dict(name="norm_fp8_4096", op="norm", T=4096, H=2048, out="fp8", delta=True),
        # norm of a few decoded tokens, a width that is no multiple of a warp's: latency
        dict(name="norm_bf16_5_ragged", op="norm", T=5, H=1000, out="bf16", delta=True),
        # norm into 4-bit rows and the projection behind it, a decode batch, odd widths
        dict(name="norm_nvfp4_dense_33", op="norm_dense", T=33, H=2016, N=5003, delta=True),
        # activations of a prefill call into 4-bit rows and back (what the rows stand for)
        dict(name="quantize_4096", op="quantize", R=4096, K=2048),
        # a small decode batch with a ragged width: latency
        dict(name="quantize_7_ragged", op="quantize", R=7, K=1056),
        # between gate/up and down of a prefill call with 8-bit experts
        dict(name="swiglu_fp8_4096", op="swiglu", R=4096 * 8, I=512, out="fp8", fp32=False),
        # SwiGLU into 4-bit rows and down of a 64-token decode batch, rows put back into the tokens' order
        dict(name="swiglu_nvfp4_down_64", op="swiglu_down", T=64, E=256, k=8, N=2048, I=512),
        # 4-bit dense projection of one decoded token (fp32 logits): latency and weight streaming
        dict(name="dense_1", op="dense", T=1, N=8192, K=2048, fp32=True),
        # 4-bit dense projection of a prefill call
        dict(name="dense_4096", op="dense", T=4096, N=8192, K=2048, fp32=False),
        # gate/up of a prefill call over 4-bit experts, two tensor scales a matrix
        dict(name="gate_up_4096", op="grouped", T=4096, E=256, k=8, N=1024, K=2048, parts=2, rows="gather", fp32=False),
        # rows of a 64-token decode batch sorted by expert, and back with the router's weights and the residual
        dict(name="sort_64", op="sort", T=64, E=256, k=8, N=2048, backward=False, fp32=False),
        # the same for 4096 tokens with the gradients of rows, weights and tokens
        dict(name="sort_backward_4096", op="sort", T=4096, E=256, k=8, N=2048, backward=True, fp32=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


_FLOPS = 2.0 * 4096 * 8 * 1024 * 2048      # the largest listed case


def draw(rng):
    op = rng.choice(["norm", "norm_dense", "quantize", "swiglu", "swiglu_down", "dense", "grouped", "grouped", "sort", "sort"])
    if op == "norm":
        out = rng.choice(["bf16", "fp8"])
        unit = 8 if out == "bf16" else 16
        return dict(op=op, T=_log(rng, 1, 8192), H=unit * _log(rng, 64 // unit, 8192 // unit), out=out, delta=rng.random() < 0.7)
    if op == "norm_dense":
        return dict(op=op, T=_log(rng, 16, 512), H=32 * _log(rng, 16, 128), N=_log(rng, 128, 8192), delta=rng.random() < 0.7)
    if op == "quantize":
        return dict(op=op, R=_log(rng, 1, 16384), K=32 * _log(rng, 2, 256))
    if op == "swiglu":
        out = rng.choice(["bf16", "fp8"])
        unit = 8 if out == "bf16" else 16
        return dict(op=op, R=_log(rng, 1, 16384), I=unit * _log(rng, 64 // unit, 2048 // unit), out=out, fp32=rng.random() < 0.3)
    if op == "dense":
        N, K = _log(rng, 128, 8192), 32 * _log(rng, 4, 256)
        T = min(_log(rng, 1, 4096), max(1, int(_FLOPS / (2.0 * N * K))))
        return dict(op=op, T=T, N=N, K=K, fp32=rng.random() < 0.3)
    E = _log(rng, 2, 256)
    k = rng.randint(1, min(8, E))
    if op == "sort":
        return dict(op=op, T=_log(rng, 1, 4096), E=E, k=k, N=_log(rng, 64, 2048), backward=rng.random() < 0.5, fp32=rng.random() < 0.3)
    N, K = _log(rng, 64, 2048), 32 * _log(rng, 2, 64)
    T = min(_log(rng, 1, 4096), max(1, int(_FLOPS / (2.0 * N * K * k * 4))))
    if op == "swiglu_down":
        return dict(op=op, T=max(T, 16), E=E, k=k, N=N, I=K)
    return dict(op=op, T=T, E=E, k=k, N=N - N % 2, K=K, parts=rng.choice([1, 2]), rows=rng.choice(["gather", "scatter", "list"]),
                fp32=rng.random() < 0.3)


# ---------------------------------------------------------------- plain forms

def _blocks(n, size):
    return (n + size - 1) // size


def _by_block(v, size, K):
    """One value of each block -> one of each element of a row."""
    return v.repeat_interleave(size, dim=-1)[..., :K]


def _amax(x, size):
    R, K = x.shape
    padded = x.new_zeros(R, _blocks(K, size) * size)
    padded[:, :K] = x.abs()
    return padded.view(R, -1, size).amax(dim=2)


def _to_fp8(x):
    """E4M3 codes of fp32 rows and one scale per 1 x 128."""
    a = _amax(x, 128)
    some = torch.where(a == 0, torch.full_like(a, E4M3_MAX), a)
    q = x * _by_block(E4M3_MAX / some, 128, x.shape[1])
    return q.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), some / E4M3_MAX


def _power_of_two(q):
    """The smallest power of two that is not below q > 0, and at least 2^-126."""
    m, e = torch.frexp(q)
    return torch.ldexp(torch.ones_like(q), torch.where(m == 0.5, e - 1, e).clamp(min=-126))


def _nearest_e2m1(u):
    """Nearest of 0, .5, 1, 1.5, 2, 3, 4, 6 to |u|, ties to the even code, saturating."""
    a = u.abs()
    v = torch.where(a < 2, (a * 2).round() / 2, torch.where(a < 4, a.round(), (a / 2).round() * 2)).clamp(max=E2M1_MAX)
    return torch.copysign(v, u)


def _to_nvfp4(x):
    """(values of the codes, E4M3 scale per 16, power-of-two scale per row) of fp32 rows. For bf16 rows every quotient
    is exact or far enough from a border for 32 bits."""
    a = x.abs().amax(dim=1, keepdim=True)
    s = torch.where(a == 0, torch.ones_like(a), _power_of_two(a / (E2M1_MAX * E4M3_MAX)))
    v = x / s
    e = (_amax(v, 16) / E2M1_MAX).clamp(max=E4M3_MAX).to(torch.float8_e4m3fn)
    d = _by_block(e.float(), 16, x.shape[1])
    return _nearest_e2m1(torch.where(d == 0, torch.zeros_like(v), v / torch.where(d == 0, torch.ones_like(d), d))), e, s[:, 0]


_CODES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _pack(values):
    """Values on the E2M1 grid -> codes, two a byte, the first in the low four bits."""
    a = values.abs()
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8) | (torch.signbit(values).to(torch.uint8) << 3)
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _unpack(packed, scales, dtype=torch.float32):
    """code x block scale."""
    table = torch.tensor(_CODES, dtype=dtype, device=packed.device)
    v = table[torch.stack([packed & 15, packed >> 4], dim=-1).flatten(-2).long()]
    return v * scales.view(torch.float8_e4m3fn).to(dtype).repeat_interleave(16, dim=-1)


def _norm(h, w, delta):
    h = h.float()
    if delta is not None:
        h = (h + delta.float()).to(torch.bfloat16).float()      # the residual stream is bf16
    return h, h * torch.rsqrt(h.square().mean(dim=1, keepdim=True) + EPS) * (1.0 + w.float())


def _silu_up(gu):
    g, u = gu.float().chunk(2, dim=1)
    return g / (1.0 + torch.exp(-g)) * u


# ---------------------------------------------------------------- inputs

def _normal(gen, *shape, std=1.0):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.bfloat16) * std


def _tokens(gen, rows, K):
    """Activations with the few large channels that hidden states have."""
    x = _normal(gen, rows, K)
    wide = torch.randint(0, K, (max(1, K // 256),), generator=gen, device="cuda")
    x[:, wide] *= 16.0
    return x


def _weight(gen, E, N, K, parts):
    """NVFP4 weights of E matrices with one tensor scale to each of `parts` runs of rows, made in slices."""
    packed = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(E, N, K // 16, dtype=torch.uint8, device="cuda")
    tscale = torch.empty(E, parts, dtype=torch.float32, device="cuda")
    step = max(1, (1 << 25) // (N * K))
    for e in range(0, E, step):
        w = _normal(gen, min(step, E - e), N, K, std=0.02).float()
        n = w.shape[0]
        t = w.abs().view(n, parts, -1).amax(dim=2) / (E2M1_MAX * E4M3_MAX)
        v = w / t.repeat_interleave(N // parts, dim=1)[:, :, None]
        b = (v.abs().view(n, N, -1, 16).amax(dim=3) / E2M1_MAX).to(torch.float8_e4m3fn)
        packed[e:e + step] = _pack(_nearest_e2m1(v / b.float().repeat_interleave(16, dim=2)))
        scales[e:e + step] = b.view(torch.uint8)
        tscale[e:e + step] = t
    return packed, scales, tscale


def _routing(gen, s, case):
    """Top-k routing of random logits, some experts more popular than others; entries t*k + j in expert order."""
    T, E, k = case["T"], case["E"], case["k"]
    logits = torch.randn(T, E, generator=gen, device="cuda") + 0.5 * torch.randn(E, generator=gen, device="cuda")
    top = logits.topk(k, dim=1)
    ids = top.indices.reshape(-1)
    counts = torch.bincount(ids, minlength=E)
    s["weights"] = torch.softmax(top.values, dim=1)
    s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    s["token_list"] = torch.argsort(ids, stable=True).to(torch.int32)
    s["most"] = int(counts.max())


def _row_buffers(R, K, out):
    """What a program keeps for rows of K in this form."""
    e = lambda *shape, dtype: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    if out == "bf16":
        return e(R, K, dtype=torch.bfloat16)
    if out == "fp8":
        return e(R, K, dtype=torch.float8_e4m3fn), e(R, _blocks(K, 128), dtype=torch.float32)
    return e(R, K // 2, dtype=torch.uint8), e(R, K // 16, dtype=torch.uint8), e(R, dtype=torch.float32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s, op = dict(case), case["op"]
    empty = lambda *shape, dtype: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    if op in ("norm", "norm_dense"):
        T, H = case["T"], case["H"]
        s["h"] = _tokens(gen, T, H)
        s["delta"] = _normal(gen, T, H, std=0.3) if case["delta"] else None
        s["norm_w"] = _normal(gen, H, std=0.2)
        s["h_out"] = empty(T, H, dtype=torch.bfloat16)
        s["rows"] = _row_buffers(T, H, case["out"] if op == "norm" else "nvfp4")
        if op == "norm_dense":
            s["w"], s["ws"], s["wt"] = (t[0] for t in _weight(gen, 1, case["N"], H, 1))
            s["y"] = empty(T, case["N"], dtype=torch.bfloat16)
        return s
    if op == "quantize":
        s["x"] = _tokens(gen, case["R"], case["K"])
        s["rows"] = _row_buffers(case["R"], case["K"], "nvfp4")
        s["y"] = empty(case["R"], case["K"], dtype=torch.bfloat16)
        return s
    if op == "swiglu":
        s["gu"] = _normal(gen, case["R"], 2 * case["I"], std=1.5)
        if case["fp32"]:
            s["gu"] = s["gu"].float()
        s["rows"] = _row_buffers(case["R"], case["I"], case["out"])
        return s
    if op == "dense":
        v, e, s["xr"] = _to_nvfp4(_tokens(gen, case["T"], case["K"]).float())
        s["x"], s["xs"] = _pack(v), e.view(torch.uint8)
        s["w"], s["ws"], s["wt"] = (t[0] for t in _weight(gen, 1, case["N"], case["K"], 1))
        s["y"] = empty(case["T"], case["N"], dtype=torch.float32 if case["fp32"] else torch.bfloat16)
        return s
    _routing(gen, s, case)
    R, N = case["T"] * case["k"], case["N"]
    if op == "sort":
        out = torch.float32 if case["fp32"] else torch.bfloat16       # of the rows that experts return
        s["x"] = _tokens(gen, case["T"], N)
        s["add"] = _normal(gen, case["T"], N)
        s["rows"], s["positions"] = empty(R, N, dtype=torch.bfloat16), empty(R, dtype=torch.int32)
        s["back"] = _normal(gen, R, N).to(out)
        s["y"] = empty(case["T"], N, dtype=torch.bfloat16)
        if case["backward"]:
            s["dy"] = _normal(gen, case["T"], N)
            s["d_back"], s["d_w"] = empty(R, N, dtype=out), empty(case["T"], case["k"], dtype=torch.float32)
            s["d_rows"], s["d_x"] = _normal(gen, R, N), empty(case["T"], N, dtype=torch.bfloat16)
        return s
    if op == "swiglu_down":
        s["gu"] = _normal(gen, R, 2 * case["I"], std=1.5)
        s["rows"] = _row_buffers(R, case["I"], "nvfp4")
        s["w"], s["ws"], s["wt"] = _weight(gen, case["E"], N, case["I"], 1)
        s["y"] = empty(R, N, dtype=torch.bfloat16)
        return s
    v, e, s["xr"] = _to_nvfp4(_tokens(gen, case["T"] if case["rows"] == "gather" else R, case["K"]).float())
    s["x"], s["xs"] = _pack(v), e.view(torch.uint8)
    s["w"], s["ws"], s["wt"] = _weight(gen, case["E"], N, case["K"], case["parts"])
    s["y"] = empty(R, N, dtype=torch.float32 if case["fp32"] else torch.bfloat16)
    return s


# ---------------------------------------------------------------- one pass

def _rows_of(s, rows):
    """x row, y row and expert of every list position."""
    R = s["T"] * s["k"]
    r = torch.arange(R, device="cuda")
    entry = s["token_list"].long()
    expert = torch.searchsorted(s["offsets"].long(), r, right=True) - 1
    return (entry // s["k"] if rows == "gather" else r), (entry if rows == "scatter" else r), expert


def _plain_grouped(s, x, rows):
    """x: fp32 values of the rows."""
    src, dst, expert = _rows_of(s, rows)
    R, E, N = s["T"] * s["k"], s["E"], s["N"]
    parts = s["wt"].shape[1]
    matrices = lambda at: _unpack(s["w"][at], s["ws"][at]) * s["wt"][at].repeat_interleave(N // parts, dim=1)[:, :, None]  # noqa: E731
    x = x[src]
    if R <= E:             # few rows: each with its expert's matrix
        y_rows = torch.bmm(matrices(expert), x[:, :, None])[:, :, 0]
    else:                  # the experts' rows padded to the longest
        at = torch.arange(R, device="cuda") - s["offsets"].long()[expert]
        padded = x.new_zeros(E, s["most"], x.shape[1])
        padded[expert, at] = x
        y_rows = torch.bmm(padded, matrices(slice(None)).transpose(1, 2))[expert, at]
    y = torch.empty_like(y_rows)
    y[dst] = y_rows
    return y.to(s["y"].dtype)


def _run_own(s):
    import nvfp4_w4a16_moe_gb300 as nv
    kinds = {"bf16": nv.ROWS_BF16, "fp8": nv.ROWS_FP8}
    op = s["op"]
    if op == "norm":
        return nv.rmsnorm_residual(s["h"], s["norm_w"], EPS, delta=s["delta"], kind=kinds[s["out"]], h_out=s["h_out"], out=s["rows"])
    if op == "norm_dense":
        h, rows = nv.rmsnorm_residual(s["h"], s["norm_w"], EPS, delta=s["delta"], kind=nv.ROWS_NVFP4, h_out=s["h_out"], out=s["rows"])
        return h, nv.nvfp4_gemm_w4a4(*rows, nv.NVFP4Weight(s["w"], s["ws"], s["wt"], s["N"], s["H"], nv.SCALE_E4M3), y=s["y"])
    if op == "quantize":
        packed, scales, row_scales = nv.nvfp4_quantize_rows(s["x"], out=s["rows"])
        y = nv.nvfp4_dequantize_rows(packed, scales, row_scales, y=s["y"])
        return y, scales.view(torch.float8_e4m3fn), row_scales
    if op == "swiglu":
        return nv.moe_swiglu(s["gu"], kind=kinds[s["out"]], out=s["rows"])
    if op == "dense":
        W = nv.NVFP4Weight(s["w"], s["ws"], s["wt"], s["N"], s["K"], nv.SCALE_E4M3)
        return nv.nvfp4_gemm_w4a4(s["x"], s["xs"], s["xr"], W, y=s["y"])
    if op == "sort":
        rows, positions = nv.moe_permute(s["x"], s["token_list"], s["k"], rows=s["rows"], positions=s["positions"])
        y = nv.moe_combine(s["back"], s["k"], s["weights"], positions, add=s["add"], y=s["y"])
        if not s["backward"]:
            return rows, positions, y
        d_back, d_w = nv.moe_combine_backward(s["dy"], s["back"], s["weights"], positions, d_rows=s["d_back"], d_w=s["d_w"])
        d_x = nv.moe_combine(s["d_rows"], s["k"], None, positions, y=s["d_x"])
        return rows, positions, y, d_back, d_w, d_x
    if op == "swiglu_down":
        rows = nv.moe_swiglu(s["gu"], kind=nv.ROWS_NVFP4, out=s["rows"])
        return nv.moe_grouped_gemm_nvfp4(*rows, s["w"], s["ws"], s["wt"], s["offsets"], s["token_list"], s["k"], scatter=True, y=s["y"])
    return nv.moe_grouped_gemm_nvfp4(s["x"], s["xs"], s["xr"], s["w"], s["ws"], s["wt"], s["offsets"],
                                     token_list=None if s["rows"] == "list" else s["token_list"], k=s["k"],
                                     gather=s["rows"] == "gather", scatter=s["rows"] == "scatter", y=s["y"])


def run(s):
    if own:
        return _run_own(s)
    op = s["op"]
    if op in ("norm", "norm_dense"):
        h, x = _norm(s["h"], s["norm_w"], s["delta"])
        h = h.to(torch.bfloat16)
        if op == "norm":
            return h, (x.to(torch.bfloat16) if s["out"] == "bf16" else _to_fp8(x))
        v, e, r = _to_nvfp4(x)
        x = v * _by_block(e.float(), 16, s["H"]) * r[:, None]
        return h, (x @ (_unpack(s["w"], s["ws"]) * s["wt"]).t()).to(torch.bfloat16)
    if op == "quantize":
        v, e, r = _to_nvfp4(s["x"].float())
        return (v * _by_block(e.float(), 16, s["K"]) * r[:, None]).to(torch.bfloat16), e, r
    if op == "swiglu":
        h = _silu_up(s["gu"])
        return h.to(torch.bfloat16) if s["out"] == "bf16" else _to_fp8(h)
    if op == "dense":
        x = _unpack(s["x"], s["xs"]) * s["xr"][:, None]
        return (x @ (_unpack(s["w"], s["ws"]) * s["wt"]).t()).to(s["y"].dtype)
    if op == "sort":
        T, k, N = s["T"], s["k"], s["N"]
        entry = s["token_list"].long()
        positions = torch.empty_like(s["token_list"])
        positions[entry] = torch.arange(T * k, dtype=torch.int32, device="cuda")
        at = positions.long()
        back = s["back"][at].float().view(T, k, N)
        y = (s["add"].float() + (back * s["weights"][:, :, None]).sum(1)).to(torch.bfloat16)
        rows = s["x"][entry // k]
        if not s["backward"]:
            return rows, positions, y
        dy = s["dy"].float()
        d_back = torch.empty_like(s["back"])
        d_back[at] = (dy[:, None, :] * s["weights"][:, :, None]).view(T * k, N).to(d_back.dtype)
        d_w = (back * dy[:, None, :]).sum(2)
        return rows, positions, y, d_back, d_w, s["d_rows"][at].float().view(T, k, N).sum(1).to(torch.bfloat16)
    if op == "swiglu_down":
        v, e, r = _to_nvfp4(_silu_up(s["gu"]))
        return _plain_grouped(s, v * _by_block(e.float(), 16, s["I"]) * r[:, None], "scatter")
    return _plain_grouped(s, _unpack(s["x"], s["xs"]) * s["xr"][:, None], s["rows"])


_OUT_BYTES = {"bf16": 2.0, "fp8": 1.0 + 4.0 / 128, "nvfp4": 0.5 + 1.0 / 16}


def work(case):
    """Every input once and every output once. For the grouped products the matrices of the experts that an even routing
    of so many tokens reaches; chained calls hand their rows over without memory."""
    op = case["op"]
    if op == "norm":
        n = case["T"] * case["H"]
        return {"bytes": n * (4.0 + (2.0 if case["delta"] else 0.0) + _OUT_BYTES[case["out"]]) + 2.0 * case["H"], "flops": 6.0 * n}
    if op == "norm_dense":
        T, H, N = case["T"], case["H"], case["N"]
        return {"bytes": T * H * (4.0 + (2.0 if case["delta"] else 0.0)) + 2.0 * H + N * H * 0.5625 + 2.0 * T * N,
                "flops": 2.0 * T * N * H + 6.0 * T * H}
    if op == "quantize":
        n = case["R"] * case["K"]
        return {"bytes": n * (2.0 + 0.5625 + 2.0) + 4.0 * case["R"], "flops": 3.0 * n}
    if op == "swiglu":
        n = case["R"] * case["I"]
        return {"bytes": n * ((8.0 if case["fp32"] else 4.0) + _OUT_BYTES[case["out"]]), "flops": 6.0 * n}
    if op == "dense":
        T, N, K = case["T"], case["N"], case["K"]
        return {"bytes": 0.5625 * (T + N) * K + 4.0 * T + (4.0 if case["fp32"] else 2.0) * T * N, "flops": 2.0 * T * N * K}
    T, E, k, N = case["T"], case["E"], case["k"], case["N"]
    R = T * k
    if op == "sort":
        es = 4.0 if case["fp32"] else 2.0
        bytes_ = 2.0 * T * N + 2.0 * R * N + 8.0 * R + es * R * N + 4.0 * R + 4.0 * T * N      # permute, combine
        if case["backward"]:
            bytes_ += 2.0 * T * N + es * R * N + 4.0 * R + 2.0 * R * N + 2.0 * T * N             # rows are read once for both directions
        return {"bytes": bytes_, "flops": (8.0 if case["backward"] else 2.0) * R * N}
    active = E * (1.0 - (1.0 - k / E) ** T)
    index = 4.0 * (E + 1 + R)
    if op == "swiglu_down":
        I = case["I"]
        return {"bytes": active * N * I * 0.5625 + R * I * 4.0 + index + 2.0 * R * N, "flops": 2.0 * R * N * I + 6.0 * R * I}
    K = case["K"]
    xrows = T if case["rows"] == "gather" else R
    return {"bytes": (active * N + xrows) * K * 0.5625 + 4.0 * xrows + index + (4.0 if case["fp32"] else 2.0) * R * N,
            "flops": 2.0 * R * N * K}


# ---------------------------------------------------------------- the definitions in 64 bits

_E4M3 = [0.0]          # the non-negative finite codes' values
for _c in range(1, 127):
    _e, _m = _c >> 3, _c & 7
    _E4M3.append((_m / 8.0) * 2.0 ** -6 if _e == 0 else (1 + _m / 8.0) * 2.0 ** (_e - 7))


def _nearest(grid, v):
    """The value of an ascending grid nearest to each |v| up to its last, ties to the even index, by search."""
    grid = torch.tensor(grid, dtype=torch.float64, device=v.device)
    a = v.abs().clamp(max=float(grid[-1]))
    hi = torch.searchsorted(grid, a).clamp_(max=len(grid) - 1)
    lo = (hi - 1).clamp_(min=0)
    up, down = grid[hi] - a, a - grid[lo]
    return torch.copysign(grid[torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)], v)


def _exact_fp8(x):
    q, sc = torch.empty_like(x), x.new_empty(x.shape[0], _blocks(x.shape[1], 128))
    for j in range(sc.shape[1]):
        part = x[:, j * 128:(j + 1) * 128]
        a = part.abs().amax(dim=1, keepdim=True)
        a = torch.where(a == 0, torch.full_like(a, E4M3_MAX), a)
        sc[:, j] = a[:, 0] / E4M3_MAX
        q[:, j * 128:(j + 1) * 128] = _nearest(_E4M3, part * (E4M3_MAX / a))
    return q, sc


def _exact_nvfp4(x):
    """(values, block scales, row scales) of 64-bit rows."""
    a = x.abs().amax(dim=1, keepdim=True)
    s = torch.exp2(torch.ceil(torch.log2(torch.where(a == 0, torch.ones_like(a), a) / 2688.0)))
    s = torch.where(s / 2 >= a / 2688.0, s / 2, torch.where(s < a / 2688.0, s * 2, s))       # log2 next to a power of two
    s = torch.where(a == 0, torch.ones_like(a), s)
    b = x.abs().view(x.shape[0], -1, 16).amax(dim=2)
    e = _nearest(_E4M3, b / (6.0 * s))
    d = (e * s)[:, :, None]
    v = x.view(x.shape[0], -1, 16)
    q = _nearest(_CODES[:8], torch.where(d == 0, torch.zeros_like(v), v / torch.where(d == 0, torch.ones_like(d), d)))
    return (q * d).view(x.shape), e, s[:, 0]


def _exact_norm(s):
    h = s["h"].double()
    if s["delta"] is not None:
        h = (h + s["delta"].double()).to(torch.bfloat16).double()
    return h, h / torch.sqrt((h * h).sum(1, keepdim=True) / s["H"] + EPS) * (1.0 + s["norm_w"].double())


def _exact_silu(gu):
    gu = gu.double()
    I = gu.shape[1] // 2
    return gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]


def _decoded(packed, scales):
    out = torch.empty(packed.shape[0], packed.shape[1] * 2, dtype=torch.float64, device="cuda")
    table = torch.tensor(_CODES, dtype=torch.float64, device="cuda")
    out[:, 0::2], out[:, 1::2] = table[(packed & 15).long()], table[(packed >> 4).long()]
    return (out.view(out.shape[0], -1, 16) * scales.view(torch.float8_e4m3fn).double()[:, :, None]).view(out.shape)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op in ("norm", "norm_dense"):
        h, x = _exact_norm(s)
        if op == "norm":
            return h, (x if case["out"] == "bf16" else _exact_fp8(x))
        return h, _exact_nvfp4(x)[0] @ _decoded(s["w"], s["ws"]).t() * s["wt"].double()
    if op == "quantize":
        return _exact_nvfp4(s["x"].double())
    if op == "swiglu":
        h = _exact_silu(s["gu"])
        return h if case["out"] == "bf16" else _exact_fp8(h)
    if op == "dense":
        y = _decoded(s["x"], s["xs"]) @ _decoded(s["w"], s["ws"]).t()
        return y * s["xr"].double()[:, None] * s["wt"].double()
    T, k, N = case["T"], case["k"], case["N"]
    entries = s["token_list"].long()
    if op == "sort":
        rows = s["x"][entries // k].double()
        y = s["add"].double()
        for lo in range(0, T * k, 4096):          # list positions, a slice at a time
            e = entries[lo:lo + 4096]
            y.index_add_(0, e // k, s["back"][lo:lo + 4096].double() * s["weights"].double().view(-1)[e][:, None])
        if not case["backward"]:
            return rows, None, y
        d_back, d_w = torch.empty(T * k, N, dtype=torch.float64, device="cuda"), torch.empty(T * k, dtype=torch.float64, device="cuda")
        d_x = torch.zeros(T, N, dtype=torch.float64, device="cuda")
        for lo in range(0, T * k, 4096):
            e = entries[lo:lo + 4096]
            dy = s["dy"].double()[e // k]
            d_back[lo:lo + 4096] = dy * s["weights"].double().view(-1)[e][:, None]
            d_w[e] = (dy * s["back"][lo:lo + 4096].double()).sum(1)
            d_x.index_add_(0, e // k, s["d_rows"][lo:lo + 4096].double())
        return rows, None, y, d_back, d_w.view(T, k), d_x
    if op == "swiglu_down":
        x, mode = _exact_nvfp4(_exact_silu(s["gu"]))[0], "scatter"
    else:
        x, mode = _decoded(s["x"], s["xs"]) * s["xr"].double()[:, None], case["rows"]
    y = torch.zeros(T * k, N, dtype=torch.float64, device="cuda")
    off = s["offsets"].tolist()
    for e in range(case["E"]):
        lo, hi = off[e], off[e + 1]
        if hi == lo:
            continue
        here = torch.arange(lo, hi, device="cuda")
        part = torch.arange(N, device="cuda") * s["wt"].shape[1] // N
        src = entries[lo:hi] // k if mode == "gather" else here
        dst = entries[lo:hi] if mode == "scatter" else here
        y[dst] = x[src] @ _decoded(s["w"][e], s["ws"][e]).t() * s["wt"][e].double()[part]
    return y
