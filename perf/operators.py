"""Cases of the 8-bit block quantiser, the 8-bit block product and the products grouped by expert.

``run`` computes one pass of an operator: with ``own`` false in elementary torch operations, with
``own`` true through this package's entry points. The sizes are those of the Qwen3.6-35B-A3B-shaped
layer that the tests and the benchmark use (hidden 2048, 256 experts, 8 per token, intermediate 512)
and of its dense 8192 x 2048 projection, with ragged sizes around them.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
BLOCK = 128


def listed():
    return [
        # activations of one prefill call, before an 8-bit product
        dict(name="quantize_rows_4096", op="quantize", batch=1, rows=4096, K=2048, block_rows=1),
        # activations of a small decode batch with a ragged width: latency
        dict(name="quantize_rows_7_ragged", op="quantize", batch=1, rows=7, K=1040, block_rows=1),
        # the down matrices of 64 experts, laid out once when a checkpoint is loaded
        dict(name="quantize_experts_64", op="quantize", batch=64, rows=2048, K=512, block_rows=128),
        # dense projection of one decoded token: latency and weight streaming
        dict(name="fp8_dense_1", op="fp8_dense", T=1, N=8192, K=2048, fp32=False),
        # dense projection of a decode batch, odd sizes, fp32 out (logits of a reduced vocabulary)
        dict(name="fp8_dense_77_odd", op="fp8_dense", T=77, N=5003, K=2000, fp32=True),
        # dense projection of a prefill call
        dict(name="fp8_dense_4096", op="fp8_dense", T=4096, N=8192, K=2048, fp32=False),
        # gate/up of one decoded token: 8 experts with one row each
        dict(name="grouped_bf16_gate_up_1", op="grouped_bf16", T=1, E=256, k=8, N=1024, K=2048, rows="gather", fp32=False),
        # gate/up of a 64-token decode batch: about two rows an expert
        dict(name="grouped_bf16_gate_up_64", op="grouped_bf16", T=64, E=256, k=8, N=1024, K=2048, rows="gather", fp32=False),
        # gate/up of a prefill call
        dict(name="grouped_bf16_gate_up_4096", op="grouped_bf16", T=4096, E=256, k=8, N=1024, K=2048, rows="gather", fp32=False),
        # down of a 64-token decode batch in 8 bits, rows put back into the tokens' order, fp32 for the weighted sum
        dict(name="grouped_fp8_down_64", op="grouped_fp8", T=64, E=256, k=8, N=2048, K=512, rows="scatter", fp32=True),
        # gate/up of a prefill call in 8 bits
        dict(name="grouped_fp8_gate_up_4096", op="grouped_fp8", T=4096, E=256, k=8, N=1024, K=2048, rows="gather", fp32=False),
        # a few large experts with odd widths, rows already in expert order
        dict(name="grouped_fp8_odd_1500", op="grouped_fp8", T=1500, E=17, k=3, N=1111, K=1296, rows="list", fp32=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


_FLOPS = 2.0 * 4096 * 8 * 1024 * 2048      # the largest listed case


def draw(rng):
    op = rng.choice(["quantize", "fp8_dense", "grouped_bf16", "grouped_fp8"])
    if op == "quantize":
        if rng.random() < 0.6:
            return dict(op=op, batch=1, rows=_log(rng, 1, 16384), K=16 * _log(rng, 4, 256), block_rows=1)
        return dict(op=op, batch=_log(rng, 1, 16), rows=_log(rng, 64, 2048), K=16 * _log(rng, 8, 128), block_rows=128)
    if op == "fp8_dense":
        N, K = _log(rng, 128, 8192), 16 * _log(rng, 8, 512)
        T = min(_log(rng, 1, 4096), max(1, int(_FLOPS / (2.0 * N * K))))
        return dict(op=op, T=T, N=N, K=K, fp32=rng.random() < 0.3)
    E, step = _log(rng, 2, 256), 8 if op == "grouped_bf16" else 16
    k = rng.randint(1, min(8, E))
    N, K = _log(rng, 64, 2048), step * _log(rng, 64 // step, 2048 // step)
    T = min(_log(rng, 1, 4096), max(1, int(_FLOPS / (2.0 * N * K * k * 4))))
    return dict(op=op, T=T, E=E, k=k, N=N, K=K, rows=rng.choice(["gather", "scatter", "list"]), fp32=rng.random() < 0.3)


# ---------------------------------------------------------------- inputs

def _blocks(n, size):
    return (n + size - 1) // size


def _spread(v, block_rows, R, K):
    """One value of each block -> one of each element."""
    v = v.repeat_interleave(BLOCK, dim=-1)[..., :K]
    return v if block_rows == 1 else v.repeat_interleave(block_rows, dim=-2)[..., :R, :]


def _block_amax(x, block_rows):
    B, R, K = x.shape
    rb, kb = _blocks(R, block_rows), _blocks(K, BLOCK)
    padded = x.new_zeros(B, rb * block_rows, kb * BLOCK)
    padded[:, :R, :K] = x.abs()
    return padded.view(B, rb, block_rows, kb, BLOCK).amax(dim=(2, 4))


def _quantized(x, block_rows):
    """Codes and scales of bf16 [B, R, K]: scale amax / 448, code nearest to 448 x / amax. In 64 bits:
    the quotient decides between two codes, and ties are exact there."""
    d = x.double()
    amax = _block_amax(d, block_rows)
    scales = torch.where(amax == 0, torch.ones_like(amax), amax / E4M3_MAX).float()
    safe = torch.where(amax == 0, torch.ones_like(amax), amax)
    q = (d * E4M3_MAX / _spread(safe, block_rows, x.shape[1], x.shape[2])).float().to(torch.float8_e4m3fn)
    return q, scales


def _normal(gen, *shape, std=1.0):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.bfloat16) * std


def _tokens(gen, rows, K):
    """Activations with the few large channels that hidden states have."""
    x = _normal(gen, rows, K)
    wide = torch.randint(0, K, (max(1, K // 256),), generator=gen, device="cuda")
    x[:, wide] *= 16.0
    return x


def _quantized_weight(gen, E, N, K):
    """8-bit weights of E matrices, made in slices of a bounded size."""
    q = torch.empty(E, N, K, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty(E, _blocks(N, BLOCK), _blocks(K, BLOCK), dtype=torch.float32, device="cuda")
    step = max(1, (1 << 26) // (N * K))
    for e in range(0, E, step):
        w = _normal(gen, min(step, E - e), N, K, std=0.02)
        amax = _block_amax(w.float(), BLOCK)
        s[e:e + step] = amax / E4M3_MAX
        q[e:e + step] = (w.float() / _spread(s[e:e + step], BLOCK, N, K)).to(torch.float8_e4m3fn)
    return q, s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s = dict(case)
    if case["op"] == "quantize":
        B, R, K = case["batch"], case["rows"], case["K"]
        std = 1.0 if case["block_rows"] == 1 else 0.02
        x = _tokens(gen, B * R, K).view(B, R, K) if std == 1.0 else _normal(gen, B, R, K, std=std)
        s["x"] = x
        s["q"] = torch.empty(B, R, K, dtype=torch.float8_e4m3fn, device="cuda")
        s["scales"] = torch.empty(B, _blocks(R, case["block_rows"]), _blocks(K, BLOCK), device="cuda")
        return s
    out = torch.float32 if case["fp32"] else torch.bfloat16
    T, N, K = case["T"], case["N"], case["K"]
    if case["op"] == "fp8_dense":
        q, xs = _quantized(_tokens(gen, T, K)[None], 1)
        w, ws = _quantized_weight(gen, 1, N, K)
        s.update(x=q[0], xs=xs[0], w=w[0], ws=ws[0], y=torch.empty(T, N, dtype=out, device="cuda"))
        return s
    # top-k routing of random logits, some experts more popular than others; entries t*k + j in expert order
    E, k = case["E"], case["k"]
    logits = torch.randn(T, E, generator=gen, device="cuda") + 0.5 * torch.randn(E, generator=gen, device="cuda")
    ids = logits.topk(k, dim=1).indices.reshape(-1)
    order = torch.argsort(ids, stable=True)
    counts = torch.bincount(ids, minlength=E)
    s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    s["token_list"] = order.to(torch.int32)
    s["most"] = int(counts.max())
    x = _tokens(gen, T if case["rows"] == "gather" else T * k, K)
    if case["op"] == "grouped_bf16":
        s.update(x=x, w=_normal(gen, E, N, K, std=0.02))
    else:
        q, xs = _quantized(x[None], 1)
        w, ws = _quantized_weight(gen, E, N, K)
        s.update(x=q[0], xs=xs[0], w=w, ws=ws)
    s["y"] = torch.empty(T * k, N, dtype=out, device="cuda")
    return s


# ---------------------------------------------------------------- one pass

def _rows_of(s):
    """x row, y row and expert of every list position."""
    R = s["T"] * s["k"]
    r = torch.arange(R, device="cuda")
    entry = s["token_list"].long()
    expert = torch.searchsorted(s["offsets"].long(), r, right=True) - 1
    return (entry // s["k"] if s["rows"] == "gather" else r), (entry if s["rows"] == "scatter" else r), expert


def _plain_grouped(s):
    src, dst, expert = _rows_of(s)
    R, N, K = s["T"] * s["k"], s["N"], s["K"]
    x, w = s["x"].float(), s["w"]
    if "xs" in s:
        x = x * _spread(s["xs"], 1, 0, K)
    x = x[src]
    if R <= s["E"]:        # few rows: each with its expert's matrix
        m = w[expert].float() if "ws" not in s else w.view(torch.uint8)[expert].view(w.dtype).float() * _spread(s["ws"][expert], BLOCK, N, K)
        rows = torch.bmm(m, x[:, :, None])[:, :, 0]
    else:                  # the experts' rows padded to the longest
        m = w.float() if "ws" not in s else w.float() * _spread(s["ws"], BLOCK, N, K)
        at = torch.arange(R, device="cuda") - s["offsets"].long()[expert]
        padded = x.new_zeros(s["E"], s["most"], K)
        padded[expert, at] = x
        rows = torch.bmm(padded, m.transpose(1, 2))[expert, at]
    y = torch.empty_like(rows)
    y[dst] = rows
    return y.to(s["y"].dtype)


def run(s):
    if own:
        import nvfp4_w4a16_moe_gb300 as nv
        if s["op"] == "quantize":
            return nv.fp8_quantize_block128(s["x"], s["block_rows"], q=s["q"], scales=s["scales"])
        if s["op"] == "fp8_dense":
            return nv.fp8_gemm_block128(s["x"], s["xs"], s["w"], s["ws"], y=s["y"])
        rows = dict(token_list=None if s["rows"] == "list" else s["token_list"], k=s["k"],
                    gather=s["rows"] == "gather", scatter=s["rows"] == "scatter", y=s["y"])
        if s["op"] == "grouped_bf16":
            return nv.moe_grouped_gemm_bf16(s["x"], s["w"], s["offsets"], **rows)
        return nv.moe_grouped_gemm_fp8(s["x"], s["xs"], s["w"], s["ws"], s["offsets"], **rows)
    if s["op"] == "quantize":
        return _quantized(s["x"], s["block_rows"])
    if s["op"] == "fp8_dense":
        x = s["x"].float() * _spread(s["xs"], 1, 0, s["K"])
        w = s["w"].float() * _spread(s["ws"], BLOCK, s["N"], s["K"])
        return (x @ w.t()).to(s["y"].dtype)
    return _plain_grouped(s)


def work(case):
    """Every input once and every output once. For the grouped products the matrices of the experts that
    an even routing of so many tokens reaches."""
    if case["op"] == "quantize":
        n = case["batch"] * case["rows"] * case["K"]
        b = case["batch"] * _blocks(case["rows"], case["block_rows"]) * _blocks(case["K"], BLOCK)
        return {"bytes": 3.0 * n + 4.0 * b, "flops": 2.0 * n}
    T, N, K, out = case["T"], case["N"], case["K"], 4.0 if case["fp32"] else 2.0
    kb, nb = _blocks(K, BLOCK), _blocks(N, BLOCK)
    if case["op"] == "fp8_dense":
        return {"bytes": T * K + N * K + 4.0 * (T * kb + nb * kb) + out * T * N, "flops": 2.0 * T * N * K}
    E, k = case["E"], case["k"]
    R = T * k
    active = E * (1.0 - (1.0 - k / E) ** T)
    xrows = T if case["rows"] == "gather" else R
    index = 4.0 * (E + 1 + (0 if case["rows"] == "list" else R))
    each = 2.0 * K if case["op"] == "grouped_bf16" else K + 4.0 * kb
    matrix = 2.0 * N * K if case["op"] == "grouped_bf16" else N * K + 4.0 * nb * kb
    return {"bytes": active * matrix + xrows * each + index + out * R * N, "flops": 2.0 * R * N * K}


# ---------------------------------------------------------------- the definition in 64 bits

_E4M3 = [0.0]          # the non-negative finite codes' values
for _c in range(1, 127):
    _e, _m = _c >> 3, _c & 7
    _E4M3.append((_m / 8.0) * 2.0 ** -6 if _e == 0 else (1 + _m / 8.0) * 2.0 ** (_e - 7))


def _nearest_e4m3(v):
    """The E4M3 value nearest to each |v| <= 448, ties to the even code, by search among the values."""
    grid = torch.tensor(_E4M3, dtype=torch.float64, device=v.device)
    a = v.abs()
    hi = torch.searchsorted(grid, a).clamp_(max=126)
    lo = (hi - 1).clamp_(min=0)
    up, down = grid[hi] - a, a - grid[lo]
    pick = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return torch.copysign(grid[pick], v)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        B, R, K = s["x"].shape
        br = case["block_rows"]
        q = torch.empty(B, R, K, dtype=torch.float64, device="cuda")
        sc = torch.empty(B, _blocks(R, br), _blocks(K, BLOCK), dtype=torch.float64, device="cuda")
        for j in range(_blocks(K, BLOCK)):
            part = s["x"][:, :, j * BLOCK:(j + 1) * BLOCK].double()
            step = R if br == 1 else br
            for i in range(0, R, step):
                p = part[:, i:i + step]
                a = p.abs().amax(dim=2, keepdim=True) if br == 1 else p.abs().amax(dim=(1, 2), keepdim=True)
                one = torch.where(a == 0, torch.full_like(a, E4M3_MAX), a)
                q[:, i:i + step, j * BLOCK:(j + 1) * BLOCK] = _nearest_e4m3(p * E4M3_MAX / one)
                if br == 1:
                    sc[:, :, j] = one[:, :, 0] / E4M3_MAX
                else:
                    sc[:, i // br, j] = one[:, 0, 0] / E4M3_MAX
        return q, sc
    K, N = case["K"], case["N"]

    def product(x, xs, w, ws):
        """Sums of whole blocks, each times its two scales."""
        y = torch.zeros(x.shape[0], N, dtype=torch.float64, device="cuda")
        col = torch.arange(N, device="cuda") // BLOCK
        for b in range(_blocks(K, BLOCK)):
            at = slice(b * BLOCK, (b + 1) * BLOCK)
            y += (x[:, at].double() @ w[:, at].double().t()) * xs[:, b:b + 1].double() * ws[col, b].double()
        return y

    if case["op"] == "fp8_dense":
        return product(s["x"], s["xs"], s["w"], s["ws"])
    y = torch.zeros(case["T"] * case["k"], N, dtype=torch.float64, device="cuda")
    off, entries = s["offsets"].tolist(), s["token_list"].long()
    for e in range(case["E"]):
        lo, hi = off[e], off[e + 1]
        if hi == lo:
            continue
        here = torch.arange(lo, hi, device="cuda")
        src = entries[lo:hi] // case["k"] if case["rows"] == "gather" else here
        dst = entries[lo:hi] if case["rows"] == "scatter" else here
        if case["op"] == "grouped_bf16":
            y[dst] = s["x"][src].double() @ s["w"][e].double().t()
        else:
            y[dst] = product(s["x"].view(torch.uint8)[src].view(torch.float8_e4m3fn), s["xs"][src], s["w"][e], s["ws"][e])
    return y
