// Operators on rows that end in rows of a product: NVFP4 quantisation, the RMSNorm with the residual add, the
// SwiGLU, each written in bf16, in E4M3 blocks of 1 x 128 or as NVFP4 rows; and NVFP4 rows back.
//
//   norm     h' = bf16(h + delta), x = h' / sqrt(mean h'^2 + eps) * (1 + w)
//   SwiGLU   x = g / (1 + exp(-g)) * u
//   E4M3     scale = amax / 448 of 128, code nearest to 448 x / amax
//   NVFP4    s = the power of two >= amax / 2688 of the row, e = E4M3(amax / (6 s)) of 16, code = E2M1(x / (e s))
//
// A group of threads holds a row in registers (fp32, eight neighbouring elements a thread and unit) from its one
// read to its one write. How a row is split over threads depends on its length alone, so a row's result does not
// depend on the others. The sums and maxima over a row go over the lanes by shuffles, then over the warps in order.
//
// Bound: HBM, 2 to 8 bytes read and 0.56 to 4 written per element; from launch to the first bytes pass some 1.5 us (5 x
// 1000 takes 1.6). us of 4096 x 2048 / 65536 x 2048, and of the latter's bytes at the copy rate (6.8 TB/s): norm with
// delta to bf16 11.8 / 155 (158), to E4M3 12.4 / 152 (139), to NVFP4 11.8 / 148 (129); SwiGLU 7.7 / 114 (118), 9.6 / 122
// (99), 9.9 / 126 (90); quantise 6.6 / 72 (51); back 5.6 / 68 (51). Where rows end in 4 bits the instructions of the blocks
// (a maximum, a scale and its reciprocal, 16 codes) bound it: 82 % of the issue slots and 77 % of the integer pipe are
// used in the quantiser, 86 % and 65 % in the SwiGLU.
#include "common.cuh"
#include "kernels.cuh"
#include "quant.cuh"

namespace nvfp4 {

namespace {

constexpr int kRowThreads = 128;      // of a CTA, or one row's threads where those are more

enum RowSource { kPlain, kNorm, kNormDelta, kSwiglu16, kSwiglu32 };

struct RowParams {
    const void* in;            // x / h / gu
    const uint16_t* delta;
    const uint16_t* w;
    uint16_t* h_out;
    float eps;
    int R, K, group;           // threads of a row
    nvfp4_rows out;
};

__device__ __forceinline__ void unpack8(const uint4 u, float (&v)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = bf16lo(w[i]), v[2 * i + 1] = bf16hi(w[i]);
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
    return make_uint4(w[0], w[1], w[2], w[3]);
}
// Eight elements as they lie in memory (16-byte aligned), or zeros: asked for without a branch, so that many are under way.
template <bool F32>
struct Raw8 {
    uint4 a, b;

    __device__ __forceinline__ void ask(const void* base, size_t at, bool there) {
        const uint8_t* p = static_cast<const uint8_t*>(base) + at * (F32 ? 4 : 2);
        a = ld_if(p, there);
        if (F32) b = ld_if(p + 16, there);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        if constexpr (F32) {
            v[0] = __uint_as_float(a.x), v[1] = __uint_as_float(a.y), v[2] = __uint_as_float(a.z), v[3] = __uint_as_float(a.w);
            v[4] = __uint_as_float(b.x), v[5] = __uint_as_float(b.y), v[6] = __uint_as_float(b.z), v[7] = __uint_as_float(b.w);
        } else {
            unpack8(a, v);
        }
    }
    static __device__ __forceinline__ uint4 ld_if(const void* p, bool there) {
        uint4 v = make_uint4(0, 0, 0, 0);
        asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %5, 0;\n"
                     " @p ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n}"
                     : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w) : "l"(p), "r"((uint32_t)there));
        return v;
    }
};
// Largest |v| as fp32 bits: NaN above infinity above every number.
__device__ __forceinline__ uint32_t absmax8(const float (&v)[8]) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; i += 2) asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(v[i]), "f"(v[i + 1]));
    return __float_as_uint(m) & 0x7FFFFFFFu;
}

// g / (1 + exp(-g)), for g < 0 as g exp(g) / (1 + exp(g)): exp(-g) passes fp32 from g = -88.7 down, where the quotient is
// still a normal number to -92. Digits go with those of a subnormal exp(g), all of them below -104.
__device__ __forceinline__ float silu(float g) {
    const float e = __expf(-fabsf(g));
    return __fdividef(g < 0.f ? g * e : g, 1.0f + e);
}

// Over the threads of a row; s: one word a warp. All threads of the CTA call it.
__device__ __forceinline__ float row_sum(float v, int group, float* s) {
    const int warp = threadIdx.x >> 5, warps = group >> 5, first = warp / warps * warps;
    v = warp_sum(v);
    if (warps == 1) return v;
    if ((threadIdx.x & 31) == 0) s[warp] = v;
    __syncthreads();
    v = 0.f;
    for (int i = 0; i < warps; ++i) v += s[first + i];
    return v;
}
__device__ __forceinline__ uint32_t row_max(uint32_t v, int group, uint32_t* s) {
    const int warp = threadIdx.x >> 5, warps = group >> 5, first = warp / warps * warps;
    v = __reduce_max_sync(0xffffffffu, v);
    if (warps == 1) return v;
    if ((threadIdx.x & 31) == 0) s[warp] = v;
    __syncthreads();
    for (int i = 0; i < warps; ++i) v = max(v, s[first + i]);
    return v;
}

template <int SRC, int OUT, int U>
__global__ void __launch_bounds__(U >= 4 ? NVFP4_MAX_ROW_K / 64 : kRowThreads)
rows_kernel(const RowParams P) {
    __shared__ float s_sum[32];
    __shared__ uint32_t s_max[32];
    pdl_wait_then_trigger();
    const int group = P.group, lane = threadIdx.x % group, units = P.K >> 3;
    const size_t row = (size_t)blockIdx.x * (blockDim.x / group) + threadIdx.x / group;
    const bool here = row < (size_t)P.R;
    constexpr bool norm = SRC == kNorm || SRC == kNormDelta, two = SRC != kPlain && SRC != kNorm, f32 = SRC == kSwiglu32;
    Raw8<f32> in[U], in2[two ? U : 1];       // x / h / g, and delta / u
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int unit = lane + u * group;
        const bool there = here && unit < units;
        const size_t at = row * P.K + unit * 8, wide = at + row * P.K;
        in[u].ask(P.in, SRC == kSwiglu16 || f32 ? wide : at, there);
        if (SRC == kNormDelta) in2[u].ask(P.delta, at, there);
        if (SRC == kSwiglu16 || f32) in2[u].ask(P.in, wide + P.K, there);
    }
    float v[U][8];
    float ss = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int unit = lane + u * group;
        in[u].get(v[u]);
        if constexpr (SRC == kNormDelta) {
            float d[8];
            in2[u].get(d);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[u][i] += d[i];
            in[u].a = pack8(v[u]);
            unpack8(in[u].a, v[u]);             // the residual stream is bf16: the norm sees what is stored
        }
        if constexpr (norm) {
            if (P.h_out != nullptr && here && unit < units)
                *reinterpret_cast<uint4*>(P.h_out + row * P.K + unit * 8) = in[u].a;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(v[u][i], v[u][i], ss);
        }
        if constexpr (SRC == kSwiglu16 || f32) {
            float up[8];
            in2[u].get(up);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[u][i] = silu(v[u][i]) * up[i];
        }
    }
    if constexpr (norm) {
        Raw8<false> w[U];
#pragma unroll
        for (int u = 0; u < U; ++u) w[u].a = Raw8<false>::ld_if(P.w + (lane + u * group) * 8, lane + u * group < units);
        const float r = 1.0f / sqrtf(row_sum(ss, group, s_sum) / (float)P.K + P.eps);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float g[8];
            w[u].get(g);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[u][i] = v[u][i] * r * (1.0f + g[i]);
        }
    }
    if constexpr (OUT == NVFP4_ROWS_BF16) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int unit = lane + u * group;
            if (here && unit < units)
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(P.out.data) + row * P.K + unit * 8) = pack8(v[u]);
        }
    } else if constexpr (OUT == NVFP4_ROWS_FP8) {
        // sixteen neighbouring lanes hold a block
        const int KB = (P.K + 127) >> 7;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int unit = lane + u * group;
            uint32_t m = absmax8(v[u]);
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
            if (!here || unit >= units) continue;
            // a / 448 and 448 / a as the quantiser of bf16 rows has them; the codes are those of fl32(x (448 / a))
            const float inv = block_inverse(m);
            if ((unit & 15) == 0) static_cast<float*>(P.out.scales)[row * KB + (unit >> 4)] = block_scale(m);
            if (__uint_as_float(m) < kTinyAmax)
#pragma unroll
                for (int i = 0; i < 8; ++i) v[u][i] *= 0x1p64f;
#pragma unroll
            for (int i = 0; i < 8; i += 2) mul2(v[u][i], v[u][i + 1], inv);
            uint32_t h[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) h[i] = e4m3x2(v[u][2 * i], v[u][2 * i + 1]);
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(P.out.data) + row * P.K + unit * 8) =
                make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
        }
    } else {
        uint32_t m[U], all = 0;
#pragma unroll
        for (int u = 0; u < U; ++u) all = max(all, m[u] = absmax8(v[u]));
        all = row_max(all, group, s_max);
        const float s = row_scale(all);
        const bool finite = all < 0x7F800000u;
        float is = finite ? inverse_pow2(s) : 0.f;
        if (is > 0x1p100f) {              // 1 / (e s) would not be a number: bring the row up first, exactly
            is *= 0x1p-64f;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                m[u] = m[u] == 0u ? 0u : __float_as_uint(__uint_as_float(m[u]) * 0x1p64f);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[u][i] *= 0x1p64f;
            }
        }
        if (here && lane == 0) P.out.row_scales[row] = s;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int unit = lane + u * group;
            m[u] = max(m[u], __shfl_xor_sync(0xffffffffu, m[u], 1));     // two lanes hold a block of 16
            if (!here || unit >= units) continue;
            float inv;
            const uint32_t e = nvfp4_block_scale<SRC == kPlain>(finite ? __uint_as_float(m[u]) * is : 0.f, &inv);
            const size_t at = row * (P.K >> 3) + unit;
            static_cast<uint32_t*>(P.out.data)[at] = nvfp4_codes8<SRC == kPlain>(v[u], inv * is);
            if ((unit & 1) == 0) static_cast<uint8_t*>(P.out.scales)[at >> 1] = (uint8_t)e;
        }
    }
}

template <int SRC, int OUT, int U>
cudaError_t launch_u(RowParams P, cudaStream_t s) {
    const int units = P.K >> 3;
    P.group = ((units + U - 1) / U + 31) / 32 * 32;
    const int threads = P.group > kRowThreads ? P.group : kRowThreads / P.group * P.group;
    const int per = threads / P.group;
    return launch_pdl(rows_kernel<SRC, OUT, U>, (unsigned)(((long long)P.R + per - 1) / per), threads, 0, s, P);
}

// Up to 1024 columns: a warp a row, no barriers. More: four units a thread in the quantiser, two where a norm's sum stands
// between reading and writing or an exponential is to be taken (us, two / four units a thread: quantiser of 65536 x 2048
// 85 / 72; norm of it into bf16 154 / 156, E4M3 153 / 168, NVFP4 149 / 145; SwiGLU 114 / 114, 122 / 125, 126 / 125; 7 x 1056
// norm 1.6 / 1.8, SwiGLU into E4M3 1.6 / 2.3). The rule goes by the columns alone, so that a row's sum does not depend on
// how many rows there are.
template <int SRC, int OUT>
cudaError_t launch_rows(const RowParams& P, cudaStream_t s) {
    const int units = P.K >> 3;
    if (units <= 32) return launch_u<SRC, OUT, 1>(P, s);
    if (units <= (SRC == kPlain ? 64 : 2 * kRowThreads)) return launch_u<SRC, OUT, 2>(P, s);
    if (units <= NVFP4_MAX_ROW_K / 16) return launch_u<SRC, OUT, 4>(P, s);
    return launch_u<SRC, OUT, 8>(P, s);
}

template <int SRC>
cudaError_t launch_kind(const RowParams& P, cudaStream_t s) {
    if (P.out.kind == NVFP4_ROWS_BF16) return launch_rows<SRC, NVFP4_ROWS_BF16>(P, s);
    if (P.out.kind == NVFP4_ROWS_FP8) return launch_rows<SRC, NVFP4_ROWS_FP8>(P, s);
    return launch_rows<SRC, NVFP4_ROWS_NVFP4>(P, s);
}

// One block of 16 elements a thread. bf16 leaves the caches first (32768 x 512: 11.2 us, so 9.8).
template <bool F32>
__global__ void __launch_bounds__(256)
dequantize_rows_kernel(const uint8_t* packed, const uint8_t* scales, const float* scale, int scale_rows, size_t blocks,
                       int KB, void* y) {
    pdl_wait_then_trigger();
    const size_t b = (size_t)blockIdx.x * 256 + threadIdx.x;
    if (b >= blocks) return;
    const size_t row = b / KB;
    const uint2 c = *reinterpret_cast<const uint2*>(packed + b * 8);
    const float e = e4m3_to_f32(scales[b]), s = scale[row / scale_rows];
    float v[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 f = e2m1x2_to_f32x2((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
        v[2 * i] = f.x * e * s, v[2 * i + 1] = f.y * e * s;
    }
    if constexpr (F32) {
        float4* o = reinterpret_cast<float4*>(static_cast<float*>(y) + b * 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    } else {
        uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(y) + b * 16);
        __stcs(o, pack8(*reinterpret_cast<const float(*)[8]>(v)));
        __stcs(o + 1, pack8(*reinterpret_cast<const float(*)[8]>(v + 8)));
    }
}

}  // namespace

cudaError_t launch_quantize_rows(const uint16_t* x, int R, int K, const nvfp4_rows& out, cudaStream_t s) {
    RowParams P{};
    P.in = x, P.R = R, P.K = K, P.out = out;
    return launch_rows<kPlain, NVFP4_ROWS_NVFP4>(P, s);
}

cudaError_t launch_norm_rows(const uint16_t* h, const uint16_t* delta, const uint16_t* w, float eps, int T, int H,
                             uint16_t* h_out, const nvfp4_rows& out, cudaStream_t s) {
    RowParams P{};
    P.in = h, P.delta = delta, P.w = w, P.h_out = h_out == h ? (delta ? h_out : nullptr) : h_out, P.eps = eps;
    P.R = T, P.K = H, P.out = out;
    return delta != nullptr ? launch_kind<kNormDelta>(P, s) : launch_kind<kNorm>(P, s);
}

cudaError_t launch_swiglu_rows(const void* gu, bool f32, int R, int I, const nvfp4_rows& out, cudaStream_t s) {
    RowParams P{};
    P.in = gu, P.R = R, P.K = I, P.out = out;
    return f32 ? launch_kind<kSwiglu32>(P, s) : launch_kind<kSwiglu16>(P, s);
}

cudaError_t launch_dequantize_rows(const uint8_t* packed, const uint8_t* scales, const float* scale, int scale_rows,
                                   int R, int K, void* y, bool f32, cudaStream_t s) {
    const size_t blocks = (size_t)R * (K / 16);
    if ((blocks + 255) / 256 > 0x7FFFFFFFu) return cudaErrorInvalidConfiguration;
    const unsigned grid = (unsigned)((blocks + 255) / 256);
    if (f32) return launch_pdl(dequantize_rows_kernel<true>, grid, 256, 0, s, packed, scales, scale, scale_rows, blocks, K / 16, y);
    return launch_pdl(dequantize_rows_kernel<false>, grid, 256, 0, s, packed, scales, scale, scale_rows, blocks, K / 16, y);
}

}  // namespace nvfp4
