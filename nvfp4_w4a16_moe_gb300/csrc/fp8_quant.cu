// Block quantiser of the 8-bit products: bf16 -> E4M3 codes with one fp32 scale per block of
// 1 x 128 (rows of activations) or 128 x 128 elements (weights).
//
//   a = max |x| over the block,  scale = fl32(a / 448)  (1 where a = 0),
//   code = the E4M3 value nearest to 448 x / a, ties to even.
//
// The nearest value is found without a division per element. x and a are bf16 (8 significant
// bits m_x, m_a <= 255), a point where the rounding changes is j * 2^c with j odd and below 32,
// so 448 x / a = 7 (m_x / m_a) 2^d either equals such a point or is off it by a relative
//   |7 m_x 2^d' - j m_a| / (j m_a) >= 1 / (31 * 255) > 2^-13.
// p = fl(x * fl(448 / a)) is within 2^-22 of the quotient; rounding p to 16 significant bits
// (an add and a mask on its bits) puts it back on the point where the quotient is on one, and
// moves it by less than 2^-16 otherwise, so the conversion of that value is the exact one.
//
// Bound: HBM, 2 bytes read and 1 written per element, one pass: each block stays in registers
// between its maximum and its codes.
#include <type_traits>

#include "common.cuh"
#include "kernels.cuh"
#include "quant.cuh"

namespace nvfp4 {

namespace {

constexpr int kQThreads = 256;
// Fewer blocks than this: one pair of blocks a warp and short latency (us, 1 against 4 pairs: 1 x 2048 1.6 / 1.9,
// 512 x 2048 2.3 / 2.4); more: four pairs, whose divisions are done together (4096 x 2048 6.3 / 5.3, 262144 x 2048
// 351 / 251, 6.4 TB/s).
constexpr size_t kFewBlocks = 1u << 14;

// Larger of two |x| as fp32 bits: NaN above infinity above every number, so a NaN is kept.
__device__ __forceinline__ uint32_t absmax8(const uint4 v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m = max(m, (w[i] << 16) & 0x7FFFFFFFu);
        m = max(m, w[i] & 0x7FFF0000u);
    }
    return m;
}

// Eight bf16 of a block with this amax -> eight codes.
__device__ __forceinline__ uint2 quantize8(const uint4 v, uint32_t amax_bits, float inv) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if (__uint_as_float(amax_bits) < kTinyAmax) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = (uint32_t)f32_to_bf16(bf16lo(w[i]) * 0x1p64f) | ((uint32_t)f32_to_bf16(bf16hi(w[i]) * 0x1p64f) << 16);
    }
    const uint32_t half = amax_bits < 0x7F800000u ? 0x80u : 0u;
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = e4m3x2(snap16(bf16lo(w[i]) * inv, half), snap16(bf16hi(w[i]) * inv, half));
    return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

// 1 x 128 blocks: 16 lanes hold one block, a warp takes kUnroll pairs of neighbouring blocks.
// WHOLE: K is a multiple of 128, the blocks follow one another without a gap.
template <int kUnroll, bool WHOLE>
__global__ void __launch_bounds__(kQThreads)
quantize_rows_kernel(const uint16_t* x, size_t blocks, int K, unsigned KB, uint8_t* q, float* scales) {
    pdl_wait_then_trigger();
    const int lane = threadIdx.x & 31, unit = lane & 15, half = lane >> 4;
    const size_t warp = (size_t)blockIdx.x * (kQThreads / 32) + (threadIdx.x >> 5);
    const size_t first = warp * (2 * kUnroll) + half;
    uint4 v[kUnroll];
    size_t at[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const size_t blk = first + 2 * u;
        v[u] = make_uint4(0, 0, 0, 0);
        at[u] = ~size_t(0);
        if (blk < blocks) {
            if (WHOLE) {
                at[u] = blk * 128 + unit * 8;
            } else {
                // 32-bit division where the numbers allow it
                const size_t row = blocks >> 32 ? blk / KB : (size_t)((unsigned)blk / KB);
                const int col = (int)(blk - row * KB) * 128 + unit * 8;
                if (col < K) at[u] = row * K + col;
            }
            if (at[u] != ~size_t(0)) v[u] = ld_once_v4(x + at[u]);
        }
    }
    // lane u of a half warp keeps the maximum of block u, so that the divisions are done once for all blocks
    uint32_t m[kUnroll], mine = 0;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        m[u] = absmax8(v[u]);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m[u] = max(m[u], __shfl_xor_sync(0xffffffffu, m[u], o));
        if (unit == u) mine = m[u];
    }
    const float inv = block_inverse(mine);
    if (unit < kUnroll && first + 2 * unit < blocks) scales[first + 2 * unit] = block_scale(mine);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const float iu = __shfl_sync(0xffffffffu, inv, u, 16);
        if (at[u] != ~size_t(0)) *reinterpret_cast<uint2*>(q + at[u]) = quantize8(v[u], m[u], iu);
    }
}

// 128 x 128 blocks: one CTA per block, which it keeps in registers (eight 16-byte units a thread).
__global__ void __launch_bounds__(kQThreads)
quantize_tiles_kernel(const uint16_t* x, int R, int K, int RB, int KB, uint8_t* q,
                      float* scales) {
    __shared__ uint32_t s_max[kQThreads / 32];
    pdl_wait_then_trigger();
    const size_t blk = blockIdx.x;
    const size_t mat = blk / ((size_t)RB * KB);
    const int in = (int)(blk - mat * ((size_t)RB * KB));
    const int rb = in / KB, kb = in - rb * KB;
    const int col = kb * 128 + (threadIdx.x & 15) * 8, row0 = rb * 128 + (threadIdx.x >> 4);
    const size_t base = (mat * R + row0) * K + col;
    uint4 v[8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i] = make_uint4(0, 0, 0, 0);
        if (col < K && row0 + 16 * i < R) v[i] = ld_once_v4(x + base + (size_t)16 * i * K);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, absmax8(v[i]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kQThreads / 32; ++i) m = max(m, s_max[i]);
    const float inv = block_inverse(m);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (col < K && row0 + 16 * i < R)
            *reinterpret_cast<uint2*>(q + base + (size_t)16 * i * K) = quantize8(v[i], m, inv);
    if (threadIdx.x == 0) scales[blk] = block_scale(m);
}

}  // namespace

cudaError_t launch_fp8_quantize(const uint16_t* x, int B, int R, int K, int block_rows, uint8_t* q, float* scales,
                                cudaStream_t s) {
    const int KB = (K + 127) / 128;
    if (block_rows == 1) {
        const size_t blocks = (size_t)B * R * KB;
        auto run = [&](auto unroll) -> cudaError_t {
            constexpr int kUnroll = decltype(unroll)::value;
            const size_t per = (kQThreads / 32) * 2 * kUnroll;
            if ((blocks + per - 1) / per > 0x7FFFFFFFu) return cudaErrorInvalidConfiguration;
            const unsigned grid = (unsigned)((blocks + per - 1) / per);
            if (K % 128 == 0)
                return launch_pdl(quantize_rows_kernel<kUnroll, true>, grid, kQThreads, 0, s, x, blocks, K, KB, q, scales);
            return launch_pdl(quantize_rows_kernel<kUnroll, false>, grid, kQThreads, 0, s, x, blocks, K, KB, q, scales);
        };
        return blocks < kFewBlocks ? run(std::integral_constant<int, 1>{}) : run(std::integral_constant<int, 4>{});
    }
    const int RB = (R + 127) / 128;
    const size_t blocks = (size_t)B * RB * KB;
    if (blocks > 0x7FFFFFFFu) return cudaErrorInvalidConfiguration;
    return launch_pdl(quantize_tiles_kernel, (unsigned)blocks, kQThreads, 0, s, x, R, K, RB, KB, q, scales);
}

}  // namespace nvfp4
