// Products of few rows with one matrix or with each expert's matrix, on the warp-level tensor
// cores: y[o(r), n] = sum_k W[e(r)][n, k] x[i(r), k].
//
// With few rows a call is bound by the bytes of W, so the kernel only has to keep them coming:
//  - A CTA owns 16 or more rows of one expert's W (below) and up to 8 of the expert's list positions;
//    its warps split K in chunks of 128 bytes of a row. A lane reads whole 16-byte units of W and x
//    straight from global memory into the fragment registers of mma.sync m16n8k16: the lane in
//    column group c takes units c and 4 + c of a chunk, and the words of a unit feed two (bf16) or
//    four MMAs (8-bit). This permutes K inside a chunk, in the same way for both operands, so the sum is
//    over the same products; no shared memory or transposition is needed.
//  - One chunk a warp at a time and four CTAs on an SM: 64 KB of W in flight. A grid that fills the device
//    less than that requests the next chunk before it uses this one (AHEAD: 80 registers, three CTAs). Device
//    time with / without, weights that are not in the L2: one row of 2048 x 8192 in bf16 11.5 / 14.5 us, in
//    8 bits 7.1 / 10.1; on the larger grid of 8 bf16 experts of 1024 x 2048 with a row each 10.4 / 8.1 (in the
//    L2 5.9 / 5.4). With AHEAD the 8-bit kernel spills (48 bytes of stack); it is the faster one all the same.
//  - The warps' fp32 partial sums are added in warp order in shared memory: the same bits on
//    every run.
//  - Rows so short that eight warps would not have two chunks each share a CTA instead: with K = 512 in
//    8 bits the 512 rows of a 64-token batch over 256 experts fell from 147 to 58 us (on this kernel; the tiles
//    take 32).
//  - 8-bit operands are converted to f16, exactly, in registers (as fast as the 8-bit form of mma.sync, or
//    3 % faster). The conversions bound large matrices: one token and 248320 x 2048 takes 93 us, 5.5 TB/s,
//    where bf16 streams the same matrix at 6.6 TB/s, 97 % of the measured copy rate. A chunk is one block
//    of 128, summed from zero in fp32 and added to the running sum times the block's two scales.
// Widths that are no multiple of a chunk read zero units past the end.
#include "common.cuh"
#include "kernels.cuh"

namespace nvfp4 {

namespace {

constexpr int kSWarps = 8;
constexpr int kSThreads = kSWarps * 32;
constexpr int kAheadCtas = 3;        // CTAs on an SM that request a chunk ahead
constexpr int kRows = 8;             // list positions of a pass: the columns of an MMA

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Two E4M3 pairs of a word -> two f16x2 (exact).
__device__ __forceinline__ void e4m3x4_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}"
        : "=r"(lo), "=r"(hi) : "r"(w));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Four k of a lane of two rows of W and one of x, in E4M3.
__device__ __forceinline__ void mma_e4m3_word(float (&d)[4], uint32_t p, uint32_t q, uint32_t x) {
    uint32_t p0, p1, q0, q1, x0, x1;
    e4m3x4_f16(p, p0, p1);
    e4m3x4_f16(q, q0, q1);
    e4m3x4_f16(x, x0, x1);
    mma_f16(d, p0, q0, p1, q1, x0, x1);
}

// Pass `p` of the call -> its expert, first list position and rows. Passes are numbered over the
// experts in order, up to kRows positions each. Returns false past the last pass.
__device__ __forceinline__ bool locate_pass(const RowsProduct& P, int p, int* e, int* r0, int* n) {
    if (P.offsets == nullptr) {
        *e = 0;
        *r0 = p * kRows;
        *n = min(kRows, P.R - *r0);
        return *n > 0;
    }
    __shared__ int s_sum[kSWarps], s_e, s_r0, s_n;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int lo = 0, cnt = 0;
    static_assert(NVFP4_MAX_EXPERTS <= kSThreads, "an expert a thread");
    if ((int)threadIdx.x < P.E) {
        lo = min(max(P.offsets[threadIdx.x], 0), P.R);
        cnt = max(min(max(P.offsets[threadIdx.x + 1], 0), P.R) - lo, 0);
    }
    const int mine = (cnt + kRows - 1) / kRows;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
    }
    if (lane == 31) s_sum[warp] = incl;
    if (threadIdx.x == 0) s_n = 0;
    __syncthreads();
    int before = incl - mine;
#pragma unroll
    for (int w = 0; w < kSWarps; ++w)
        if (w < warp) before += s_sum[w];
    if (p >= before && p < before + mine) {
        s_e = threadIdx.x;
        s_r0 = lo + (p - before) * kRows;
        s_n = min(kRows, cnt - (p - before) * kRows);
    }
    __syncthreads();
    *e = s_e;
    *r0 = s_r0;
    *n = s_n;
    return s_n > 0;
}

template <bool FP8, bool AHEAD>
__global__ void __launch_bounds__(kSThreads, AHEAD ? kAheadCtas : kAheadCtas + 1)
rows_stream_kernel(const RowsProduct P, int n_tiles, int k_split) {
    __shared__ float s_acc[kSWarps][16][kRows + 1];
    pdl_wait_then_trigger();
    // row tiles of this CTA: one for every k_split warps
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int k_part = warp & (k_split - 1), n_part = warp / k_split;
    const int pass = blockIdx.x / n_tiles;
    const int n0 = ((blockIdx.x - pass * n_tiles) * (kSWarps / k_split) + n_part) * 16;
    int e, r0, rows;
    if (!locate_pass(P, pass, &e, &r0, &rows)) return;

    constexpr int kUnit = FP8 ? 16 : 8;            // elements of a 16-byte unit
    const int g = lane >> 2, c = lane & 3;
    const int units = P.K / kUnit;                 // units of a row
    const int chunks = (units + 7) >> 3;
    const int KB = (P.K + 127) >> 7;
    const uint4 zero = make_uint4(0, 0, 0, 0);

    const uint4* w0 = nullptr;
    const uint4* w1 = nullptr;
    {
        const uint4* w = static_cast<const uint4*>(P.w) + ((size_t)e * P.N + n0) * units;
        if (n0 + g < P.N) w0 = w + (size_t)g * units;
        if (n0 + g + 8 < P.N) w1 = w + (size_t)(g + 8) * units;
    }
    uint4 a[2][2];
    auto load_w = [&](int ch, uint4 (&v)[2][2]) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int u = ch * 8 + 4 * h + c;
            v[h][0] = w0 != nullptr && u < units ? ld_once_v4(w0 + u) : zero;
            v[h][1] = w1 != nullptr && u < units ? ld_once_v4(w1 + u) : zero;
        }
    };
    load_w(k_part, a);                             // on its way while the list is read

    const int row = g < rows ? x_row(P, r0 + g) : -1;
    const uint4* xr = row < 0 ? nullptr : static_cast<const uint4*>(P.x) + (size_t)row * units;
    const float* xs[2] = {nullptr, nullptr};
    if constexpr (FP8) {
        // the rows of this lane's two columns are those of the lanes 4 * column
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int cr = __shfl_sync(0xffffffffu, row, 4 * (2 * c + j));
            if (cr >= 0) xs[j] = P.xs + (size_t)cr * KB;
        }
    }
    const float* wsc = FP8 ? P.ws + ((size_t)e * ((P.N + 127) >> 7) + (min(n0, P.N - 1) >> 7)) * KB : nullptr;

    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int ch = k_part; ch < chunks; ch += k_split) {
        uint4 next[2][2];
        if (AHEAD) load_w(ch + k_split, next);
        const float sw = FP8 ? wsc[ch] : 0.f;
        float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int u = ch * 8 + 4 * h + c;
            const uint4 x = xr != nullptr && u < units ? xr[u] : zero;
            const uint4 p = a[h][0], q = a[h][1];
            if constexpr (FP8) {
                mma_e4m3_word(part, p.x, q.x, x.x);
                mma_e4m3_word(part, p.y, q.y, x.y);
                mma_e4m3_word(part, p.z, q.z, x.z);
                mma_e4m3_word(part, p.w, q.w, x.w);
            } else {
                mma_bf16(acc, p.x, q.x, p.y, q.y, x.x, x.y);
                mma_bf16(acc, p.z, q.z, p.w, q.w, x.z, x.w);
            }
        }
        if constexpr (FP8) {
            const float s0 = xs[0] != nullptr ? xs[0][ch] * sw : 0.f;
            const float s1 = xs[1] != nullptr ? xs[1][ch] * sw : 0.f;
            acc[0] = fmaf(part[0], s0, acc[0]);
            acc[1] = fmaf(part[1], s1, acc[1]);
            acc[2] = fmaf(part[2], s0, acc[2]);
            acc[3] = fmaf(part[3], s1, acc[3]);
        }
        if (AHEAD) {
#pragma unroll
            for (int h = 0; h < 2; ++h) a[h][0] = next[h][0], a[h][1] = next[h][1];
        } else if (ch + k_split < chunks) {
            load_w(ch + k_split, a);
        }
    }
    s_acc[warp][g][2 * c] = acc[0];
    s_acc[warp][g][2 * c + 1] = acc[1];
    s_acc[warp][g + 8][2 * c] = acc[2];
    s_acc[warp][g + 8][2 * c + 1] = acc[3];
    __syncthreads();
    // the K parts of a tile are added in order; neighbouring threads write neighbouring outputs
    const int span = kSWarps / k_split * 16, first = (blockIdx.x - pass * n_tiles) * span;
    for (int i = threadIdx.x; i < span * rows; i += kSThreads) {
        const int col = i / span, m = i - col * span;
        if (first + m >= P.N) continue;
        float v = 0.f;
        for (int w = 0; w < k_split; ++w) v += s_acc[(m >> 4) * k_split + w][m & 15][col];
        const int row = y_row(P, r0 + col);
        if (row < 0) continue;
        const size_t at = (size_t)row * P.N + first + m;
        if (P.y_f32) static_cast<float*>(P.y)[at] = v;
        else static_cast<uint16_t*>(P.y)[at] = f32_to_bf16(v);
    }
}

template <bool FP8>
cudaError_t launch_stream(const RowsProduct& P, const DeviceInfo& dev, cudaStream_t s) {
    // warps to a row's K: as many as leave each two chunks, so that short rows share a CTA instead
    const int chunks = (P.K * (FP8 ? 1 : 2) + 127) / 128;
    int k_split = kSWarps;
    while (k_split > 1 && chunks < 2 * k_split) k_split /= 2;
    const int span = kSWarps / k_split * 16, n_tiles = (P.N + span - 1) / span;
    // passes at most: every expert has rows, and its last pass one
    const int groups = std::min(P.R, P.E);
    const long long passes = (P.R - groups) / kRows + groups;
    const long long grid = passes * n_tiles;
    if (grid > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
    if (grid <= kAheadCtas * dev.num_sms)
        return launch_pdl(rows_stream_kernel<FP8, true>, (unsigned)grid, kSThreads, 0, s, P, n_tiles, k_split);
    return launch_pdl(rows_stream_kernel<FP8, false>, (unsigned)grid, kSThreads, 0, s, P, n_tiles, k_split);
}

}  // namespace

cudaError_t launch_rows_stream(const RowsProduct& P, const DeviceInfo& dev, cudaStream_t s) {
    return P.xs != nullptr ? launch_stream<true>(P, dev, s) : launch_stream<false>(P, dev, s);
}

}  // namespace nvfp4
