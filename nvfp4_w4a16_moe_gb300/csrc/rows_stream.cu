// Products of few rows with one matrix or with each expert's matrix, on the warp-level tensor
// cores: y[o(r), n] = sum_k W[e(r)][n, k] x[i(r), k].
//
// With few rows a call is bound by the bytes of W, so the kernel only has to keep them coming:
//  - A CTA owns 16 rows of one expert's W and up to 8 * NB of the expert's list positions; its
//    warps split K in chunks of 128 bytes of a row. A lane reads whole 16-byte units of W and x
//    straight from global memory into the fragment registers of mma.sync m16n8: the lane in
//    column group c takes units c and 4 + c of a chunk, and the four words of a unit feed two
//    MMAs. This permutes K inside a chunk, in the same way for both operands, so the sum is
//    over the same products; no shared memory or transposition is needed.
//  - The warps' fp32 partial sums are added in warp order in shared memory: the same bits on
//    every run.
//  - 8-bit operands: a chunk is one block of 128, summed from zero in fp32 and added to the
//    running sum times the block's two scales.
// Widths that are no multiple of a chunk read zero units past the end.
#include "common.cuh"
#include "kernels.cuh"

namespace nvfp4 {

namespace {

constexpr int kSWarps = 8;
constexpr int kSThreads = kSWarps * 32;
constexpr int kSAhead = 2;      // chunks of W a lane requests before it uses them

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Pass `p` of the call -> its expert, first list position and rows. Passes are numbered over the
// experts in order, up to kRows positions each. Returns false past the last pass.
template <int kRows>
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
    if ((int)threadIdx.x < P.E) {   // NVFP4_MAX_EXPERTS = kSThreads
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

template <bool FP8, int NB>
__global__ void __launch_bounds__(kSThreads, 2)
rows_stream_kernel(const RowsProduct P, int n_tiles, int k_split) {
    constexpr int kRows = 8 * NB;
    __shared__ float s_acc[kSWarps][16][kRows + 1];
    // row tiles of this CTA: one for every k_split warps
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int k_part = warp & (k_split - 1), n_part = warp / k_split;
    const int pass = blockIdx.x / n_tiles;
    const int n0 = ((blockIdx.x - pass * n_tiles) * (kSWarps / k_split) + n_part) * 16;
    int e, r0, rows;
    if (!locate_pass<kRows>(P, pass, &e, &r0, &rows)) return;

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
    uint4 a[kSAhead][2][2];
    auto load_w = [&](int ch0) {
#pragma unroll
        for (int i = 0; i < kSAhead; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int u = (ch0 + i * k_split) * 8 + 4 * h + c;
                a[i][h][0] = w0 != nullptr && u < units ? ld_once_v4(w0 + u) : zero;
                a[i][h][1] = w1 != nullptr && u < units ? ld_once_v4(w1 + u) : zero;
            }
    };
    load_w(k_part);                                // on its way while the list is read

    const uint4* xr[NB];
    const float* xs[NB][2];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const int row = 8 * b + g < rows ? x_row(P, r0 + 8 * b + g) : -1;
        xr[b] = row < 0 ? nullptr : static_cast<const uint4*>(P.x) + (size_t)row * units;
        if constexpr (FP8) {
            // the rows of this lane's two columns are those of the lanes 4 * column
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int cr = __shfl_sync(0xffffffffu, row, 4 * (2 * c + j));
                xs[b][j] = cr < 0 ? nullptr : P.xs + (size_t)cr * KB;
            }
        }
    }
    const float* wsc = FP8 ? P.ws + ((size_t)e * ((P.N + 127) >> 7) + (min(n0, P.N - 1) >> 7)) * KB : nullptr;

    float acc[NB][4];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[b][i] = 0.f;

    for (int ch0 = k_part; ch0 < chunks; ch0 += k_split * kSAhead) {
#pragma unroll
        for (int i = 0; i < kSAhead; ++i) {
            const int ch = ch0 + i * k_split;
            if (ch >= chunks) break;
            const float sw = FP8 ? wsc[ch] : 0.f;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int u = ch * 8 + 4 * h + c;
                    const uint4 x = xr[b] != nullptr && u < units ? xr[b][u] : zero;
                    const uint4 p = a[i][h][0], q = a[i][h][1];
                    if constexpr (FP8) {
                        mma_e4m3(part, p.x, q.x, p.y, q.y, x.x, x.y);
                        mma_e4m3(part, p.z, q.z, p.w, q.w, x.z, x.w);
                    } else {
                        mma_bf16(acc[b], p.x, q.x, p.y, q.y, x.x, x.y);
                        mma_bf16(acc[b], p.z, q.z, p.w, q.w, x.z, x.w);
                    }
                }
                if constexpr (FP8) {
                    const float s0 = xs[b][0] != nullptr ? xs[b][0][ch] * sw : 0.f;
                    const float s1 = xs[b][1] != nullptr ? xs[b][1][ch] * sw : 0.f;
                    acc[b][0] = fmaf(part[0], s0, acc[b][0]);
                    acc[b][1] = fmaf(part[1], s1, acc[b][1]);
                    acc[b][2] = fmaf(part[2], s0, acc[b][2]);
                    acc[b][3] = fmaf(part[3], s1, acc[b][3]);
                }
            }
        }
        if (ch0 + k_split * kSAhead < chunks) load_w(ch0 + k_split * kSAhead);
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        s_acc[warp][g][8 * b + 2 * c] = acc[b][0];
        s_acc[warp][g][8 * b + 2 * c + 1] = acc[b][1];
        s_acc[warp][g + 8][8 * b + 2 * c] = acc[b][2];
        s_acc[warp][g + 8][8 * b + 2 * c + 1] = acc[b][3];
    }
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

template <bool FP8, int NB>
cudaError_t launch_stream(const RowsProduct& P, cudaStream_t s) {
    constexpr int rows = 8 * NB;
    // warps to a row's K: as many as leave each two chunks, so that short rows share a CTA instead
    const int chunks = (P.K * (FP8 ? 1 : 2) + 127) / 128;
    int k_split = kSWarps;
    while (k_split > 1 && chunks < 2 * k_split) k_split /= 2;
    const int span = kSWarps / k_split * 16, n_tiles = (P.N + span - 1) / span;
    // passes at most: every expert has rows, and its last pass one
    const int groups = std::min(P.R, P.E);
    const long long passes = (P.R - groups) / rows + groups;
    const long long grid = passes * n_tiles;
    if (grid > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
    rows_stream_kernel<FP8, NB><<<(unsigned)grid, kSThreads, 0, s>>>(P, n_tiles, k_split);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rows_stream(const RowsProduct& P, cudaStream_t s) {
    if (P.R <= 8) return P.xs != nullptr ? launch_stream<true, 1>(P, s) : launch_stream<false, 1>(P, s);
    return P.xs != nullptr ? launch_stream<true, 2>(P, s) : launch_stream<false, 2>(P, s);
}

}  // namespace nvfp4
