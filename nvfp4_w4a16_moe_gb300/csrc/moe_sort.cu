// Rows sorted by expert and back, and the gradients.
//
//   permute   rows[r] = x[list[r] / k],  positions[list[r]] = r
//   combine   y[t] = add[t] + sum_j w[t,j] rows[positions[t k + j]]
//   backward  d_rows[p] = w[t,j] dy[t],  d_w[t,j] = <dy[t], rows[p]>,  p = positions[t k + j]
//
// Sums are fp32, in the order of j (combine) or in a fixed order over threads, warps and the warps' partial sums
// (d_w): the same bits on every run, no atomics. A token's output has one owner.
//
// Bound: HBM. A row is read once and written once: T * k * N elements either way.
#include "common.cuh"
#include "kernels.cuh"

namespace nvfp4 {

namespace {

constexpr int kSortThreads = 256;
constexpr int kAhead = 8;          // rows of a token requested together

// Eight columns of a row that starts at `row`. WIDE: neighbouring ones, from 8 * unit on, rows 16-byte aligned.
// Otherwise (N not a multiple of 8) columns unit / 32 * 256 + unit % 32 + 32 i, so that a warp's loads are of
// neighbouring elements at any alignment.
template <bool WIDE>
__device__ __forceinline__ int column(int unit, int i) {
    return WIDE ? unit * 8 + i : (unit >> 5) * 256 + (unit & 31) + 32 * i;
}
template <bool F32, bool WIDE>
__device__ __forceinline__ void get8(const void* base, size_t row, int N, int unit, float (&v)[8]) {
    if constexpr (WIDE && F32) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + row * N + unit * 8);
        const float4 a = p[0], b = p[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else if constexpr (WIDE) {
        const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + row * N + unit * 8);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) v[2 * i] = bf16lo(w[i]), v[2 * i + 1] = bf16hi(w[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = column<false>(unit, i);
            v[i] = 0.f;
            if (c < N)
                v[i] = F32 ? static_cast<const float*>(base)[row * N + c]
                           : bf16_to_f32(static_cast<const uint16_t*>(base)[row * N + c]);
        }
    }
}
template <bool F32, bool WIDE>
__device__ __forceinline__ void put8(void* base, size_t row, int N, int unit, const float (&v)[8]) {
    if constexpr (WIDE && F32) {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + row * N + unit * 8);
        p[0] = make_float4(v[0], v[1], v[2], v[3]);
        p[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else if constexpr (WIDE) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + row * N + unit * 8) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int c = column<false>(unit, i);
            if (c >= N) continue;
            if (F32) static_cast<float*>(base)[row * N + c] = v[i];
            else static_cast<uint16_t*>(base)[row * N + c] = f32_to_bf16(v[i]);
        }
    }
}
// Threads that cover the columns of a row, eight each.
__host__ __device__ inline int units_of(int N, bool wide) { return wide ? N >> 3 : (N + 255) / 256 * 32; }

// One warp a list position.
template <bool F32, bool WIDE>
__global__ void __launch_bounds__(kSortThreads)
permute_kernel(const void* x, const int32_t* list, int R, int k, int N, void* rows, int32_t* positions) {
    pdl_wait_then_trigger();
    const int r = blockIdx.x * (kSortThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (r >= R) return;
    const int entry = list[r];
    const bool good = (unsigned)entry < (unsigned)R;
    if (good && lane == 0) positions[entry] = r;
    if (rows == nullptr) return;
    const int units = units_of(N, WIDE);
    const size_t t = good ? entry / k : 0;
#pragma unroll 4
    for (int u = lane; u < units; u += 32) {
        float v[8];
        get8<F32, WIDE>(x, t, N, u, v);
        if (!good)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = 0.f;
        put8<F32, WIDE>(rows, r, N, u, v);
    }
}

// One thread per eight columns of a token.
template <bool F32, bool YF32, bool WIDE>
__global__ void __launch_bounds__(kSortThreads)
combine_rows_kernel(const void* rows, const float* w, const int32_t* positions, const uint16_t* add, size_t total,
                    unsigned units, int R, int k, int N, void* y) {
    pdl_wait_then_trigger();
    const size_t at = (size_t)blockIdx.x * kSortThreads + threadIdx.x;
    if (at >= total) return;
    const size_t t = at / units;
    const int unit = (int)(at - t * units);
    float acc[8] = {};
    for (int j0 = 0; j0 < k; j0 += kAhead) {
        float v[kAhead][8], c[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            c[j] = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[j][i] = 0.f;
            if (j0 + j >= k) continue;
            const size_t entry = t * k + j0 + j;
            const int p = positions != nullptr ? positions[entry] : (int)entry;
            if ((unsigned)p >= (unsigned)R) continue;
            c[j] = w != nullptr ? w[entry] : 1.f;
            get8<F32, WIDE>(rows, p, N, unit, v[j]);
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = fmaf(c[j], v[j][i], acc[i]);
    }
    if (add != nullptr) {
        float a[8];
        get8<false, WIDE>(add, t, N, unit, a);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += a[i];
    }
    put8<YF32, WIDE>(y, t, N, unit, acc);
}

// One CTA a token.
template <bool F32, bool DYF32, bool WIDE>
__global__ void __launch_bounds__(kSortThreads)
combine_backward_kernel(const void* dy, const void* rows, const float* w, const int32_t* positions, int R, int k, int N,
                        void* d_rows, float* d_w) {
    __shared__ float s_part[kSortThreads / 32][kAhead];
    pdl_wait_then_trigger();
    const size_t t = blockIdx.x;
    const int units = units_of(N, WIDE), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int j0 = 0; j0 < k; j0 += kAhead) {
        int p[kAhead];
        float c[kAhead], part[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            p[j] = -1, c[j] = part[j] = 0.f;
            if (j0 + j >= k) continue;
            const size_t entry = t * k + j0 + j;
            p[j] = positions != nullptr ? positions[entry] : (int)entry;
            if ((unsigned)p[j] >= (unsigned)R) p[j] = -1;
            c[j] = w != nullptr ? w[entry] : 1.f;
        }
        for (int u = threadIdx.x; u < units; u += kSortThreads) {
            float g[8], v[kAhead][8];
            get8<DYF32, WIDE>(dy, t, N, u, g);
            if (d_w != nullptr) {
#pragma unroll
                for (int j = 0; j < kAhead; ++j)
                    if (p[j] >= 0) get8<F32, WIDE>(rows, p[j], N, u, v[j]);
#pragma unroll
                for (int j = 0; j < kAhead; ++j)
                    if (p[j] >= 0)
#pragma unroll
                        for (int i = 0; i < 8; ++i) part[j] = fmaf(g[i], v[j][i], part[j]);
            }
            if (d_rows != nullptr)
#pragma unroll
                for (int j = 0; j < kAhead; ++j) {
                    if (p[j] < 0) continue;
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[j][i] = c[j] * g[i];
                    put8<F32, WIDE>(d_rows, p[j], N, u, v[j]);
                }
        }
        if (d_w == nullptr) continue;
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            part[j] = warp_sum(part[j]);
            if (lane == 0) s_part[warp][j] = part[j];
        }
        __syncthreads();
        if (threadIdx.x < kAhead && j0 + threadIdx.x < k) {
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < kSortThreads / 32; ++i) sum += s_part[i][threadIdx.x];
            d_w[t * k + j0 + threadIdx.x] = sum;
        }
        __syncthreads();
    }
}

}  // namespace

cudaError_t launch_permute(const void* x, bool f32, const int32_t* list, int T, int k, int N, void* rows,
                           int32_t* positions, cudaStream_t s) {
    const int R = T * k;
    const unsigned grid = (unsigned)((R + kSortThreads / 32 - 1) / (kSortThreads / 32));
    const auto run = [&](auto kernel) { return launch_pdl(kernel, grid, kSortThreads, 0, s, x, list, R, k, N, rows, positions); };
    if (N % 8 == 0) return f32 ? run(permute_kernel<true, true>) : run(permute_kernel<false, true>);
    return f32 ? run(permute_kernel<true, false>) : run(permute_kernel<false, false>);
}

template <bool F32, bool YF32, bool WIDE>
static cudaError_t combine_as(const void* rows, const float* w, const int32_t* positions, const uint16_t* add, int T,
                              int k, int N, void* y, cudaStream_t s) {
    const unsigned units = (unsigned)units_of(N, WIDE);
    const size_t total = (size_t)T * units, grid = (total + kSortThreads - 1) / kSortThreads;
    if (grid > 0x7FFFFFFFu) return cudaErrorInvalidConfiguration;
    return launch_pdl(combine_rows_kernel<F32, YF32, WIDE>, (unsigned)grid, kSortThreads, 0, s, rows, w, positions, add,
                      total, units, T * k, k, N, y);
}

cudaError_t launch_combine(const void* rows, bool rows_f32, const float* w, const int32_t* positions,
                           const uint16_t* add, int T, int k, int N, void* y, bool y_f32, cudaStream_t s) {
    const int which = (rows_f32 ? 4 : 0) | (y_f32 ? 2 : 0) | (N % 8 == 0 ? 1 : 0);
    switch (which) {
        case 0: return combine_as<false, false, false>(rows, w, positions, add, T, k, N, y, s);
        case 1: return combine_as<false, false, true>(rows, w, positions, add, T, k, N, y, s);
        case 2: return combine_as<false, true, false>(rows, w, positions, add, T, k, N, y, s);
        case 3: return combine_as<false, true, true>(rows, w, positions, add, T, k, N, y, s);
        case 4: return combine_as<true, false, false>(rows, w, positions, add, T, k, N, y, s);
        case 5: return combine_as<true, false, true>(rows, w, positions, add, T, k, N, y, s);
        case 6: return combine_as<true, true, false>(rows, w, positions, add, T, k, N, y, s);
        default: return combine_as<true, true, true>(rows, w, positions, add, T, k, N, y, s);
    }
}

cudaError_t launch_combine_backward(const void* dy, bool dy_f32, const void* rows, bool rows_f32, const float* w,
                                    const int32_t* positions, int T, int k, int N, void* d_rows, float* d_w,
                                    cudaStream_t s) {
    const auto run = [&](auto kernel) {
        return launch_pdl(kernel, (unsigned)T, kSortThreads, 0, s, dy, rows, w, positions, T * k, k, N, d_rows, d_w);
    };
    const int which = (rows_f32 ? 4 : 0) | (dy_f32 ? 2 : 0) | (N % 8 == 0 ? 1 : 0);
    switch (which) {
        case 0: return run(combine_backward_kernel<false, false, false>);
        case 1: return run(combine_backward_kernel<false, false, true>);
        case 2: return run(combine_backward_kernel<false, true, false>);
        case 3: return run(combine_backward_kernel<false, true, true>);
        case 4: return run(combine_backward_kernel<true, false, false>);
        case 5: return run(combine_backward_kernel<true, false, true>);
        case 6: return run(combine_backward_kernel<true, true, false>);
        default: return run(combine_backward_kernel<true, true, true>);
    }
}

}  // namespace nvfp4
