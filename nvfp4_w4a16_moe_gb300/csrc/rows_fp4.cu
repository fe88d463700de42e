// Products of NVFP4 rows with one NVFP4 matrix or with each expert's:
//   y[o(r), n] = xr[i(r)] wt[e, n] sum_b xs[i(r), b] ws[n, b] sum_{k in b} x[i(r), k] w[n, k]
// One CTA computes 32 list positions of an expert times 32 outputs, both operands expanded to fp32 in shared memory
// 64 columns at a time (code times block scale is exact there).
#include "common.cuh"
#include "kernels.cuh"

namespace nvfp4 {

namespace {

constexpr int kTile = 32, kCols = 64, kPitch = kCols + 1;

__global__ void __launch_bounds__(256)
rows_fp4_kernel(const Fp4Product Q) {
    __shared__ float sx[kTile][kPitch], sw[kTile][kPitch];
    pdl_wait_then_trigger();
    const RowsProduct& P = Q.r;
    const int e = blockIdx.y, n0 = blockIdx.x * kTile;
    int lo = 0, hi = P.R;
    if (P.offsets != nullptr) {
        lo = min(max(P.offsets[e], 0), P.R);
        hi = max(min(max(P.offsets[e + 1], 0), P.R), lo);
    }
    const uint8_t *x = static_cast<const uint8_t*>(P.x), *w = static_cast<const uint8_t*>(P.w);
    const int tr = threadIdx.x >> 5, tn = threadIdx.x & 31, half = P.K / 2, KB = P.K / 16;
    for (int r0 = lo; r0 < hi; r0 += kTile) {
        float acc[4] = {};
        for (int k0 = 0; k0 < P.K; k0 += kCols) {
            for (int i = threadIdx.x; i < kTile * (kCols / 2); i += 256) {
                const int row = i / (kCols / 2), k = k0 + 2 * (i % (kCols / 2));
                float2 a = make_float2(0.f, 0.f), b = a;
                if (k < P.K) {
                    const int src = r0 + row < hi ? x_row(P, r0 + row) : -1;
                    if (src >= 0) {
                        a = e2m1x2_to_f32x2(x[(size_t)src * half + k / 2]);
                        const float s = e4m3_to_f32(Q.xs[(size_t)src * KB + k / 16]);
                        a.x *= s, a.y *= s;
                    }
                    if (n0 + row < P.N) {
                        const size_t at = (size_t)e * P.N + n0 + row;
                        b = e2m1x2_to_f32x2(w[at * half + k / 2]);
                        const float s = e4m3_to_f32(Q.ws[at * KB + k / 16]);
                        b.x *= s, b.y *= s;
                    }
                }
                sx[row][k - k0] = a.x, sx[row][k - k0 + 1] = a.y;
                sw[row][k - k0] = b.x, sw[row][k - k0 + 1] = b.y;
            }
            __syncthreads();
            for (int k = 0; k < kCols; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[i] = fmaf(sx[tr + 8 * i][k], sw[tn][k], acc[i]);
            __syncthreads();
        }
        const int n = n0 + tn;
        if (n >= P.N) continue;
        const float wt = Q.wt[e * Q.parts + n / (P.N / Q.parts)];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = r0 + tr + 8 * i;
            if (r >= hi) continue;
            const int src = x_row(P, r), dst = y_row(P, r);
            if (dst < 0) continue;
            const float v = src < 0 ? 0.f : acc[i] * (Q.xr[src] * wt);
            if (P.y_f32) static_cast<float*>(P.y)[(size_t)dst * P.N + n] = v;
            else static_cast<uint16_t*>(P.y)[(size_t)dst * P.N + n] = f32_to_bf16(v);
        }
    }
}

}  // namespace

cudaError_t launch_rows_fp4(const Fp4Product& P, WsHeader* hdr, const DeviceInfo& dev, uint64_t wait_limit,
                            cudaStream_t s) {
    rows_fp4_kernel<<<dim3((P.r.N + kTile - 1) / kTile, P.r.E), 256, 0, s>>>(P);
    return cudaGetLastError();
}

}  // namespace nvfp4
