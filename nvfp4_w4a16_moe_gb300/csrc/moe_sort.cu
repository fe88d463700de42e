// Rows sorted by expert and back, and the gradients.
//
//   permute   rows[r] = x[list[r] / k],  positions[list[r]] = r
//   combine   y[t] = add[t] + sum_j w[t,j] rows[positions[t k + j]]
//   backward  d_rows[p] = w[t,j] dy[t],  d_w[t,j] = <dy[t], rows[p]>,  p = positions[t k + j]
//
// Sums are fp32, in the order of j (combine) or in a fixed order over threads, warps and the warps' partial sums
// (d_w): the same bits on every run, no atomics. A token's output has one owner.
//
// Bound: HBM. A row is read once and written once: T * k * N elements either way. All rows of a token are asked for
// before the first is used: entries that a token does not have read the row of one that it has, and rows that are not
// there row 0, and what was read is taken out afterwards. (Asked for one behind the other's branch, the combine of 4096
// tokens of 8 x 2048 took 84 us.) us of 4096 tokens of 8 x 2048 in bf16, and of the bytes at the copy rate: permute 21.6
// (22.2), combine 27.9 (24.7), backward 50.7 (41.9): the gradients' reads and writes mixed reach 5.6 TB/s. Asking for the
// next token's positions ahead changes nothing. Rows of 2046 take 25, 28 and 50; of 2047, which start at odd elements and
// are read two bytes at a time, 36, 52 and 144.
#include <type_traits>

#include "common.cuh"
#include "kernels.cuh"

namespace nvfp4 {

namespace {

constexpr int kSortThreads = 256;
constexpr int kAhead = 8;          // rows of a token requested together, at most

// Eight columns of a row a thread. V: columns of one load. 8 (rows of whole 16-byte pieces): neighbouring ones, from
// 8 * unit on. 2, 1 (bf16 rows at 4-byte places; others): a warp's 256 columns in pieces of V, 32 neighbouring pieces a
// load.
template <int V>
__device__ __forceinline__ int column(int unit, int i) {        // of load i
    return V == 8 ? unit * 8 : (unit >> 5) * 256 + ((unit & 31) + 32 * i) * V;
}
// Threads that cover the columns of a row.
__host__ __device__ inline int units_of(int N, int V) { return V == 8 ? N >> 3 : (N + 255) / 256 * 32; }

// Eight columns as they lie in memory; those past the end of the row are 0.
template <bool F32, int V>
struct Piece {
    static constexpr int kWords = F32 ? 8 : V == 1 ? 8 : 4;      // bf16: pairs, or (V = 1) one a word
    uint32_t w[kWords];

    // Rows that a call reads or writes once leave the caches first, but not where two accesses of a thread share a sector
    // (us, 4096 tokens of 8 x 2048 in bf16, without / with: permute 24.8 / 21.6, combine 32.9 / 27.9, backward 53.9 / 50.7;
    // of 4 x 2048 in fp32 backward 52.0 / 57.1).
    static constexpr bool kOnce = !(F32 && V == 8);
    template <bool ONCE, typename T>
    static __device__ __forceinline__ T get_at(const T* p) {
        if constexpr (ONCE) return __ldcs(p);
        else return *p;
    }
    template <bool ONCE, typename T>
    static __device__ __forceinline__ void put_at(T* p, T v) {
        if constexpr (ONCE) __stcs(p, v);
        else *p = v;
    }
    template <bool ONCE>                // kOnce or false
    __device__ __forceinline__ void load(const void* base, size_t row, int N, int unit) {
        if constexpr (V == 8) {
            const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(base) + (row * N + unit * 8) * (F32 ? 4 : 2));
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i) {
                const uint4 u = get_at<ONCE>(p + i);
                w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8 / V; ++i) {
                const int c = column<V>(unit, i);
                w[i] = 0u;
                if (c < N) {
                    const uint16_t* p = static_cast<const uint16_t*>(base) + row * N + c;       // bf16
                    if constexpr (F32) w[i] = get_at<ONCE>(static_cast<const uint32_t*>(base) + row * N + c);
                    else if constexpr (V == 2) w[i] = get_at<ONCE>(reinterpret_cast<const uint32_t*>(p));
                    else w[i] = get_at<ONCE>(p);
                }
            }
        }
    }
    template <bool ONCE>
    __device__ __forceinline__ void store(void* base, size_t row, int N, int unit) const {
        if constexpr (V == 8) {
            uint4* p = reinterpret_cast<uint4*>(static_cast<uint8_t*>(base) + (row * N + unit * 8) * (F32 ? 4 : 2));
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i)
                put_at<ONCE>(p + i, make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]));
        } else {
#pragma unroll
            for (int i = 0; i < 8 / V; ++i) {
                const int c = column<V>(unit, i);
                if (c >= N) continue;
                uint16_t* p = static_cast<uint16_t*>(base) + row * N + c;                       // bf16
                if constexpr (F32) put_at<ONCE>(static_cast<uint32_t*>(base) + row * N + c, w[i]);
                else if constexpr (V == 2) put_at<ONCE>(reinterpret_cast<uint32_t*>(p), w[i]);
                else put_at<ONCE>(p, (uint16_t)w[i]);
            }
        }
    }
    __device__ __forceinline__ void keep(bool there) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = there ? w[i] : 0u;
    }
    __device__ __forceinline__ float get(int i) const {          // the same column for every type of one V
        if constexpr (F32) return __uint_as_float(w[i]);
        else if constexpr (V == 1) return __uint_as_float(w[i] << 16);
        else return i & 1 ? bf16hi(w[i >> 1]) : bf16lo(w[i >> 1]);
    }
    __device__ __forceinline__ void set(const float (&v)[8]) {
        if constexpr (F32) {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[i]);
        } else if constexpr (V == 1) {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = f32_to_bf16(v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
        }
    }
};

// One warp a list position.
template <bool F32, int V>
__global__ void __launch_bounds__(kSortThreads)
permute_kernel(const void* x, const int32_t* list, int R, int k, int N, void* rows, int32_t* positions) {
    pdl_wait_then_trigger();
    const int r = blockIdx.x * (kSortThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (r >= R) return;
    const int entry = list[r];
    const bool good = (unsigned)entry < (unsigned)R;
    if (good && lane == 0) positions[entry] = r;
    if (rows == nullptr) return;
    const int units = units_of(N, V);
    const size_t t = good ? entry / k : 0;
    constexpr int kTogether = F32 || V < 8 ? 4 : 8;
    for (int u0 = lane; u0 < units; u0 += 32 * kTogether) {
        Piece<F32, V> p[kTogether];
#pragma unroll
        for (int i = 0; i < kTogether; ++i)
            if (u0 + 32 * i < units) p[i].template load<false>(x, t, N, u0 + 32 * i);
#pragma unroll
        for (int i = 0; i < kTogether; ++i) {
            if (u0 + 32 * i >= units) break;
            p[i].keep(good);
            p[i].template store<Piece<F32, V>::kOnce>(rows, r, N, u0 + 32 * i);
        }
    }
}

// Entries j0 .. j0 + KA - 1 of token t: rows (0 where there is none) and whether each is there.
template <int KA>
__device__ __forceinline__ void find_entries(const int32_t* positions, const float* w, size_t t, int j0, int k, int R,
                                             int (&p)[KA], bool (&there)[KA], float (&c)[KA]) {
#pragma unroll
    for (int j = 0; j < KA; ++j) {
        const size_t entry = t * k + min(j0 + j, k - 1);
        p[j] = positions != nullptr ? positions[entry] : (int)entry;
        c[j] = w != nullptr ? w[entry] : 1.f;
    }
#pragma unroll
    for (int j = 0; j < KA; ++j) {
        there[j] = j0 + j < k && (unsigned)p[j] < (unsigned)R;
        p[j] = (unsigned)p[j] < (unsigned)R ? p[j] : 0;
    }
}

// One thread per eight columns of a token.
template <bool F32, bool YF32, int V, int KA>
__global__ void __launch_bounds__(kSortThreads)
combine_rows_kernel(const void* rows, const float* w, const int32_t* positions, const uint16_t* add, size_t total,
                    unsigned units, int R, int k, int N, void* y) {
    pdl_wait_then_trigger();
    const size_t at = (size_t)blockIdx.x * kSortThreads + threadIdx.x;
    if (at >= total) return;
    const size_t t = total >> 32 ? at / units : (size_t)((unsigned)at / units);
    const int unit = (int)(at - t * units);
    Piece<false, F32 || YF32 ? (V == 8 ? 8 : 1) : V> a;
    if (add != nullptr) a.template load<decltype(a)::kOnce>(add, t, N, unit);
    float acc[8] = {};
    for (int j0 = 0; j0 < k; j0 += KA) {
        int p[KA];
        bool there[KA];
        float c[KA];
        Piece<F32, V> v[KA];
        find_entries<KA>(positions, w, t, j0, k, R, p, there, c);
#pragma unroll
        for (int j = 0; j < KA; ++j) v[j].template load<Piece<F32, V>::kOnce>(rows, p[j], N, unit);
#pragma unroll
        for (int j = 0; j < KA; ++j) {
            v[j].keep(there[j]);
            const float cj = there[j] ? c[j] : 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = fmaf(cj, v[j].get(i), acc[i]);
        }
    }
    if (add != nullptr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += a.get(i);
    }
    Piece<YF32, V> out;
    out.set(acc);
    out.template store<false>(y, t, N, unit);
}

// One CTA a token.
template <bool F32, bool DYF32, int V, int KA>
__global__ void __launch_bounds__(kSortThreads)
combine_backward_kernel(const void* dy, const void* rows, const float* w, const int32_t* positions, int R, int k, int N,
                        void* d_rows, float* d_w) {
    __shared__ float s_part[kSortThreads / 32][KA];
    pdl_wait_then_trigger();
    const size_t t = blockIdx.x;
    const int units = units_of(N, V), lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    for (int j0 = 0; j0 < k; j0 += KA) {
        int p[KA];
        bool there[KA];
        float c[KA], part[KA];
        find_entries<KA>(positions, w, t, j0, k, R, p, there, c);
#pragma unroll
        for (int j = 0; j < KA; ++j) part[j] = 0.f;
        for (int u = threadIdx.x; u < units; u += blockDim.x) {
            Piece<DYF32, V> gp;
            gp.template load<Piece<DYF32, V>::kOnce>(dy, t, N, u);
            if (d_w != nullptr) {
                Piece<F32, V> v[KA];
#pragma unroll
                for (int j = 0; j < KA; ++j) v[j].template load<Piece<F32, V>::kOnce>(rows, p[j], N, u);
#pragma unroll
                for (int j = 0; j < KA; ++j) {
                    v[j].keep(there[j]);
#pragma unroll
                    for (int i = 0; i < 8; ++i) part[j] = fmaf(gp.get(i), v[j].get(i), part[j]);
                }
            }
            if (d_rows != nullptr)
#pragma unroll
                for (int j = 0; j < KA; ++j) {
                    if (!there[j]) continue;
                    float g[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) g[i] = c[j] * gp.get(i);
                    Piece<F32, V> out;
                    out.set(g);
                    out.template store<Piece<F32, V>::kOnce>(d_rows, p[j], N, u);
                }
        }
        if (d_w == nullptr) continue;
        // a token's dy may hold infinities or NaN: no product of its entries without a row counts
#pragma unroll
        for (int j = 0; j < KA; ++j) part[j] = there[j] ? part[j] : 0.f;
        // KA sums over the lanes: each exchange of halves leaves a lane with half as many sums, the rest as usual
        int mine = 0;                  // which sum part[0] is in the end
#pragma unroll
        for (int h = KA / 2, o = 16; h > 0; h >>= 1, o >>= 1) {
            const bool up = (lane & o) != 0;
            mine += up ? h : 0;
#pragma unroll
            for (int j = 0; j < h; ++j) {
                const float give = up ? part[j] : part[j + h], hold = up ? part[j + h] : part[j];
                part[j] = hold + __shfl_xor_sync(0xffffffffu, give, o);
            }
        }
#pragma unroll
        for (int o = 16 / KA; o > 0; o >>= 1) part[0] += __shfl_xor_sync(0xffffffffu, part[0], o);
        if ((lane & (32 / KA - 1)) == 0) s_part[warp][mine] = part[0];
        __syncthreads();
        if (threadIdx.x < KA && j0 + threadIdx.x < k) {
            float sum = 0.f;
            for (int i = 0; i < warps; ++i) sum += s_part[i][threadIdx.x];
            d_w[t * k + j0 + threadIdx.x] = sum;
        }
        __syncthreads();
    }
}

// Columns of a load: rows of 8 columns each are whole 16-byte pieces; bf16 rows of an even number of columns start at
// 4-byte places. Different types have to split a row alike, so pairs are for bf16 alone.
int load_columns(int N, bool all16) { return N % 8 == 0 ? 8 : all16 && N % 2 == 0 ? 2 : 1; }

template <int n>
using Int = std::integral_constant<int, n>;

// f(columns of a load, rows asked for together)
template <bool PAIRS, typename F>
cudaError_t by_shape(int V, int k, const F& f) {
    const auto ahead = [&](auto v) {
        if (k == 1) return f(v, Int<1>{});
        if (k == 2) return f(v, Int<2>{});
        if (k <= 4) return f(v, Int<4>{});
        return f(v, Int<kAhead>{});
    };
    if (V == 8) return ahead(Int<8>{});
    if constexpr (PAIRS)
        if (V == 2) return ahead(Int<2>{});
    return ahead(Int<1>{});
}

template <bool F32, bool YF32>
cudaError_t combine_as(const void* rows, const float* w, const int32_t* positions, const uint16_t* add, int T, int k,
                       int N, void* y, cudaStream_t s) {
    const int V = load_columns(N, !F32 && !YF32);
    const unsigned units = (unsigned)units_of(N, V);
    const size_t total = (size_t)T * units, grid = (total + kSortThreads - 1) / kSortThreads;
    if (grid > 0x7FFFFFFFu) return cudaErrorInvalidConfiguration;
    return by_shape<!F32 && !YF32>(V, k, [&](auto v, auto ahead) {
        return launch_pdl(combine_rows_kernel<F32, YF32, decltype(v)::value, decltype(ahead)::value>, (unsigned)grid, kSortThreads, 0, s, rows, w, positions,
                          add, total, units, T * k, k, N, y);
    });
}

template <bool F32, bool DYF32>
cudaError_t backward_as(const void* dy, const void* rows, const float* w, const int32_t* positions, int T, int k, int N,
                        void* d_rows, float* d_w, cudaStream_t s) {
    const int V = load_columns(N, !F32 && !DYF32);
    const unsigned threads = (unsigned)std::min((units_of(N, V) + 31) / 32 * 32, kSortThreads);
    return by_shape<!F32 && !DYF32>(V, k, [&](auto v, auto ahead) {
        return launch_pdl(combine_backward_kernel<F32, DYF32, decltype(v)::value, decltype(ahead)::value>, (unsigned)T, threads, 0, s, dy, rows, w, positions,
                          T * k, k, N, d_rows, d_w);
    });
}

}  // namespace

cudaError_t launch_permute(const void* x, bool f32, const int32_t* list, int T, int k, int N, void* rows,
                           int32_t* positions, cudaStream_t s) {
    const int R = T * k;
    const unsigned grid = (unsigned)((R + kSortThreads / 32 - 1) / (kSortThreads / 32));
    const auto run = [&](auto kernel) { return launch_pdl(kernel, grid, kSortThreads, 0, s, x, list, R, k, N, rows, positions); };
    const int V = load_columns(N, !f32);
    if (V == 8) return f32 ? run(permute_kernel<true, 8>) : run(permute_kernel<false, 8>);
    if (V == 2) return run(permute_kernel<false, 2>);
    return f32 ? run(permute_kernel<true, 1>) : run(permute_kernel<false, 1>);
}

cudaError_t launch_combine(const void* rows, bool rows_f32, const float* w, const int32_t* positions,
                           const uint16_t* add, int T, int k, int N, void* y, bool y_f32, cudaStream_t s) {
    if (rows_f32) return y_f32 ? combine_as<true, true>(rows, w, positions, add, T, k, N, y, s)
                               : combine_as<true, false>(rows, w, positions, add, T, k, N, y, s);
    return y_f32 ? combine_as<false, true>(rows, w, positions, add, T, k, N, y, s)
                 : combine_as<false, false>(rows, w, positions, add, T, k, N, y, s);
}

cudaError_t launch_combine_backward(const void* dy, bool dy_f32, const void* rows, bool rows_f32, const float* w,
                                    const int32_t* positions, int T, int k, int N, void* d_rows, float* d_w,
                                    cudaStream_t s) {
    if (rows_f32) return dy_f32 ? backward_as<true, true>(dy, rows, w, positions, T, k, N, d_rows, d_w, s)
                                : backward_as<true, false>(dy, rows, w, positions, T, k, N, d_rows, d_w, s);
    return dy_f32 ? backward_as<false, true>(dy, rows, w, positions, T, k, N, d_rows, d_w, s)
                  : backward_as<false, false>(dy, rows, w, positions, T, k, N, d_rows, d_w, s);
}

}  // namespace nvfp4
