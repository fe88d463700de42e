// Pairs of CTAs (cta_group::2) that compute tiles of 256 weight rows of one expert times up to NT of its list
// positions: what the tile kernels of the bf16, 8-bit and NVFP4 products share. How they use it is described in
// rows_tc.cu.
#pragma once

#include "common.cuh"
#include "kernels.cuh"
#include "tc_common.cuh"

namespace nvfp4 {

namespace {

constexpr int kM = 128;                  // weight rows of a CTA's half of a tile
constexpr int kStepBytes = 128;          // K bytes of a step: one row of the swizzle atom
constexpr int kNRound = 64;              // a tile's columns are a multiple of this
constexpr int kMaxTiles = 1 << 30;
constexpr unsigned long long kCopyDrainNs = 10000000ull;
constexpr unsigned long long kShortLimitNs = 1000000ull;
static_assert(NVFP4_MAX_EXPERTS <= 8 * 32, "eight experts a lane");

// Output staging of an epilogue warp (bf16): 16 rows of y, 32 neighbouring outputs of each. The pitch of
// 80 bytes puts the eight 16-byte rows of a stmatrix on different banks.
constexpr int kStgRows = 16, kStgPitch = 80;

// ---------------------------------------------------------------- pair of CTAs
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release;\n barrier.cluster.wait.acquire;" ::: "memory");
}
// The address of this CTA's shared-memory location in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
// Arrive on a barrier of either CTA. What the arrival orders are tensor-memory loads (fenced before it)
// and copies that a barrier has already reported, no plain stores: a release at cluster scope, which
// waits for every store of the thread, cost the epilogue warps 1 us a step.
__device__ __forceinline__ void arrive_cluster(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" :: "r"(cluster_addr) : "memory");
}
// The same where it hands plain stores to this CTA's shared memory, its own and those of the lanes it has met since, to a
// thread of either CTA that waits at the scope of the cluster. The release is of shared memory alone (one that waits for
// global memory too, at every arrival of NVFP4 scales: 4096 x 8192 x 2048 in 45 us for 33).
__device__ __forceinline__ void arrive_cluster_release_smem(uint32_t cluster_addr) {
    asm volatile("fence.release.sync_restrict::shared::cta.cluster;\n"
                 " mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" :: "r"(cluster_addr) : "memory");
}

// One look at a barrier's phase, without suspending the thread.
__device__ __forceinline__ bool mbar_test_wait(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok) : "r"(su32(bar)), "r"(parity) : "memory");
    return ok != 0;
}
// This and mbar_try_wait that see what arrivals of either CTA released to the cluster.
__device__ __forceinline__ bool mbar_test_wait_cluster(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok) : "r"(su32(bar)), "r"(parity) : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok) : "r"(su32(bar)), "r"(parity) : "memory");
    return ok != 0;
}

// Bounded wait on a barrier that either CTA of the pair, or its MMAs, arrive on. One that runs out
// records the timeout and raises the abort flag of both CTAs; once raised, every wait gives up.
struct Waiter {
    volatile int* abort_flag;
    uint32_t peer_flag;          // the other CTA's flag
    WsHeader* hdr;
    unsigned long long limit_ns;

    // By all lanes of a warp; the answer is the same in each. Reading the clock takes longer than most waits, and a
    // suspended poll sleeps up to some 10 us, so the clock starts after 64 polls. A short limit (kShortLimitNs) would
    // be over by then: it counts from the first poll that fails, and no poll suspends.
    __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) const {
        if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;
        const bool brief = limit_ns < kShortLimitNs;
        if (!brief) {
#pragma unroll 1
            for (int i = 0; i < 64; ++i)
                if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        }
        const unsigned long long t0 = global_timer_ns();
        while (!__all_sync(0xffffffffu, brief ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity))) {
            const bool late = global_timer_ns() - t0 > limit_ns;
            if (__any_sync(0xffffffffu, late || *abort_flag)) {
                if (late) {
                    *abort_flag = 1;
                    asm volatile("st.volatile.shared::cluster.u32 [%0], %1;" :: "r"(peer_flag), "r"(1) : "memory");
                    if (hdr != nullptr) record_status(hdr, NVFP4_ERR_DEVICE_TIMEOUT);
                }
                return false;
            }
        }
        return true;
    }
    // The same by one thread alone. CLUSTER: it sees what the arrivals released to the cluster.
    template <bool CLUSTER = false>
    __device__ __forceinline__ bool one(uint64_t* bar, uint32_t parity) const {
        const auto test = [&] { return CLUSTER ? mbar_test_wait_cluster(bar, parity) : mbar_test_wait(bar, parity); };
        const auto try_wait = [&] { return CLUSTER ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity); };
        if (test()) return true;
        const bool brief = limit_ns < kShortLimitNs;
        if (!brief) {
#pragma unroll 1
            for (int i = 0; i < 64; ++i)
                if (try_wait()) return true;
        }
        const unsigned long long t0 = global_timer_ns();
        while (!(brief ? test() : try_wait())) {
            const bool late = global_timer_ns() - t0 > limit_ns;
            if (late) {
                *abort_flag = 1;
                asm volatile("st.volatile.shared::cluster.u32 [%0], %1;" :: "r"(peer_flag), "r"(1) : "memory");
                if (hdr != nullptr) record_status(hdr, NVFP4_ERR_DEVICE_TIMEOUT);
            }
            if (late || *abort_flag) return false;
        }
        return true;
    }
};

// One lane of the (converged) warp. The tensor-core and TMA instructions take uniform registers: under
// `lane == 0` the compiler cannot know that one thread is left and builds a loop around each.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// Arrive on this barrier in both CTAs (cluster mask) once every MMA issued so far by this thread has completed.
__device__ __forceinline__ void commit_pair(uint64_t* bar, uint16_t mask) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
        :: "r"(su32(bar)), "h"(mask) : "memory");
}
// 32 lanes x 16 columns in fragments: v[8 L + 4 j + 2 u + b] is lane 16 L + 8 u + (thread / 4), column
// 8 j + 2 (thread % 4) + b. Valid after tmem_wait16. A thread needs the scales of a quarter of the columns
// this way; with a lane to a thread it needs all of them, 1024 clocks of shared-memory reads a step.
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, float (&v)[16]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
        asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=f"(v[8 * h + 0]), "=f"(v[8 * h + 1]), "=f"(v[8 * h + 2]), "=f"(v[8 * h + 3]),
                       "=f"(v[8 * h + 4]), "=f"(v[8 * h + 5]), "=f"(v[8 * h + 6]), "=f"(v[8 * h + 7])
                     : "r"(taddr + ((uint32_t)(16 * h) << 16)));
}
// The loads so far are done; the values pass through, so that no use of them moves before the wait.
__device__ __forceinline__ void tmem_wait16(float (&v)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                   "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]),
                   "+f"(v[15]));
}

// Four rows of a 2D tensor (a map of single rows), bytes [x, x + 128) of each.
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap* map, int x, int r0, int r1, int r2, int r3,
                                            uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];"
        :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(r0), "r"(r1), "r"(r2), "r"(r3), "r"(su32(bar))
        : "memory");
}

// ---------------------------------------------------------------- tiles
// ROUND: a tile's columns are a multiple of it, and so are the parts of an expert's rows.
template <int ROUND>
struct TileOf {
    int e, r0, n, m0;   // expert, first list position, rows, first weight row
    __device__ __forceinline__ int mma_n() const { return (n + ROUND - 1) & ~(ROUND - 1); }
};
using Tile = TileOf<kNRound>;

// The tiles of a pair: token tile tt (numbered over the experts) and weight tile mt of i = first, first +
// step, ... below total. tab: token-tile prefix [E + 1], first position [E], rows [E].
template <int ROUND>
struct WalkOf {
    const int* tab;
    int E, m_tiles, i, step, total, tt, mt, dt, dm;

    __device__ __forceinline__ WalkOf(const int* tab_, int E_, int m_tiles_, int first, int step_, int total_)
        : tab(tab_), E(E_), m_tiles(m_tiles_), i(first), step(step_), total(total_), tt(first / m_tiles_),
          mt(first - tt * m_tiles_), dt(step_ / m_tiles_), dm(step_ - dt * m_tiles_) {}
    __device__ __forceinline__ bool more() const { return i < total; }
    __device__ __forceinline__ void next() {
        i += step, tt += dt, mt += dm;
        if (mt >= m_tiles) mt -= m_tiles, ++tt;
    }
    // By all lanes of a warp: the last expert whose first token tile is at most tt (an empty one before it
    // has the same first), found among every eighth and then among eight.
    __device__ __forceinline__ TileOf<ROUND> tile() const {
        const int lane = threadIdx.x & 31;
        const int b = __popc(__ballot_sync(0xffffffffu, 8 * lane < E && tab[min(8 * lane, E)] <= tt)) - 1;
        const int e8 = 8 * b + (lane & 7);
        const int e = 8 * b + __popc(__ballot_sync(0xffffffffu, lane < 8 && e8 < E && tab[min(e8, E)] <= tt)) - 1;
        const int cnt = tab[E + 1 + E + e], parts = tab[e + 1] - tab[e], l = tt - tab[e];
        // nearly equal parts in multiples of ROUND: parts = ceil(cnt / NT), so none is empty
        const int per = parts == 1 ? cnt : ((cnt + parts - 1) / parts + ROUND - 1) & ~(ROUND - 1);
        TileOf<ROUND> t;
        t.e = uniform(e);
        t.r0 = uniform(tab[E + 1 + e] + l * per);
        t.n = uniform(min(per, cnt - l * per));
        t.m0 = mt * (2 * kM);
        return t;
    }
};
using Walk = WalkOf<kNRound>;

// The table of a call, by one warp: the tiles of NT rows of every expert, eight experts a lane, then a prefix sum over
// the lanes. tab: token-tile prefix [E + 1], first position [E], rows [E].
template <int NT>
__device__ __forceinline__ void tile_table(const RowsProduct& P, int* tab) {
    const int lane = threadIdx.x & 31;
    int cnt[8], sum = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int e = lane * 8 + i;
        int lo = 0, n = 0;
        if (e < P.E) {
            if (P.offsets == nullptr) {
                n = P.R;
            } else {
                lo = min(max(P.offsets[e], 0), P.R);
                n = max(min(max(P.offsets[e + 1], 0), P.R) - lo, 0);
            }
            tab[P.E + 1 + e] = lo;
            tab[P.E + 1 + P.E + e] = n;
        }
        cnt[i] = (n + NT - 1) / NT;
        sum += cnt[i];
    }
    int before = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += t;
    }
    before -= sum;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int e = lane * 8 + i;
        if (e <= P.E) tab[e] = before;
        before += cnt[i];
    }
    if (lane == 31 && P.E == NVFP4_MAX_EXPERTS) tab[P.E] = before;
}

// Write 16 columns (rows of y) x 32 lanes (outputs n0 ..) of a tile, held as by tmem_ld_frag. `row`: lane j's
// (j < 16) row of y for column j, or -1.
__device__ __forceinline__ void store_frag(const RowsProduct& P, const float (&v)[16], int row, int n0, uint8_t* stg) {
    const int lane = threadIdx.x & 31, g = lane >> 2, p = lane & 3;
    if (P.y_f32) {
        // eight neighbouring outputs of a row are one 32-byte sector
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int r = __shfl_sync(0xffffffffu, row, 8 * j + 2 * p + b);
                float* y = static_cast<float*>(P.y) + (size_t)max(r, 0) * P.N + n0 + g;
#pragma unroll
                for (int h = 0; h < 4; ++h)
                    if (r >= 0 && n0 + g + 8 * h < P.N) y[8 * h] = v[8 * (h >> 1) + 4 * j + 2 * (h & 1) + b];
            }
        return;
    }
    // transposed through shared memory: rows of y with 32 neighbouring outputs
    const uint32_t at = su32(stg) + (lane & 7) * kStgPitch + 16 * (lane >> 3);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        uint32_t w[4];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            const int i = 8 * (h >> 1) + 4 * j + 2 * (h & 1);
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[h]) : "f"(v[i + 1]), "f"(v[i]));
        }
        asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};"
                     :: "r"(at + 8 * j * kStgPitch), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
    }
    __syncwarp();
    if ((P.N & 7) == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int c = 8 * i + g, r = __shfl_sync(0xffffffffu, row, c);
            const uint4 u = *reinterpret_cast<const uint4*>(stg + c * kStgPitch + 16 * p);
            if (r >= 0 && n0 + 8 * p < P.N)
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(P.y) + (size_t)r * P.N + n0 + 8 * p) = u;
        }
    } else {
        // Rows of y start at any even address: two rows at a time as 32-bit words from the row's first whole
        // word on, then the single outputs before and after the words of all rows at once.
        uint16_t* y = static_cast<uint16_t*>(P.y);
        const int i = lane & 15;
#pragma unroll
        for (int c = 0; c < 16; c += 2) {
            const int cc = c + (lane >> 4), r = __shfl_sync(0xffffffffu, row, cc);
            const size_t at = (size_t)max(r, 0) * P.N + n0;
            const int odd = (int)(at & 1), e = odd + 2 * i;         // outputs e, e + 1
            const uint32_t* words = reinterpret_cast<const uint32_t*>(stg + cc * kStgPitch) + i;
            const uint32_t w = odd ? __byte_perm(words[0], words[1], 0x5432) : words[0];
            if (r >= 0 && e + 1 < 32 && n0 + e + 1 < P.N) *reinterpret_cast<uint32_t*>(y + at + e) = w;
        }
        {
            const int r = __shfl_sync(0xffffffffu, row, i);
            const size_t at = (size_t)max(r, 0) * P.N + n0;
            const int odd = (int)(at & 1), in = min(32, P.N - n0);  // outputs of this row here
            const int e = lane < 16 ? 0 : in - 1;
            const bool single = lane < 16 ? odd != 0 : ((in - odd) & 1) != 0 && in - 1 >= odd;
            if (r >= 0 && single && in > 0)
                y[at + e] = *reinterpret_cast<const uint16_t*>(stg + i * kStgPitch + 2 * e);
        }
    }
    __syncwarp();
}

// The pairs of a cluster add up their sums of a tile. Columns go in chunks of 16, chunk g of the tile to
// pair g % pairs; a pair's CTA sends the chunks that are not its own to the CTA that has the same weight
// rows there, into that one's ring of stages (every MMA and copy of the cluster is over by then).
// kCols: columns of a warp at most.
template <int kCols, int pairs>
struct Exchange {
    uint8_t* ring;
    int pair, rank;

    // [source pair][lane quadrant][own chunk][4][32 lanes] float4
    __device__ __forceinline__ uint32_t place(int src, int q, int g, int width) const {
        return (uint32_t)(((src * 4 + q) * (width / 4 / pairs) + g / pairs) * 2048) + (threadIdx.x & 31) * 16;
    }
    // Called by all epilogue warps (the CTA's other warps call join). `width` columns a warp from c0 on;
    // sums(c, v) gives the sums of columns c0 + c ...
    template <typename Sums>
    __device__ __forceinline__ void send(const Sums& sums, const Tile& t, int width, int c0, int part, int q) const {
        cluster_sync_all();      // everyone's MMAs are done
#pragma unroll
        for (int c = 0; c < kCols; c += 16) {
            if (c >= width || c0 + c >= t.n) break;
            const int g = (part * width + c) / 16, owner = g % pairs;
            float v[16];
            sums(c, v);
            if (owner == pair) continue;
            const uint32_t to = map_rank(su32(ring) + place(pair, q, g, width), (uint32_t)(2 * owner + rank));
#pragma unroll
            for (int j = 0; j < 4; ++j)
                asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};"
                             :: "r"(to + 512 * j), "f"(v[4 * j]), "f"(v[4 * j + 1]), "f"(v[4 * j + 2]),
                                "f"(v[4 * j + 3]) : "memory");
        }
        cluster_sync_all();      // everyone's sums have arrived
    }
    static __device__ __forceinline__ void join() {
        cluster_sync_all();
        cluster_sync_all();
    }
    // Adds the other pairs' sums, in their order, to this pair's own chunk at c; false: not its own.
    __device__ __forceinline__ bool finish(float (&v)[16], int c, int width, int part, int q) const {
        const int g = (part * width + c) / 16;
        if (g % pairs != pair) return false;
#pragma unroll 1
        for (int src = 0; src < pairs; ++src) {
            if (src == pair) continue;
            const float4* from = reinterpret_cast<const float4*>(ring + place(src, q, g, width));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float4 f = from[32 * j];
                v[4 * j] += f.x, v[4 * j + 1] += f.y, v[4 * j + 2] += f.z, v[4 * j + 3] += f.w;
            }
        }
        return true;
    }
};

// [rows, K] elements of 1 or 2 bytes, read as box_rows x 128 bytes, 128-byte swizzled in shared memory.
inline bool encode_rows(PFN_cuTensorMapEncodeTiled_v12000 fn, CUtensorMap* m, const void* base, bool fp8, uint64_t K,
                 uint64_t rows, uint32_t box_rows) {
    const uint64_t es = fp8 ? 1 : 2;
    const cuuint64_t dims[2] = {K, rows};
    const cuuint64_t strides[1] = {K * es};
    const cuuint32_t box[2] = {(cuuint32_t)(kStepBytes / es), box_rows};
    const cuuint32_t one[2] = {1, 1};
    return fn(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base),
              dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

}  // namespace nvfp4
