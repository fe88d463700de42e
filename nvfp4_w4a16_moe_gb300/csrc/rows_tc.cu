// Products of many rows with one matrix or with each expert's matrix on the 5th-generation tensor
// cores: y[o(r), n] = sum_k W[e(r)][n, k] x[i(r), k], in bf16 or in E4M3 with block scales.
//
// A pair of CTAs (cta_group::2) computes a tile of 256 weight rows of one expert times up to NT of its
// list positions. The weights are the MMA's A operand (M = 256: 128 rows in each CTA's shared memory) and
// the rows of x its B operand (N = the tile's rows, rounded up to 64; each CTA holds half of them), so an
// expert with few rows costs few MMA cycles, and any number of rows per expert works without padding in
// memory. The pair is what feeds the tensor cores: one CTA alone (128 x 256 tiles) needs 48 KB of operands
// per 64 columns of bf16 from L2 where a CTA of a pair needs 32: 4096 x 8192 x 2048 took 107 us that way
// and takes 72 us (1.91 PFLOP/s, 99 % of the measured cuBLAS rate).
//
// An expert's rows are cut into tiles of nearly equal size. The tiles of the whole call are numbered
// over the experts (prefix sums over the offsets, made by every CTA for itself: the host never sees the
// counts), and a persistent grid of pairs walks them. Grouped calls of the layer's shape are bound by the
// bytes of the experts' matrices: gate/up of 256 bf16 experts of 1024 x 2048, 207 us at 4096 tokens (83 %
// of the copy rate), 101 us for the experts that 64 tokens reach.
//
// Warp roles of a CTA (both CTAs of a pair but where said):
//   TMA warp: brings step s (128 bytes of K) of the CTA's weight rows and, for rows in list order, of
//     its rows of x into a ring of 128-byte-swizzled stages, each operand in one box: there is a tensor
//     map for every height a tile's share can have. Coordinates past a matrix read zeros, which also pads
//     K. (Boxes of 16 rows, one to a lane, ran the ring at half its rate.)
//   Gather warps: rows read through the list, four tokens' rows a copy (tile::gather4), so no permuted
//     copy of x is ever written; as fast as rows in order where the experts' bytes bound the call.
//   Scale warps (8-bit): x_scale * w_scale of every column of four steps, in a ring of their own.
//   MMA warp: in the pair's first CTA, the MMAs of a step for both. In the second CTA it tells the first
//     that the step's operands have landed here.
//   Epilogue warps. bf16: a whole tile is summed in one tensor-memory buffer, then read and written out. The
//     tensor core's running sum loses more than a register sum would: an fp32 output of K = 2048 is off by
//     2.2e-6 (norm, against 64 bits; in 8 bits, where blocks of 128 are added in registers, by 8e-8).
//     8-bit: the operands carry a scale per 128 of K, so every step starts a buffer from zero; the warps
//     read it, multiply each column with its scale and add it to the tile's sum in registers (fp32),
//     while the MMAs fill the next buffer. That bounds 8-bit tiles, not the MMAs: a step of 256 x 256 takes
//     0.58 us where the MMAs alone need 0.27 (over a quarter of it are the multiply-adds; sixteen warps
//     issue half of their scheduler's slots, eight warps with twice the sums each took 0.82 us). 4096 x 8192
//     x 2048: 80 us, 1.7 PFLOP/s: seven rounds of 16 steps, 65 us, and of about 2 us in which the same warps
//     write the tile out and the MMAs, 512 / NT steps ahead at most, stand still. Gate/up of 4096 tokens over
//     256 experts of 1024 x 2048: 135 us. Separate buffers for the two column halves cost more in operand reads
//     than they hid.
// Tensor memory holds 512 / NT buffers: as many tiles (bf16) or steps (8-bit) the MMAs can run ahead.
//
// Few tiles (few rows of W, a small batch): a cluster of two or four pairs shares a tile's K, and the
// pairs' sums are exchanged through distributed shared memory, each pair finishing a part of the columns: to
// its own sum it adds the others' in the order of the pairs, the same order on every run. (64 rows times
// 2048 x 8192 in 8 bits: 24 us with one pair a tile, 9.0 with four. The 8-bit forms of 256 columns with two and
// four pairs spill 32 bytes a thread.)
//
// Every wait is bounded; one that runs out records NVFP4_ERR_DEVICE_TIMEOUT (where the caller passed a
// workspace) and makes the pair fill its remaining tiles with NaN.
#include <atomic>
#include <cstring>

#include "common.cuh"
#include "kernels.cuh"
#include "tc_common.cuh"

namespace nvfp4 {

namespace {

constexpr int kM = 128;                  // weight rows of a CTA's half of a tile
constexpr int kStepBytes = 128;          // K bytes of a step: one row of the swizzle atom
constexpr int kABytes = kM * kStepBytes;
constexpr int kMaxStages = 9;
constexpr int kMaxTiles = 1 << 30;
constexpr int kMinSteps = 4;             // steps of each pair that shares a tile's K, at least
constexpr unsigned long long kCopyDrainNs = 10000000ull;
constexpr unsigned long long kShortLimitNs = 1000000ull;
constexpr int kGroup = 4;                // steps whose scales are handed over together
constexpr int kNRound = 64;              // a tile's columns are a multiple of this

// Warps: 16 of epilogue, TMA, MMA, two of scales, four of gather.
constexpr int kEpiWarps = 16, kTmaWarp = 16, kMmaWarp = 17, kScaleWarp0 = 18, kGatherWarp0 = 20;
constexpr int kScaleThreads = 64, kGatherWarps = 4;
constexpr int kThreads = 768;
// Registers of a thread, 8-bit kernel: 80 at launch (65536 / 768 in steps of 8), then moved to the
// epilogue, which keeps 64 sums a thread.
constexpr int kLaunchRegs = 80, kEpiRegs = 96, kOtherRegs = 48;
static_assert(512 * kEpiRegs + 256 * kOtherRegs <= kThreads * kLaunchRegs, "register split");
static_assert(NVFP4_MAX_EXPERTS <= 8 * 32, "eight experts a lane");

// Output staging of an epilogue warp (bf16): 16 rows of y, 32 neighbouring outputs of each. The pitch of
// 80 bytes puts the eight 16-byte rows of a stmatrix on different banks.
constexpr int kStgRows = 16, kStgPitch = 80;

template <bool FP8, int NT>
struct Cfg {
    static constexpr int kBoxRows = kNRound / 2;                 // heights of a box of x: this times
    static constexpr int kBoxes = NT / kNRound;                  // ... 1 .. kBoxes
    static constexpr int kStage = kABytes + NT / 2 * kStepBytes;
    static constexpr int kStages = std::min(kMaxStages, (192 * 1024) / kStage);
    static constexpr int kBufs = 512 / NT;                       // tensor-memory buffers of NT columns
    static constexpr int kCols = NT / 4;                         // columns of an epilogue warp, at most
    static constexpr int kOffScales = kStages * kStage;          // [2][kGroup][NT] fp32
    static constexpr int kOffStg = kOffScales + (FP8 ? 2 * kGroup * NT * 4 : 0);
    static constexpr int kOffBars = kOffStg + kEpiWarps * kStgRows * kStgPitch;
    static constexpr int kNumBars = 2 * kStages + 2 * kBufs + 4 + 1;
    static constexpr int kOffTab = kOffBars + kNumBars * 8 + 16; // tile prefix [E + 1], first position [E], rows [E]
    static constexpr int kSmem = 1024 + kOffTab + (3 * NVFP4_MAX_EXPERTS + 1) * 4;
    static_assert(NT % kNRound == 0 && NT <= 256 && kStage % 1024 == 0 && kCols % 16 == 0, "swizzle atoms, fragments");
    static_assert(kSmem <= 227 * 1024, "shared memory");
    static_assert(4 * NT / 16 * 2048 <= kOffScales, "exchanged sums fit in the ring");
};

struct TcRowMaps {
    CUtensorMap w, x[4];   // x: boxes of one to kBoxes times Cfg::kBoxRows rows; x[0] single rows to gather
};

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
// waits for every store of the thread, cost 1 us a step.
__device__ __forceinline__ void arrive_cluster(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" :: "r"(cluster_addr) : "memory");
}

// One look at a barrier's phase, without suspending the thread.
__device__ __forceinline__ bool mbar_test_wait(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
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
};

// One lane of the (converged) warp. The tensor-core and TMA instructions take uniform registers: under
// `lane == 0` the compiler cannot know that one thread is left and builds a loop around each.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

template <bool FP8>
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    if constexpr (FP8)
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
            " tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}"
            :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
    else
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
            " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}"
            :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}
// Arrive on this barrier in both CTAs (cluster mask) once every MMA issued so far by this thread has completed.
__device__ __forceinline__ void commit_pair(uint64_t* bar, uint16_t mask) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
        :: "r"(su32(bar)), "h"(mask) : "memory");
}
// Instruction descriptor of kind::f8f6f4: E4M3 A and B (format 0, both K-major), fp32 D, M x N.
__device__ __forceinline__ uint32_t e4m3_idesc(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
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

// (a.x, a.y) += (v.x, v.y) * (s.x, s.y), each fused and rounded once: the packed fp32 pipe.
__device__ __forceinline__ void fma2(float2& a, float vx, float vy, float sx, float sy) {
    asm("{\n .reg .b64 a, v, s;\n mov.b64 a, {%0, %1};\n mov.b64 v, {%2, %3};\n mov.b64 s, {%4, %5};\n"
        " fma.rn.f32x2 a, v, s, a;\n mov.b64 {%0, %1}, a;\n}"
        : "+f"(a.x), "+f"(a.y) : "f"(vx), "f"(vy), "f"(sx), "f"(sy));
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
struct Tile {
    int e, r0, n, m0;   // expert, first list position, rows, first weight row
    __device__ __forceinline__ int mma_n() const { return (n + kNRound - 1) & ~(kNRound - 1); }
};

// The tiles of a pair: token tile tt (numbered over the experts) and weight tile mt of i = first, first +
// step, ... below total. tab: token-tile prefix [E + 1], first position [E], rows [E].
struct Walk {
    const int* tab;
    int E, m_tiles, i, step, total, tt, mt, dt, dm;

    __device__ __forceinline__ Walk(const int* tab_, int E_, int m_tiles_, int first, int step_, int total_)
        : tab(tab_), E(E_), m_tiles(m_tiles_), i(first), step(step_), total(total_), tt(first / m_tiles_),
          mt(first - tt * m_tiles_), dt(step_ / m_tiles_), dm(step_ - dt * m_tiles_) {}
    __device__ __forceinline__ bool more() const { return i < total; }
    __device__ __forceinline__ void next() {
        i += step, tt += dt, mt += dm;
        if (mt >= m_tiles) mt -= m_tiles, ++tt;
    }
    // By all lanes of a warp: the last expert whose first token tile is at most tt (an empty one before it
    // has the same first), found among every eighth and then among eight.
    __device__ __forceinline__ Tile tile() const {
        const int lane = threadIdx.x & 31;
        const int b = __popc(__ballot_sync(0xffffffffu, 8 * lane < E && tab[min(8 * lane, E)] <= tt)) - 1;
        const int e8 = 8 * b + (lane & 7);
        const int e = 8 * b + __popc(__ballot_sync(0xffffffffu, lane < 8 && e8 < E && tab[min(e8, E)] <= tt)) - 1;
        const int cnt = tab[E + 1 + E + e], parts = tab[e + 1] - tab[e], l = tt - tab[e];
        // nearly equal parts in multiples of kNRound: parts = ceil(cnt / NT), so none is empty
        const int per = parts == 1 ? cnt : ((cnt + parts - 1) / parts + kNRound - 1) & ~(kNRound - 1);
        Tile t;
        t.e = uniform(e);
        t.r0 = uniform(tab[E + 1 + e] + l * per);
        t.n = uniform(min(per, cnt - l * per));
        t.m0 = mt * (2 * kM);
        return t;
    }
};

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

// SPLITS: pairs of a cluster, which share a tile's K.
template <bool FP8, int NT, int SPLITS>
__global__ void __cluster_dims__(2 * SPLITS, 1, 1) __launch_bounds__(kThreads, 1)
rows_tc_kernel(const RowsProduct P, const __grid_constant__ TcRowMaps maps, int m_tiles, int max_tiles, WsHeader* hdr,
               unsigned long long wait_limit) {
    using C = Cfg<FP8, NT>;
    extern __shared__ uint8_t rows_smem_raw[];
    // the swizzle pattern follows shared-memory address bits: align the base to 1024 (both CTAs of a
    // pair have the same layout)
    uint8_t* sm = rows_smem_raw + ((1024u - (su32(rows_smem_raw) & 1023u)) & 1023u);
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    // CTA of its pair, pair of its cluster
    const int crank = (int)cluster_rank(), rank = crank & 1, pair = SPLITS == 1 ? 0 : crank >> 1, first_rank = 2 * pair;
    const uint16_t pair_mask = (uint16_t)(3u << first_rank);

    float* scale_ring = reinterpret_cast<float*>(sm + C::kOffScales);
    uint64_t* full = reinterpret_cast<uint64_t*>(sm + C::kOffBars);   // step landed (first CTA: in both)
    uint64_t* empty = full + C::kStages;                               // MMAs done with the step
    uint64_t* acc_full = empty + C::kStages;                           // tensor-memory buffer summed
    uint64_t* acc_empty = acc_full + C::kBufs;                         // first CTA: ... and read in both
    uint64_t* sc_full = acc_empty + C::kBufs;                          // [2] scales of a group of steps written
    uint64_t* sc_empty = sc_full + 2;                                  // ... and read
    uint64_t* done = sc_empty + 2;                                     // every MMA of the pair
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* tab = reinterpret_cast<int*>(sm + C::kOffTab);

    if (warp == kMmaWarp) {
        if (lane == 0) {
            for (int i = 0; i < C::kStages; ++i) {
                // the TMA warp, each gather warp, and in the first CTA the second's word
                mbar_init(&full[i], 1 + (P.gather ? kGatherWarps : 0) + (rank == 0 ? 1 : 0));
                mbar_init(&empty[i], 1);
            }
            for (int i = 0; i < C::kBufs; ++i) {
                mbar_init(&acc_full[i], 1);
                mbar_init(&acc_empty[i], 2 * kEpiWarps);
            }
            for (int i = 0; i < 2; ++i) {
                mbar_init(&sc_full[i], kScaleThreads);
                mbar_init(&sc_empty[i], kEpiWarps);
            }
            mbar_init(done, 1);
            *abort_flag = 0;
            fence_mbar_init();
        }
        __syncwarp();
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" :: "r"(su32(tmem_slot)), "n"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    pdl_wait_then_trigger();       // barriers and tensor memory are set up under the kernel before
    if (warp == 0) {
        // tiles of every expert: eight experts a lane, then a prefix sum over the lanes
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
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();       // barriers are ready in both CTAs
    tc_fence_after();
    const uint32_t tmem = (uint32_t)uniform((int)*tmem_slot), sm_base = su32(sm);
    // overlapping groups of a malformed list could add up to more tiles than the host counted: those are left
    // out, in particular a second tile of a cluster of several pairs (which has as many clusters as tiles)
    constexpr int kCluster = 2 * SPLITS;
    const int total = uniform((int)min((long long)tab[P.E] * m_tiles, (long long)max_tiles));
    const int kStepK = FP8 ? 128 : 64;
    const int nk = (P.K + kStepK - 1) / kStepK;
    const int s_begin = nk * pair / SPLITS, s_end = nk * (pair + 1) / SPLITS;      // this pair's steps
    const Walk tiles(tab, P.E, m_tiles, blockIdx.x / kCluster, gridDim.x / kCluster, total);
    const Waiter wait{abort_flag, map_rank(su32(const_cast<int*>(abort_flag)), (uint32_t)crank ^ 1u), hdr, wait_limit};

    // one tile at most to a cluster of several pairs
    const Exchange<C::kCols, SPLITS> exchange{sm, pair, rank};

    // A warp that issued copies for `step` steps waits until the last fill of each stage has landed before
    // the CTA may exit. (After an abort other warps may not have issued theirs, so that the phase stays
    // open: 10 ms is a thousand copies.)
    auto drain = [&](int step) {
        for (int s = max(0, step - C::kStages); s < step; ++s)
            mbar_wait_bounded(&full[s % C::kStages], (s / C::kStages) & 1, kCopyDrainNs);
    };

    if (warp >= kEpiWarps) {
        if (FP8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kOtherRegs));
        if (warp == kTmaWarp) {
            int step = 0;
            bool ok = true;
#pragma unroll 1
            for (Walk at = tiles; at.more() && ok; at.next()) {
                const Tile t = at.tile();
                const int share = t.mma_n() / 2;                                // rows of x here
                const int wy = t.e * P.N + t.m0 + rank * kM;
                const CUtensorMap* mx = &maps.x[share / C::kBoxRows - 1];
                const uint32_t bytes = kABytes + (P.gather ? 0 : share * kStepBytes);
#pragma unroll 1
                for (int s = s_begin; s < s_end; ++s, ++step) {
                    const int st = step % C::kStages, u = step / C::kStages;
                    if (u > 0) ok = wait(&empty[st], (u - 1) & 1);
                    if (!ok) break;
                    const uint32_t a = sm_base + st * C::kStage, b = a + kABytes;
                    if (elect_one()) {
                        mbar_arrive_expect_tx(&full[st], bytes);
                        tma_load_2d(a, &maps.w, s * kStepK, wy, &full[st]);
                        if (!P.gather) tma_load_2d(b, mx, s * kStepK, t.r0 + rank * share, &full[st]);
                    }
                }
            }
            if (lane == 0) drain(step);
        } else if (warp == kMmaWarp) {
            int st = 0, buf = 0;
            uint32_t st_par = 0, buf_par = 1;          // an unused buffer's "empty" phase counts as over
            bool ok = true;
            const uint64_t stage0 = sw128_desc(sm_base);
#pragma unroll 1
            for (Walk at = tiles; at.more() && ok; at.next()) {
                const int N = at.tile().mma_n();
                const uint32_t idesc = FP8 ? e4m3_idesc(2 * kM, N) : f16_idesc(2 * kM, N);
#pragma unroll 1
                for (int s = s_begin; s < s_end; ++s) {
                    const bool first = FP8 || s == s_begin, sum_done = FP8 || s == s_end - 1;
                    ok = wait(&full[st], st_par);
                    if (!ok) break;
                    if (rank != 0) {
                        if (elect_one()) arrive_cluster(map_rank(su32(&full[st]), first_rank));
                    } else {
                        if (first) ok = wait(&acc_empty[buf], buf_par);
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t a = stage0 + st * (C::kStage / 16), b = a + kABytes / 16;
                        if (elect_one()) {
#pragma unroll
                            for (int j = 0; j < kStepBytes / 32; ++j)      // 32 bytes of K an MMA: 2 address units
                                mma_pair<FP8>(tmem + buf * NT, a + 2 * j, b + 2 * j, idesc, !first || j != 0);
                            commit_pair(&empty[st], pair_mask);
                            if (sum_done) commit_pair(&acc_full[buf], pair_mask);
                        }
                        if (sum_done && ++buf == C::kBufs) buf = 0, buf_par ^= 1;
                    }
                    if (++st == C::kStages) st = 0, st_par ^= 1;
                }
            }
            // no MMA still reads or writes either CTA's memory, nor has an arrival on the way to it, when it is freed
            if (elect_one()) {
                if (rank == 0) commit_pair(done, pair_mask);
                drain_wait(done, 0);
            }
        } else if (warp >= kGatherWarp0) {
            if (P.gather) {
                // copies of four rows, in turn over the warps: at most kPer a warp and step; lane 4 j + r has
                // row r of this warp's copy j
                constexpr int kPer = NT / 2 / 4 / kGatherWarps;
                const int w = warp - kGatherWarp0;
                int step = 0;
                bool ok = true;
#pragma unroll 1
                for (Walk at = tiles; at.more() && ok; at.next()) {
                    const Tile t = at.tile();
                    const int share = t.mma_n() / 2, copies = share / 4;
                    const int l = 4 * (w + kGatherWarps * (lane >> 2)) + (lane & 3);
                    const int col = rank * share + l;
                    int src = l < share && col < t.n ? x_row(P, t.r0 + col) : -1;
                    if (src < 0) src = P.x_rows;                     // past the last row: zeros
                    const int mine = (copies - w + kGatherWarps - 1) / kGatherWarps;
#pragma unroll 1
                    for (int s = s_begin; s < s_end; ++s, ++step) {
                        const int st = step % C::kStages, u = step / C::kStages;
                        if (u > 0) ok = wait(&empty[st], (u - 1) & 1);
                        if (!ok) break;
                        const uint32_t b = sm_base + st * C::kStage + kABytes + w * 4 * kStepBytes;
                        if (elect_one()) mbar_arrive_expect_tx(&full[st], mine * 4 * kStepBytes);
#pragma unroll
                        for (int j = 0; j < kPer; ++j) {
                            if (j >= mine) break;
                            const int r0 = __shfl_sync(0xffffffffu, src, 4 * j);
                            const int r1 = __shfl_sync(0xffffffffu, src, 4 * j + 1);
                            const int r2 = __shfl_sync(0xffffffffu, src, 4 * j + 2);
                            const int r3 = __shfl_sync(0xffffffffu, src, 4 * j + 3);
                            if (elect_one())
                                tma_gather4(b + j * (kGatherWarps * 4 * kStepBytes), &maps.x[0], s * kStepK, r0, r1, r2,
                                            r3, &full[st]);
                        }
                    }
                }
                if (lane == 0) drain(step);
            }
        } else if constexpr (FP8) {
            const int th = tid - kScaleWarp0 * 32;           // columns th, th + 64, ...
            constexpr int kPer = NT / kScaleThreads;
            const int KB = nk, NB = (P.N + 127) >> 7;
            int grp = 0;
            bool ok = true;
#pragma unroll 1
            for (Walk at = tiles; at.more() && ok; at.next()) {
                const Tile t = at.tile();
                const int nb = (t.m0 >> 7) + rank;           // past the matrix: scales 0
                const float* wsc = nb < NB ? P.ws + ((size_t)t.e * NB + nb) * KB : P.ws;
                int xs[kPer];
                float next[kGroup][kPer];
                auto load = [&](int s0) {
#pragma unroll
                    for (int d = 0; d < kGroup; ++d)
#pragma unroll
                        for (int j = 0; j < kPer; ++j)
                            next[d][j] = xs[j] >= 0 && s0 + d < s_end ? P.xs[(size_t)xs[j] * KB + s0 + d] : 0.f;
                };
#pragma unroll
                for (int j = 0; j < kPer; ++j) {
                    const int col = th + kScaleThreads * j;
                    xs[j] = nb < NB && col < t.n ? x_row(P, t.r0 + col) : -1;
                }
                load(s_begin);
#pragma unroll 1
                for (int s = s_begin; s < s_end; s += kGroup, ++grp) {
                    const int slot = grp & 1, u = grp >> 1;
                    if (u > 0) ok = wait(&sc_empty[slot], (u - 1) & 1);
                    if (!ok) break;
#pragma unroll
                    for (int d = 0; d < kGroup; ++d) {
                        const float sw = s + d < s_end ? wsc[s + d] : 0.f;
#pragma unroll
                        for (int j = 0; j < kPer; ++j)
                            scale_ring[(slot * kGroup + d) * NT + th + kScaleThreads * j] =
                                xs[j] >= 0 ? next[d][j] * sw : 0.f;
                    }
                    mbar_arrive(&sc_full[slot]);
                    if (s + kGroup < s_end) load(s + kGroup);
                }
            }
        }
        if (SPLITS > 1 && tiles.more()) exchange.join();
    } else {
        if (FP8) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(kEpiRegs));
        const int q = warp & 3, part = warp >> 2;          // lanes 32 q .., a quarter of the columns
        uint8_t* stg = sm + C::kOffStg + warp * (kStgRows * kStgPitch);
        const int p = lane & 3;
        const uint32_t first_acc_empty = map_rank(su32(acc_empty), first_rank);
        int use = 0, grp = 0;      // buffers (8-bit: steps) and groups of scales read so far
        bool ok = true;
#pragma unroll 1
        for (Walk at = tiles; at.more(); at.next()) {
            const Tile t = at.tile();
            const int width = t.mma_n() / 4, c0 = part * width;            // this warp's columns of the tile
            const uint32_t lanes = tmem + ((uint32_t)(32 * q) << 16) + c0;
            const int n0 = t.m0 + rank * kM + 32 * q;                      // first output
            // lane j (< 16): row of y of column c0 + c + j
            auto out_row = [&](int c) {
                const int col = c0 + c + (lane & 15);
                return c < width && col < t.n ? y_row(P, t.r0 + col) : -1;
            };
            if constexpr (FP8) {
                const int cols = uniform(min(width, t.n - c0));
                float2 acc[C::kCols / 2];
#pragma unroll
                for (int j = 0; j < C::kCols / 2; ++j) acc[j] = make_float2(0.f, 0.f);
#pragma unroll 1
                for (int s0 = s_begin; s0 < s_end && ok; s0 += kGroup, ++grp) {
                    const int slot = grp & 1;
                    ok = wait(&sc_full[slot], (grp >> 1) & 1);
                    if (!ok) break;
                    const float* sc = scale_ring + slot * (kGroup * NT) + c0 + 2 * p;
#pragma unroll 1
                    for (int s = s0; s < min(s0 + kGroup, s_end); ++s, ++use, sc += NT) {
                        const int buf = use % C::kBufs;
                        ok = wait(&acc_full[buf], (use / C::kBufs) & 1);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll
                        for (int c = 0; c < C::kCols; c += 16) {
                            if (c >= cols) break;                       // padding is neither read nor written
                            float v[16];
                            tmem_ld_frag(lanes + buf * NT + c, v);
                            const float2 f0 = *reinterpret_cast<const float2*>(sc + c);
                            const float2 f1 = *reinterpret_cast<const float2*>(sc + c + 8);
                            tmem_wait16(v);
#pragma unroll
                            for (int h = 0; h < 4; ++h) {
                                const int k = 8 * (h >> 1) + 2 * (h & 1);
                                fma2(acc[c / 2 + h], v[k], v[k + 1], f0.x, f0.y);
                                fma2(acc[c / 2 + 4 + h], v[k + 4], v[k + 5], f1.x, f1.y);
                            }
                        }
                        tc_fence_before();
                        __syncwarp();
                        if (elect_one()) arrive_cluster(first_acc_empty + 8 * buf);
                    }
                    if (ok && lane == 0) mbar_arrive(&sc_empty[slot]);
                }
                const auto sums = [&](int c, float (&v)[16]) {
                    const bool bad = *abort_flag != 0;
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            const int k = 8 * (h >> 1) + 4 * j + 2 * (h & 1);
                            v[k] = bad ? __uint_as_float(0x7FC00000u) : acc[c / 2 + 4 * j + h].x;
                            v[k + 1] = bad ? __uint_as_float(0x7FC00000u) : acc[c / 2 + 4 * j + h].y;
                        }
                };
                if constexpr (SPLITS > 1) exchange.send(sums, t, width, c0, part, q);
#pragma unroll
                for (int c = 0; c < C::kCols; c += 16) {
                    if (c >= width || c0 + c >= t.n) break;
                    float v[16];
                    sums(c, v);
                    if (SPLITS > 1 && !exchange.finish(v, c, width, part, q)) continue;
                    store_frag(P, v, out_row(c), n0, stg);
                }
            } else {
                const int buf = use % C::kBufs;
                if (ok) ok = wait(&acc_full[buf], (use / C::kBufs) & 1);
                tc_fence_after();
                const auto sums = [&](int c, float (&v)[16]) {
                    if (ok) {
                        tmem_ld_frag(lanes + buf * NT + c, v);
                        tmem_wait16(v);
                    }
                    if (*abort_flag)
#pragma unroll
                        for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(0x7FC00000u);
                };
                if constexpr (SPLITS > 1) exchange.send(sums, t, width, c0, part, q);
#pragma unroll
                for (int c = 0; c < C::kCols; c += 16) {
                    if (c >= width || c0 + c >= t.n) break;
                    float v[16];
                    sums(c, v);
                    if (SPLITS > 1 && !exchange.finish(v, c, width, part, q)) continue;
                    store_frag(P, v, out_row(c), n0, stg);
                }
                tc_fence_before();
                __syncwarp();
                if (ok && lane == 0) arrive_cluster(first_acc_empty + 8 * buf);
                ++use;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();       // neither CTA is still read, written or signalled by the other
    if (warp == kMmaWarp) {
        __syncwarp();
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" :: "r"(tmem), "n"(512) : "memory");
    }
}

// [rows, K] elements of 1 or 2 bytes, read as box_rows x 128 bytes, 128-byte swizzled in shared memory.
bool encode_rows(PFN_cuTensorMapEncodeTiled_v12000 fn, CUtensorMap* m, const void* base, bool fp8, uint64_t K,
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

// Sets the kernel up on the current device, once, and says how many of its clusters run there at a time
// (clusters of eight CTAs do not fill every GPC).
template <bool FP8, int NT, int SPLITS>
cudaError_t resident_clusters(const DeviceInfo& dev, int* clusters) {
    using C = Cfg<FP8, NT>;
    static std::atomic<int> known[64];           // by device: one more than the clusters
    int n = known[dev.device].load(std::memory_order_acquire) - 1;
    if (n < 0) {
        const auto kernel = rows_tc_kernel<FP8, NT, SPLITS>;
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
        if (e != cudaSuccess) return e;
        // the register split waits forever for registers that the launch did not bring
        cudaFuncAttributes a;
        if ((e = cudaFuncGetAttributes(&a, kernel)) != cudaSuccess) return e;
        if (FP8 && a.numRegs != kLaunchRegs) return cudaErrorInvalidConfiguration;
        cudaLaunchAttribute attr{};
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = 2 * SPLITS;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(2 * SPLITS * dev.num_sms);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = C::kSmem;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        if ((e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg)) != cudaSuccess) return e;
        known[dev.device].store(n + 1, std::memory_order_release);
    }
    *clusters = n;
    return cudaSuccess;
}

// How a product runs: columns of a tile, pairs to a tile, tiles at most, and an estimate of its time.
struct Plan {
    int nt, splits;
    long long tiles;
    float us;
};

// Tiles of NT columns. The estimate takes the rows to be even over the experts; its figures (us) are fitted to
// calls of one to three rounds of tiles: a step of N columns 0.08 + 0.00195 N in 8 bits, 0.05 + 0.0007 N in bf16;
// 2 to write a tile out, 0.5 + 0.009 N to exchange its sums. It leaves out what every plan pays, 2 to 4 us, and is
// too low where four pairs share 256 columns of a long K (256 x 2048 x 8192: 14.1 for 19.1 in 8 bits, 12.1 for 18.7
// in bf16).
template <bool FP8, int NT>
cudaError_t plan_tiles(const RowsProduct& P, const DeviceInfo& dev, Plan* best) {
    const int m_tiles = (P.N + 2 * kM - 1) / (2 * kM), nk = (P.K * (FP8 ? 1 : 2) + kStepBytes - 1) / kStepBytes;
    const int groups = std::min(P.R, P.E), rows = (P.R + groups - 1) / groups;
    Plan p;
    p.nt = NT;
    // tiles at most: every expert has rows, and its last tile one
    p.tiles = ((P.R - groups) / NT + groups) * (long long)m_tiles;
    // as many pairs to a tile as the device runs at a time, where each has kMinSteps steps (us, 1 / 2 or 4 pairs a
    // tile, 8 bits: 64 rows x 2048 x 8192 24.1 / 9.4, 77 x 5003 x 2000 13.2 / 10.7, 64 x 8192 x 2048 8.9 / 8.4)
    int c2 = 0, c4 = 0;
    if (nk >= 2 * kMinSteps && 2 * p.tiles <= dev.num_sms / 2)
        if (cudaError_t e = resident_clusters<FP8, NT, 2>(dev, &c2); e != cudaSuccess) return e;
    if (nk >= 4 * kMinSteps && 4 * p.tiles <= dev.num_sms / 2)
        if (cudaError_t e = resident_clusters<FP8, NT, 4>(dev, &c4); e != cudaSuccess) return e;
    p.splits = p.tiles <= c4 ? 4 : p.tiles <= c2 ? 2 : 1;
    const int parts = (rows + NT - 1) / NT, n = ((rows + parts - 1) / parts + kNRound - 1) / kNRound * kNRound;
    const long long even = (long long)groups * parts * m_tiles, rounds = (even + dev.num_sms / 2 - 1) / (dev.num_sms / 2);
    const float step = FP8 ? 0.08f + 0.00195f * n : 0.05f + 0.0007f * n;
    p.us = rounds * ((nk + p.splits - 1) / p.splits * step + 2.0f + (p.splits > 1 ? 0.5f + 0.009f * n : 0.0f));
    if (p.us < best->us) *best = p;
    return cudaSuccess;
}

template <bool FP8, int NT, int SPLITS>
cudaError_t launch_clusters(const RowsProduct& P, const TcRowMaps& maps, int tiles, WsHeader* hdr,
                            const DeviceInfo& dev, uint64_t wait_limit, cudaStream_t s) {
    int resident = 0;
    if (cudaError_t e = resident_clusters<FP8, NT, SPLITS>(dev, &resident); e != cudaSuccess) return e;
    if (resident < 1) return cudaErrorInvalidConfiguration;
    const int clusters = SPLITS > 1 ? tiles : std::min(tiles, resident), m_tiles = (P.N + 2 * kM - 1) / (2 * kM);
    return launch_pdl(rows_tc_kernel<FP8, NT, SPLITS>, 2 * SPLITS * clusters, kThreads, Cfg<FP8, NT>::kSmem, s, P, maps,
                      m_tiles, tiles, hdr, (unsigned long long)wait_limit);
}

template <bool FP8, int NT>
cudaError_t launch_tc(const RowsProduct& P, const Plan& plan, WsHeader* hdr, const DeviceInfo& dev, uint64_t wait_limit,
                      cudaStream_t s) {
    using C = Cfg<FP8, NT>;
    PFN_cuTensorMapEncodeTiled_v12000 fn = tensor_map_encoder();
    TcRowMaps maps;
    if (fn == nullptr || !encode_rows(fn, &maps.w, P.w, FP8, P.K, (uint64_t)P.E * P.N, kM)) return cudaErrorInvalidValue;
    for (int i = 0; i < (P.gather ? 1 : C::kBoxes); ++i)
        if (!encode_rows(fn, &maps.x[i], P.x, FP8, P.K, P.x_rows, P.gather ? 1 : (i + 1) * C::kBoxRows))
            return cudaErrorInvalidValue;
    const int tiles = (int)plan.tiles;
    if (plan.splits == 4) return launch_clusters<FP8, NT, 4>(P, maps, tiles, hdr, dev, wait_limit, s);
    if (plan.splits == 2) return launch_clusters<FP8, NT, 2>(P, maps, tiles, hdr, dev, wait_limit, s);
    return launch_clusters<FP8, NT, 1>(P, maps, tiles, hdr, dev, wait_limit, s);
}

// Small tiles have more and smaller stages and more tensor-memory buffers, and there are more of them to go round;
// large ones read the weights fewer times. Measured (us):
//   tiles of 64 / 256 columns: 256 experts of 1024 x 2048 with 32 rows each, bf16 171 / 175, 8 bits 95 / 101
//   tiles of 128 / 256: 8192 x 2048 in 8 bits, 128 rows 9.2 / 10.8, 256 rows 9.8 / 13.9, 1024 rows 26.6 / 25.6;
//     256 experts with uneven rows, on average 94: bf16 187 / 191; 128: bf16 206 / 204, 8 bits 134 / 154; with 160
//     even ones: 8 bits 139 / 125
//   64 / 128 / 256, 256 experts of 1024 x 2048 with 62 rows on average, the longest with 82: bf16 173 / 171 / 177,
//     8 bits 95 / 93 / 98; with 913: bf16 179 / 173 / 177, 8 bits 102 / 96 / 104; 31 on average, the longest with
//     470: bf16 164 / 164 / 172, 8 bits 89 / 87 / 98
// So: 64 where the experts' rows, were they even, fit (for very uneven rows just below that up to 9 % slower than
// 128); otherwise what the estimate says, and 128 where it is the same for both.
template <bool FP8>
cudaError_t launch_any(const RowsProduct& P, WsHeader* hdr, const DeviceInfo& dev, uint64_t wait_limit,
                       cudaStream_t s) {
    Plan plan{};
    plan.us = 3.0e38f;
    const int groups = std::min(P.R, P.E), rows = (P.R + groups - 1) / groups;
    cudaError_t e;
    if (rows <= 64) {
        if ((e = plan_tiles<FP8, 64>(P, dev, &plan)) != cudaSuccess) return e;
    } else {
        if ((e = plan_tiles<FP8, 128>(P, dev, &plan)) != cudaSuccess) return e;
        if ((e = plan_tiles<FP8, 256>(P, dev, &plan)) != cudaSuccess) return e;
    }
    if (plan.tiles > kMaxTiles) return cudaErrorInvalidConfiguration;
    if (plan.nt == 64) return launch_tc<FP8, 64>(P, plan, hdr, dev, wait_limit, s);
    if (plan.nt == 128) return launch_tc<FP8, 128>(P, plan, hdr, dev, wait_limit, s);
    return launch_tc<FP8, 256>(P, plan, hdr, dev, wait_limit, s);
}

}  // namespace

cudaError_t launch_rows_tc(const RowsProduct& P, WsHeader* hdr, const DeviceInfo& dev, uint64_t wait_limit,
                           cudaStream_t s) {
    return P.xs != nullptr ? launch_any<true>(P, hdr, dev, wait_limit, s)
                           : launch_any<false>(P, hdr, dev, wait_limit, s);
}

}  // namespace nvfp4
