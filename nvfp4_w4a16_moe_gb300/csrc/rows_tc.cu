// Products of many rows with one matrix or with each expert's matrix on the 5th-generation tensor
// cores: y[o(r), n] = sum_k W[e(r)][n, k] x[i(r), k], in bf16 or in E4M3 with block scales.
//
// A pair of CTAs (cluster of 2, cta_group::2) computes a tile of 256 weight rows of one expert times
// up to NT of its list positions. The weights are the MMA's A operand (M = 256: 128 rows in each
// CTA's shared memory) and the rows of x its B operand (N = the tile's rows, rounded up to 32; each
// CTA holds half of them), so an expert with few rows costs few MMA cycles, and any number of rows
// per expert works without padding in memory. The pair is what feeds the tensor cores: one CTA alone
// (128 x 256 tiles) needs 48 KB of operands per 64 columns of K from L2 where a CTA of a pair needs 32.
//
// An expert's rows are cut into tiles of nearly equal size. The tiles of the whole call are numbered
// over the experts (prefix sums over the offsets, made by every CTA for itself: the host never sees the
// counts), and a persistent grid of pairs walks them.
//
// Warp roles of a CTA (both CTAs of a pair but where said):
//   TMA warp: brings step s (128 bytes of K) of the CTA's weight rows (one box) and, for rows in list
//     order, of its rows of x (boxes of 64 and 16) into a ring of 128-byte-swizzled stages. Coordinates
//     past a matrix read zeros, which also pads K. (A box costs about as much as 64 rows however few it
//     has: boxes of 16 alone ran the ring at half its rate.)
//   Gather warps (rows read through the list): 16-byte cp.async from the tokens' rows straight into
//     the swizzled stage, so no permuted copy of x is ever written. (TMA's own gather of four rows a
//     copy measured 28 ns a copy, 4 times the MMA time of a step.)
//   MMA warp: in the pair's first CTA, four MMAs a step for both. In the second CTA it tells the first
//     that the step's operands have landed here.
//     bf16 sums a whole tile in one tensor-memory buffer. 8-bit operands carry a scale per 128 of K,
//     so each step starts a buffer of its own from zero.
//   Epilogue warps: bf16: read the finished tile. 8-bit: read every step's buffer, multiply each column
//     with its scale and add it to the tile's sum in registers (fp32), while the MMAs fill the next
//     buffer. Lane = weight row, column = row of x, so the stores of a warp are 32 neighbouring
//     outputs of one row of y.
//   Scale warps (8-bit): x_scale * w_scale of every column of a step, in a ring of their own.
// The buffers of tensor memory (512 / NT) let the next tile's or step's MMAs run under the epilogue.
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
constexpr int kBigBox = 64, kSmallBox = 16;   // rows of x per box (rows in list order)
constexpr int kMaxStages = 10;
constexpr int kScaleSlots = 8;
constexpr int kMaxTiles = 1 << 30;

// Warps: two warpgroups of epilogue, one of TMA, MMA and scales, one of gather.
constexpr int kEpiWarps = 8, kTmaWarp = 8, kMmaWarp = 9, kScaleWarp0 = 10, kGatherWarp0 = 12;
constexpr int kScaleThreads = 64, kGatherThreads = 128;
constexpr int kThreads = 512;
// Registers of a thread, 8-bit kernel: 128 at launch (65536 / 512), then moved to the epilogue, which
// keeps 128 sums a thread. 256 * 208 + 256 * 48 = 512 * 128.
constexpr int kLaunchRegs = 128, kEpiRegs = 208, kOtherRegs = 48;
static_assert(256 * kEpiRegs + 256 * kOtherRegs <= kThreads * kLaunchRegs, "register split");

template <bool FP8, int NT>
struct Cfg {
    static constexpr int kStage = kABytes + NT / 2 * kStepBytes;
    static constexpr int kStages = std::min(kMaxStages, (200 * 1024) / kStage);
    static constexpr int kBufs = std::min(8, 512 / NT);          // tensor-memory buffers of NT columns
    static constexpr int kCols = NT / 2;                         // columns of an epilogue warp
    static constexpr int kOffScales = kStages * kStage;          // [kScaleSlots][NT] fp32
    static constexpr int kOffBars = kOffScales + (FP8 ? kScaleSlots * NT * 4 : 0);
    static constexpr int kNumBars = 4 * kStages + 2 * kBufs + 2 * kScaleSlots + 1;
    static constexpr int kOffTab = kOffBars + kNumBars * 8 + 16; // tile prefix [E + 1], first position [E], rows [E]
    static constexpr int kSmem = 1024 + kOffTab + (3 * NVFP4_MAX_EXPERTS + 1) * 4;
    static_assert(NT % 64 == 0 && NT <= 256 && kStage % 1024 == 0, "two column halves of 32s, swizzle atoms");
    static_assert(kSmem <= 227 * 1024, "shared memory");
};

struct TcRowMaps {
    CUtensorMap w, x_big, x_small;
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

// Bounded wait on a barrier that either CTA of the pair, or its MMAs, arrive on. One that runs out
// records the timeout and raises the abort flag of both CTAs; once raised, every wait gives up.
struct Waiter {
    volatile int* abort_flag;
    uint32_t peer_flag;          // the other CTA's flag
    WsHeader* hdr;
    unsigned long long limit_ns;

    // By all lanes of a warp; the answer is the same in each.
    __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) const {
#pragma unroll 1
        for (int i = 0; i < 64; ++i)
            if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        const unsigned long long t0 = global_timer_ns();
        while (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) {
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
// Arrive on this barrier in both CTAs once every MMA issued so far by this thread has completed.
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
        :: "r"(su32(bar)), "h"((uint16_t)3) : "memory");
}
// Instruction descriptor of kind::f8f6f4: E4M3 A and B (format 0, both K-major), fp32 D, M x N.
__device__ __forceinline__ uint32_t e4m3_idesc(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// 32 consecutive fp32 columns of this thread's tensor-memory lane; valid after tmem_wait32.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
          "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
          "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
          "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(taddr));
}
// The loads so far are done; the values pass through, so that no use of them moves before the wait.
__device__ __forceinline__ void tmem_wait32(float (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
        : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
          "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]),
          "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]),
          "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31])
        :: "memory");
}

// (a.x, a.y) += (v.x, v.y) * (s.x, s.y), each fused and rounded once: the packed fp32 pipe.
__device__ __forceinline__ void fma2(float2& a, float vx, float vy, float sx, float sy) {
    asm("{\n .reg .b64 a, v, s;\n mov.b64 a, {%0, %1};\n mov.b64 v, {%2, %3};\n mov.b64 s, {%4, %5};\n"
        " fma.rn.f32x2 a, v, s, a;\n mov.b64 {%0, %1}, a;\n}"
        : "+f"(a.x), "+f"(a.y) : "f"(vx), "f"(vy), "f"(sx), "f"(sy));
}

// ---------------------------------------------------------------- tiles
struct Tile {
    int e, r0, n, m0;   // expert, first list position, rows, first weight row
    __device__ __forceinline__ int mma_n() const { return (n + 31) & ~31; }
};

// Tile i of the call, by all lanes of a warp. tab: tile prefix [E + 1], first position [E], rows [E].
__device__ __forceinline__ Tile tile_of(const int* tab, int E, int m_tiles, int i) {
    const int tt = i / m_tiles;
    int lo = 0, hi = E;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (tab[mid] <= tt) lo = mid; else hi = mid;
    }
    const int cnt = tab[E + 1 + E + lo], parts = tab[lo + 1] - tab[lo], l = tt - tab[lo];
    // nearly equal parts in multiples of 32: parts = ceil(cnt / NT), so none is empty
    const int per = ((cnt + parts - 1) / parts + 31) & ~31;
    Tile t;
    t.e = uniform(lo);
    t.r0 = uniform(tab[E + 1 + lo] + l * per);
    t.n = uniform(min(per, cnt - l * per));
    t.m0 = (i - tt * m_tiles) * (2 * kM);
    return t;
}

template <bool FP8, int NT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
rows_tc_kernel(const RowsProduct P, const __grid_constant__ TcRowMaps maps, int m_tiles, WsHeader* hdr,
               unsigned long long wait_limit) {
    using C = Cfg<FP8, NT>;
    extern __shared__ uint8_t rows_smem_raw[];
    // the swizzle pattern follows shared-memory address bits: align the base to 1024 (both CTAs of a
    // pair have the same layout)
    uint8_t* sm = rows_smem_raw + ((1024u - (su32(rows_smem_raw) & 1023u)) & 1023u);
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    const uint32_t rank = cluster_rank();

    float* scale_ring = reinterpret_cast<float*>(sm + C::kOffScales);
    uint64_t* full = reinterpret_cast<uint64_t*>(sm + C::kOffBars);   // this CTA's TMA copies landed
    uint64_t* gath = full + C::kStages;                                // this CTA's gathered rows landed
    uint64_t* peer = gath + C::kStages;                                // first CTA: the second's operands landed
    uint64_t* empty = peer + C::kStages;                               // MMAs done with the step
    uint64_t* acc_full = empty + C::kStages;                           // tensor-memory buffer summed
    uint64_t* acc_empty = acc_full + C::kBufs;                         // first CTA: ... and read in both
    uint64_t* sc_full = acc_empty + C::kBufs;                          // step's scales written
    uint64_t* sc_empty = sc_full + kScaleSlots;                        // ... and read
    uint64_t* done = sc_empty + kScaleSlots;                           // every MMA of the pair
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* tab = reinterpret_cast<int*>(sm + C::kOffTab);

    if (warp == kMmaWarp) {
        if (lane == 0) {
            for (int i = 0; i < C::kStages; ++i) {
                mbar_init(&full[i], 1);
                mbar_init(&gath[i], kGatherThreads);
                mbar_init(&peer[i], 1);
                mbar_init(&empty[i], 1);
            }
            for (int i = 0; i < C::kBufs; ++i) {
                mbar_init(&acc_full[i], 1);
                mbar_init(&acc_empty[i], 2 * kEpiWarps);
            }
            for (int i = 0; i < kScaleSlots; ++i) {
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
                    lo = min(max(__ldg(P.offsets + e), 0), P.R);
                    n = max(min(max(__ldg(P.offsets + e + 1), 0), P.R) - lo, 0);
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
    // overlapping groups of a malformed list could add up to more tiles than the host allows
    const int total = uniform((int)min((long long)tab[P.E] * m_tiles, (long long)kMaxTiles));
    const int kStepK = FP8 ? 128 : 64;
    const int nk = (P.K + kStepK - 1) / kStepK;
    const int first_tile = blockIdx.x >> 1, tile_step = gridDim.x >> 1;
    const Waiter wait{abort_flag, map_rank(su32(const_cast<int*>(abort_flag)), rank ^ 1u), hdr, wait_limit};

    if (warp >= kEpiWarps) {
        if (FP8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kOtherRegs));
        if (warp == kTmaWarp) {
            int step = 0;
            bool ok = true;
#pragma unroll 1
            for (int i = first_tile; i < total && ok; i += tile_step) {
                const Tile t = tile_of(tab, P.E, m_tiles, i);
                const int half = t.mma_n() / 2;
                const int wy = t.e * P.N + t.m0 + (int)rank * kM;
                const int xy = t.r0 + (int)rank * half;
                const int big = half / kBigBox, small = (half - big * kBigBox) / kSmallBox;
                const uint32_t bytes = kABytes + (P.gather ? 0 : half * kStepBytes);
#pragma unroll 1
                for (int s = 0; s < nk; ++s, ++step) {
                    const int st = step % C::kStages, u = step / C::kStages;
                    if (u > 0) ok = wait(&empty[st], (u - 1) & 1);
                    if (!ok) break;
                    const uint32_t a = sm_base + st * C::kStage, b = a + kABytes;
                    if (elect_one()) {
                        mbar_arrive_expect_tx(&full[st], bytes);
                        tma_load_2d(a, &maps.w, s * kStepK, wy, &full[st]);
                        if (!P.gather) {
                            for (int j = 0; j < big; ++j)
                                tma_load_2d(b + j * (kBigBox * kStepBytes), &maps.x_big, s * kStepK, xy + j * kBigBox,
                                            &full[st]);
                            for (int j = 0; j < small; ++j)
                                tma_load_2d(b + (big * kBigBox + j * kSmallBox) * kStepBytes, &maps.x_small,
                                            s * kStepK, xy + big * kBigBox + j * kSmallBox, &full[st]);
                        }
                    }
                }
            }
            // every copy has landed before the CTA may exit (the last fill of each stage)
            if (lane == 0)
                for (int s = max(0, step - C::kStages); s < step; ++s)
                    drain_wait(&full[s % C::kStages], (s / C::kStages) & 1);
        } else if (warp == kMmaWarp) {
            int step = 0, buf_use = 0;
            bool ok = true;
#pragma unroll 1
            for (int i = first_tile; i < total && ok; i += tile_step) {
                const int N = tile_of(tab, P.E, m_tiles, i).mma_n();
                const uint32_t idesc = FP8 ? e4m3_idesc(2 * kM, N) : f16_idesc(2 * kM, N);
#pragma unroll 1
                for (int s = 0; s < nk; ++s, ++step) {
                    const int st = step % C::kStages;
                    const uint32_t parity = (step / C::kStages) & 1;
                    ok = wait(&full[st], parity) && (!P.gather || wait(&gath[st], parity));
                    if (!ok) break;
                    // gathered rows were written by cp.async (generic proxy): order them before the
                    // tensor cores' reads
                    if (P.gather) fence_proxy_async_smem();
                    if (rank != 0) {
                        if (elect_one()) arrive_cluster(map_rank(su32(&peer[st]), 0));
                        continue;
                    }
                    const int buf = buf_use % C::kBufs, v = buf_use / C::kBufs;
                    const bool first = FP8 || s == 0;
                    ok = wait(&peer[st], parity) && (!first || v == 0 || wait(&acc_empty[buf], (v - 1) & 1));
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t a = sw128_desc(sm_base + st * C::kStage);
                    const uint64_t b = sw128_desc(sm_base + st * C::kStage + kABytes);
                    const uint32_t d = tmem + buf * NT;
                    const bool sum_done = FP8 || s == nk - 1;
                    if (elect_one()) {
#pragma unroll
                        for (int j = 0; j < kStepBytes / 32; ++j)      // 32 bytes of K an MMA: 2 address units
                            mma_pair<FP8>(d, a + 2 * j, b + 2 * j, idesc, !first || j != 0);
                        commit_pair(&empty[st]);
                        if (sum_done) commit_pair(&acc_full[buf]);
                    }
                    buf_use += sum_done;
                }
            }
            if (rank == 0) {
                // no MMA still reads or writes either CTA's memory when it is freed
                if (elect_one()) {
                    commit_pair(done);
                    drain_wait(done, 0);
                }
            }
        } else if (warp >= kGatherWarp0) {
            if (P.gather) {
                // thread: 16-byte unit `c` of every 16th row of this CTA's half
                const int th = tid - kGatherWarp0 * 32, c = th & 7, row0 = th >> 3;
                constexpr int kPer = NT / 2 / 16;
                const size_t row_bytes = (size_t)P.K * (FP8 ? 1 : 2);
                const uint8_t* x = static_cast<const uint8_t*>(P.x) + c * 16;
                int step = 0;
                bool ok = true;
#pragma unroll 1
                for (int i = first_tile; i < total && ok; i += tile_step) {
                    const Tile t = tile_of(tab, P.E, m_tiles, i);
                    const int half = t.mma_n() / 2;
                    int src[kPer];
#pragma unroll
                    for (int j = 0; j < kPer; ++j) {
                        const int r = (int)rank * half + row0 + 16 * j;
                        src[j] = row0 + 16 * j < half && r < t.n ? x_row(P, t.r0 + r) : -1;
                    }
#pragma unroll 1
                    for (int s = 0; s < nk; ++s, ++step) {
                        const int st = step % C::kStages, u = step / C::kStages;
                        if (u > 0) ok = wait(&empty[st], (u - 1) & 1);
                        if (!ok) break;
                        const uint32_t b = sm_base + st * C::kStage + kABytes;
                        const size_t off = (size_t)s * kStepBytes;
                        const bool in_k = off + c * 16 < row_bytes;
#pragma unroll
                        for (int j = 0; j < kPer; ++j) {
                            const int row = row0 + 16 * j;
                            if (row < half) {
                                const bool in = in_k && src[j] >= 0;
                                cp_async16_zfill(b + row * kStepBytes + ((c ^ (row & 7)) << 4),
                                                 in ? x + src[j] * row_bytes + off : static_cast<const uint8_t*>(P.x),
                                                 in ? 16u : 0u);
                            }
                        }
                        cp_async_arrive_noinc(&gath[st]);
                    }
                }
                asm volatile("cp.async.wait_all;" ::: "memory");
            }
        } else if (warp >= kScaleWarp0) {
            if constexpr (FP8) {
                const int th = tid - kScaleWarp0 * 32;
                const int KB = nk, NB = (P.N + 127) >> 7;
                constexpr int kPer = NT / kScaleThreads;
                int step = 0;
                bool ok = true;
#pragma unroll 1
                for (int i = first_tile; i < total && ok; i += tile_step) {
                    const Tile t = tile_of(tab, P.E, m_tiles, i);
                    const int nb = (t.m0 >> 7) + (int)rank;
                    const bool any = nb < NB;           // else the half tile lies past the matrix
                    const float* xs[kPer];
#pragma unroll
                    for (int j = 0; j < kPer; ++j) {
                        const int c = th + kScaleThreads * j;
                        const int row = any && c < t.n ? x_row(P, t.r0 + c) : -1;
                        xs[j] = row < 0 ? nullptr : P.xs + (size_t)row * KB;
                    }
                    const float* wsc = any ? P.ws + ((size_t)t.e * NB + nb) * KB : P.ws;
                    float next[kPer], wnext = __ldg(wsc);
#pragma unroll
                    for (int j = 0; j < kPer; ++j) next[j] = xs[j] != nullptr ? __ldg(xs[j]) : 0.f;
#pragma unroll 1
                    for (int s = 0; s < nk; ++s, ++step) {
                        const int slot = step % kScaleSlots, u = step / kScaleSlots;
                        float now[kPer];
#pragma unroll
                        for (int j = 0; j < kPer; ++j) now[j] = xs[j] != nullptr ? next[j] * wnext : 0.f;
                        if (s + 1 < nk) {
                            wnext = __ldg(wsc + s + 1);
#pragma unroll
                            for (int j = 0; j < kPer; ++j)
                                if (xs[j] != nullptr) next[j] = __ldg(xs[j] + s + 1);
                        }
                        if (u > 0 && !wait(&sc_empty[slot], (u - 1) & 1)) {
                            ok = false;
                            break;
                        }
#pragma unroll
                        for (int j = 0; j < kPer; ++j) scale_ring[slot * NT + th + kScaleThreads * j] = now[j];
                        mbar_arrive(&sc_full[slot]);
                    }
                }
            }
        }
    } else {
        if (FP8) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(kEpiRegs));
        const int q = warp & 3, c0 = (warp >> 2) * C::kCols;
        const uint32_t lane_base = tmem + ((uint32_t)(32 * q) << 16) + c0;
        int use = 0;          // tensor-memory buffers (8-bit: steps) read so far
        bool ok = true;
#pragma unroll 1
        for (int i = first_tile; i < total; i += tile_step) {
            const Tile t = tile_of(tab, P.E, m_tiles, i);
            const int n = t.m0 + (int)rank * kM + 32 * q + lane;      // output column of y
            // write 32 columns of the tile
            auto store32 = [&](int c, const float* v) {
                const int row = c + lane < t.n ? y_row(P, t.r0 + c + lane) : -1;
                const bool bad = *abort_flag != 0;
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    const int rj = __shfl_sync(0xffffffffu, row, j);
                    if (rj < 0 || n >= P.N) continue;
                    const float out = bad ? __uint_as_float(0x7FC00000u) : v[j];
                    const size_t at = (size_t)rj * P.N + n;
                    if (P.y_f32) static_cast<float*>(P.y)[at] = out;
                    else static_cast<uint16_t*>(P.y)[at] = f32_to_bf16(out);
                }
            };
            if constexpr (FP8) {
                float2 acc[C::kCols / 2];
#pragma unroll
                for (int j = 0; j < C::kCols / 2; ++j) acc[j] = make_float2(0.f, 0.f);
#pragma unroll 1
                for (int s = 0; s < nk && ok; ++s, ++use) {
                    const int buf = use % C::kBufs, slot = use % kScaleSlots;
                    ok = wait(&sc_full[slot], (use / kScaleSlots) & 1) && wait(&acc_full[buf], (use / C::kBufs) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    const float* sc = scale_ring + slot * NT + c0;
                    float v[2][32];
                    if (c0 < t.n) tmem_ld32(lane_base + buf * NT, v[0]);
#pragma unroll
                    for (int c = 0; c < C::kCols; c += 32) {
                        if (c0 + c >= t.n) break;
                        float (&now)[32] = v[(c / 32) & 1];
                        tmem_wait32(now);
                        if (c + 32 < C::kCols && c0 + c + 32 < t.n)
                            tmem_ld32(lane_base + buf * NT + c + 32, v[(c / 32 + 1) & 1]);
#pragma unroll
                        for (int j = 0; j < 32; j += 4) {
                            const float4 f = *reinterpret_cast<const float4*>(sc + c + j);
                            fma2(acc[(c + j) / 2], now[j], now[j + 1], f.x, f.y);
                            fma2(acc[(c + j) / 2 + 1], now[j + 2], now[j + 3], f.z, f.w);
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        arrive_cluster(map_rank(su32(&acc_empty[buf]), 0));
                        mbar_arrive(&sc_empty[slot]);
                    }
                }
#pragma unroll
                for (int c = 0; c < C::kCols; c += 32) {
                    if (c0 + c >= t.n) break;
                    float v[32];
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[2 * j] = acc[c / 2 + j].x, v[2 * j + 1] = acc[c / 2 + j].y;
                    store32(c0 + c, v);
                }
            } else {
                const int buf = use % C::kBufs;
                if (ok) ok = wait(&acc_full[buf], (use / C::kBufs) & 1);
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < C::kCols; c += 32) {
                    if (c0 + c >= t.n) break;
                    float v[32] = {};
                    if (ok) {
                        tmem_ld32(lane_base + buf * NT + c, v);
                        tmem_wait32(v);
                    }
                    store32(c0 + c, v);
                }
                tc_fence_before();
                __syncwarp();
                if (ok && lane == 0) arrive_cluster(map_rank(su32(&acc_empty[buf]), 0));
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

template <bool FP8, int NT>
cudaError_t launch_tc(const RowsProduct& P, WsHeader* hdr, const DeviceInfo& dev, uint64_t wait_limit,
                      cudaStream_t s) {
    using C = Cfg<FP8, NT>;
    static std::atomic<uint64_t> ready{0};      // one bit per device
    if (!(ready.load(std::memory_order_acquire) >> dev.device & 1)) {
        cudaError_t e = cudaFuncSetAttribute(rows_tc_kernel<FP8, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             C::kSmem);
        if (e != cudaSuccess) return e;
        // the register split waits forever for registers that the launch did not bring
        cudaFuncAttributes a;
        if ((e = cudaFuncGetAttributes(&a, rows_tc_kernel<FP8, NT>)) != cudaSuccess) return e;
        if (FP8 && a.numRegs != kLaunchRegs) return cudaErrorInvalidConfiguration;
        ready.fetch_or(1ull << dev.device, std::memory_order_release);
    }
    PFN_cuTensorMapEncodeTiled_v12000 fn = tensor_map_encoder();
    TcRowMaps maps;
    if (fn == nullptr || !encode_rows(fn, &maps.w, P.w, FP8, P.K, (uint64_t)P.E * P.N, kM) ||
        !encode_rows(fn, &maps.x_big, P.x, FP8, P.K, P.x_rows, kBigBox) ||
        !encode_rows(fn, &maps.x_small, P.x, FP8, P.K, P.x_rows, kSmallBox))
        return cudaErrorInvalidValue;
    const int m_tiles = (P.N + 2 * kM - 1) / (2 * kM);
    // tiles at most: every expert's last one is not full
    const long long tiles = (P.R / NT + std::min(P.R, P.E)) * (long long)m_tiles;
    if (tiles > kMaxTiles) return cudaErrorInvalidConfiguration;
    const unsigned pairs = (unsigned)std::min<long long>(tiles, dev.num_sms / 2);
    rows_tc_kernel<FP8, NT><<<2 * pairs, kThreads, C::kSmem, s>>>(P, maps, m_tiles, hdr, wait_limit);
    return cudaGetLastError();
}

template <bool FP8>
cudaError_t launch_any(const RowsProduct& P, WsHeader* hdr, const DeviceInfo& dev, uint64_t wait_limit,
                       cudaStream_t s) {
    const int rows = (P.R + P.E - 1) / P.E;      // per expert, were they even
    if (rows > 64) return launch_tc<FP8, 256>(P, hdr, dev, wait_limit, s);
    return launch_tc<FP8, 64>(P, hdr, dev, wait_limit, s);
}

}  // namespace

cudaError_t launch_rows_tc(const RowsProduct& P, WsHeader* hdr, const DeviceInfo& dev, uint64_t wait_limit,
                           cudaStream_t s) {
    return P.xs != nullptr ? launch_any<true>(P, hdr, dev, wait_limit, s)
                           : launch_any<false>(P, hdr, dev, wait_limit, s);
}

}  // namespace nvfp4
