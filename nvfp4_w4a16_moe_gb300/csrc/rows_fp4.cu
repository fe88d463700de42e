// Products of NVFP4 rows with one NVFP4 matrix or with each expert's on the block-scaled tensor cores:
//   y[o(r), n] = xr[i(r)] wt[e, n] sum_b xs[i(r), b] ws[n, b] sum_{k in b} x[i(r), k] w[n, k],  blocks b of 16
//
// tcgen05.mma kind::mxf4nvf4 takes both operands in 4 bits from shared memory and their E4M3 block scales from tensor
// memory, and keeps the running sum in fp32: the block scales cost no arithmetic outside the tensor cores, and the
// epilogue multiplies by the two fp32 scales once.
//
// Tiles, pairs of CTAs, warp roles, the walk over the experts and the exchange between pairs that share a tile's K are
// those of rows_tc.cu (pair_tc.cuh). What differs:
//   A step is 128 bytes of a row as there, 256 elements: four MMAs of 64 columns, each with 4 scales a row.
//   Scale warps bring the step's 16 block scales of every row. Both operands store them row by row, [rows, K/16],
//     while the tensor cores want, for every 64 columns, 32 lines of 16 bytes: line l holds the four scales of rows l,
//     32 + l, 64 + l and 96 + l. A lane loads the 16 bytes of those four rows, which are then lines l of the step's
//     four MMAs when read across: a transposition of registers, four 16-byte loads and stores for 2 KB of scales, no
//     second copy of the weights' scales in another order. Behind the end of K and for rows that the tile does not have
//     the scales are 0, so neither a neighbour's NaN scale nor its codes count.
//   The MMA warp copies a step's scales from the ring to tensor memory (tcgen05.cp, to all four lane quarters), right
//     before the step's MMAs: the tensor pipe runs copies and MMAs of one thread in the order of issue.
//   Tensor memory: 512 columns hold two sums of 256 columns, but not the scales as well (48). So the two buffers of a
//     256-column tile share 48 columns, which the epilogue reads first and hands back on their own.
#include <atomic>
#include <cstring>

#include "common.cuh"
#include "kernels.cuh"
#include "pair_tc.cuh"

namespace nvfp4 {

namespace {

constexpr int kABytes = kM * kStepBytes;
constexpr int kStepK = 2 * kStepBytes;   // elements of a step
constexpr int kMmas = kStepK / 64;       // MMAs of a step
constexpr int kBlkBytes = 2048;          // scales of 128 rows and a step
constexpr int kMaxStages = 9;
constexpr int kMinSteps = 2;             // steps of each pair that shares a tile's K, at least

// Warps: 16 of epilogue, TMA, MMA, four of gather, two for every 128 rows of scales (each takes every other step).
constexpr int kEpiWarps = 16, kTmaWarp = 16, kMmaWarp = 17, kGatherWarp0 = 18, kGatherWarps = 4, kScaleWarp0 = 22;

template <int NT>
struct Cfg {
    static constexpr int kXBlocks = (NT + 127) / 128, kBlocks = 1 + kXBlocks;     // of 128 rows' scales
    static constexpr int kThreads = 32 * (kScaleWarp0 + 2 * kBlocks);
    static constexpr int kBoxRows = kNRound / 2;                 // heights of a box of x: this times
    static constexpr int kBoxes = NT / kNRound;                  // ... 1 .. kBoxes
    static constexpr int kOffSf = kABytes + NT / 2 * kStepBytes; // scales of W, then of x
    static constexpr int kStage = kOffSf + kBlocks * kBlkBytes;
    static constexpr int kStages = std::min(kMaxStages, (196 * 1024) / kStage);
    // tensor memory: buffers of NT columns, then the scales of a step (two sets of them where there is room)
    static constexpr int kSfCols = 4 * kMmas * kBlocks;
    static constexpr bool kOverlap = NT == 256;
    static constexpr int kBufs = kOverlap ? 2 : 256 / NT;
    static constexpr int kBufStep = kOverlap ? 512 - kSfCols - NT : NT;
    static constexpr int kShared = kOverlap ? NT - kBufStep : 0; // columns that both buffers have
    static constexpr int kSf = kOverlap ? 512 - kSfCols : 256, kSfSets = kOverlap ? 1 : 2;
    static constexpr int kCols = NT / 4;                         // columns of an epilogue warp, at most
    static constexpr int kOffStg = kStages * kStage;
    static constexpr int kOffBars = kOffStg + kEpiWarps * kStgRows * kStgPitch;
    static constexpr int kNumBars = 2 * kStages + 3 * kBufs + 1;
    static constexpr int kOffTab = kOffBars + kNumBars * 8 + 16; // tile prefix [E + 1], first position [E], rows [E]
    static constexpr int kSmem = 1024 + kOffTab + (3 * NVFP4_MAX_EXPERTS + 1) * 4;
    static_assert(NT % kNRound == 0 && NT <= 256 && kStage % 1024 == 0 && kCols % 16 == 0, "swizzle atoms, fragments");
    static_assert(kSmem <= 227 * 1024, "shared memory");
    static_assert(4 * NT / 16 * 2048 <= kOffStg, "exchanged sums fit in the ring");
    static_assert(kShared % 16 == 0 && kSf + kSfSets * kSfCols <= 512, "tensor memory");
};

struct TcRowMaps {
    CUtensorMap w, x[4];   // x: boxes of one to kBoxes times Cfg::kBoxRows rows; x[0] single rows to gather
};

// D (256 x N over both CTAs) = A B^T of 64 columns, scaled by 4 E4M3 scales a row, plus D where accumulate.
__device__ __forceinline__ void mma_nvfp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n}"
        :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate) : "memory");
}
// 32 lines of 16 bytes to four columns of tensor memory, the same in all lane quarters, in both CTAs.
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" :: "r"(tmem), "l"(desc) : "memory");
}
// Descriptor of 32 lines of 16 bytes, one after another: groups of eight lines 128 bytes apart, not swizzled.
__device__ __forceinline__ uint64_t lines_desc(uint32_t saddr) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
}
// Instruction descriptor of kind::mxf4nvf4: E2M1 A and B (format 1, both K-major), E4M3 scales, fp32 D, M = 256, K = 64.
__device__ __forceinline__ uint32_t nvfp4_idesc(int N) {
    return (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(2 * kM >> 7) << 27);
}

// Bytes 16 s .. 16 s + 15 of a row of KB block scales, 0 behind its end. KB is even; its rows start at multiples of
// `unit` (2, 4 or 16) bytes.
__device__ __forceinline__ uint4 row_scales16(const uint8_t* row, int s, int KB, int unit) {
    const uint8_t* p = row + 16 * s;
    const int left = KB - 16 * s;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (unit == 16) return *reinterpret_cast<const uint4*>(p);
    if (unit == 4) {
        const uint32_t* q = reinterpret_cast<const uint32_t*>(p);
        if (left > 0) v.x = q[0];
        if (left > 4) v.y = q[1];
        if (left > 8) v.z = q[2];
        if (left > 12) v.w = q[3];
        return v;
    }
    const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
    uint32_t h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = left > 2 * i ? q[i] : 0u;
    return make_uint4(h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16));
}

// SPLITS: pairs of a cluster, which share a tile's K.
template <int NT, int SPLITS>
__global__ void __cluster_dims__(2 * SPLITS, 1, 1) __launch_bounds__(Cfg<NT>::kThreads, 1)
rows_fp4_kernel(const Fp4Product Q, const __grid_constant__ TcRowMaps maps, int m_tiles, int max_tiles, WsHeader* hdr,
                unsigned long long wait_limit) {
    using C = Cfg<NT>;
    const RowsProduct& P = Q.r;
    extern __shared__ uint8_t fp4_smem_raw[];
    // the swizzle pattern follows shared-memory address bits: align the base to 1024 (both CTAs of a
    // pair have the same layout)
    uint8_t* sm = fp4_smem_raw + ((1024u - (su32(fp4_smem_raw) & 1023u)) & 1023u);
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    // CTA of its pair, pair of its cluster
    const int crank = (int)cluster_rank(), rank = crank & 1, pair = SPLITS == 1 ? 0 : crank >> 1, first_rank = 2 * pair;
    const uint16_t pair_mask = (uint16_t)(3u << first_rank);

    uint64_t* full = reinterpret_cast<uint64_t*>(sm + C::kOffBars);   // step landed (first CTA: in both)
    uint64_t* empty = full + C::kStages;                               // MMAs done with the step
    uint64_t* acc_full = empty + C::kStages;                           // tensor-memory buffer summed
    uint64_t* acc_empty = acc_full + C::kBufs;                         // first CTA: ... and read in both
    uint64_t* shr_empty = acc_empty + C::kBufs;                        // first CTA: ... the columns it shares
    uint64_t* done = shr_empty + C::kBufs;                             // every MMA of the pair
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* tab = reinterpret_cast<int*>(sm + C::kOffTab);

    if (warp == kMmaWarp) {
        if (lane == 0) {
            for (int i = 0; i < C::kStages; ++i) {
                // the TMA warp, a warp for every 128 rows of scales, each gather warp, in the first CTA the second's word
                mbar_init(&full[i], 1 + C::kBlocks + (P.gather ? kGatherWarps : 0) + (rank == 0 ? 1 : 0));
                mbar_init(&empty[i], 1);
            }
            for (int i = 0; i < C::kBufs; ++i) {
                mbar_init(&acc_full[i], 1);
                mbar_init(&acc_empty[i], 2 * kEpiWarps);
                mbar_init(&shr_empty[i], 2 * kEpiWarps);
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
    if (warp == 0) tile_table<NT>(P, tab);
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();       // barriers are ready in both CTAs
    tc_fence_after();
    const uint32_t tmem = (uint32_t)uniform((int)*tmem_slot), sm_base = su32(sm);
    // tiles that overlapping groups of a malformed list add are left out (rows_tc.cu)
    constexpr int kCluster = 2 * SPLITS;
    const int total = uniform((int)min((long long)tab[P.E] * m_tiles, (long long)max_tiles));
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
                        tma_load_2d(a, &maps.w, s * kStepBytes, wy, &full[st]);
                        if (!P.gather) tma_load_2d(b, mx, s * kStepBytes, t.r0 + rank * share, &full[st]);
                    }
                }
            }
            if (lane == 0) drain(step);
        } else if (warp == kMmaWarp) {
            int st = 0, buf = 0, use = 0;
            uint32_t st_par = 0, buf_par = 1;          // an unused buffer's "empty" phase counts as over
            bool ok = true;
            const uint64_t stage0 = sw128_desc(sm_base), scales0 = lines_desc(sm_base + C::kOffSf);
#pragma unroll 1
            for (Walk at = tiles; at.more() && ok; at.next(), ++use) {
                const int N = at.tile().mma_n();
                const uint32_t idesc = nvfp4_idesc(N);
#pragma unroll 1
                for (int s = s_begin; s < s_end; ++s) {
                    ok = wait(&full[st], st_par);
                    if (!ok) break;
                    if (rank != 0) {
                        if (elect_one()) arrive_cluster(map_rank(su32(&full[st]), first_rank));
                    } else {
                        if (s == s_begin) {
                            ok = wait(&acc_empty[buf], buf_par);
                            // the tile before this one still has its buffer, but for the columns that this one shares
                            if (C::kOverlap && ok && use > 0) ok = wait(&shr_empty[buf ^ 1], ((use - 1) >> 1) & 1);
                        }
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t a = stage0 + st * (C::kStage / 16), b = a + kABytes / 16;
                        const uint64_t sf = scales0 + st * (C::kStage / 16);
                        const uint32_t tsf = tmem + C::kSf + (C::kSfSets > 1 ? (s & 1) * C::kSfCols : 0);
                        if (elect_one()) {
                            // columns: 4 for each MMA's scales of W, then 4 kXBlocks for each MMA's of x
#pragma unroll
                            for (int j = 0; j < kMmas; ++j) {
                                copy_scales(tsf + 4 * j, sf + j * (512 / 16));
#pragma unroll
                                for (int i = 0; i < C::kXBlocks; ++i)
                                    copy_scales(tsf + 4 * kMmas + 4 * (C::kXBlocks * j + i),
                                                sf + ((1 + i) * kBlkBytes + j * 512) / 16);
                            }
#pragma unroll
                            for (int j = 0; j < kMmas; ++j)      // 32 bytes of K an MMA: 2 address units
                                mma_nvfp4(tmem + buf * C::kBufStep, a + 2 * j, b + 2 * j, idesc, tsf + 4 * j,
                                          tsf + 4 * kMmas + 4 * C::kXBlocks * j, s != s_begin || j != 0);
                            commit_pair(&empty[st], pair_mask);
                            if (s == s_end - 1) commit_pair(&acc_full[buf], pair_mask);
                        }
                        if (s == s_end - 1 && ++buf == C::kBufs) buf = 0, buf_par ^= 1;
                    }
                    if (++st == C::kStages) st = 0, st_par ^= 1;
                }
            }
            // no MMA still reads or writes either CTA's memory, nor has an arrival on the way to it, when it is freed
            if (elect_one()) {
                if (rank == 0) commit_pair(done, pair_mask);
                drain_wait(done, 0);
            }
        } else if (warp < kScaleWarp0) {
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
                                tma_gather4(b + j * (kGatherWarps * 4 * kStepBytes), &maps.x[0], s * kStepBytes, r0, r1,
                                            r2, r3, &full[st]);
                        }
                    }
                }
                if (lane == 0) drain(step);
            }
        } else {
            const int blk = (warp - kScaleWarp0) % C::kBlocks, odd = (warp - kScaleWarp0) / C::kBlocks;
            const int KB = P.K / 16, unit = KB % 16 == 0 ? 16 : KB % 4 == 0 ? 4 : 2;
            int base = 0;                            // steps of the tiles so far
            bool ok = true;
#pragma unroll 1
            for (Walk at = tiles; at.more() && ok; at.next(), base += s_end - s_begin) {
                const Tile t = at.tile();
                const uint8_t* row[4];               // null: no such row
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    row[i] = nullptr;
                    if (blk == 0) {
                        const int n = t.m0 + rank * kM + 32 * i + lane;
                        if (n < P.N) row[i] = Q.ws + ((size_t)t.e * P.N + n) * KB;
                    } else {
                        const int col = (blk - 1) * 128 + 32 * i + lane;
                        const int src = col < t.n ? x_row(P, t.r0 + col) : -1;
                        if (src >= 0) row[i] = Q.xs + (size_t)src * KB;
                    }
                }
                uint4 v[4];
                auto load = [&](int s) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        v[i] = row[i] != nullptr ? row_scales16(row[i], s, KB, unit) : make_uint4(0, 0, 0, 0);
                };
                // every other step of the call is this warp's
                const int s_first = s_begin + ((base ^ odd) & 1);
                if (s_first < s_end) load(s_first);
#pragma unroll 1
                for (int s = s_first; s < s_end; s += 2) {
                    const int step = base + s - s_begin, st = step % C::kStages, u = step / C::kStages;
                    if (u > 0) ok = wait(&empty[st], (u - 1) & 1);
                    if (!ok) break;
                    uint4* to = reinterpret_cast<uint4*>(sm + st * C::kStage + C::kOffSf + blk * kBlkBytes) + lane;
                    to[0] = make_uint4(v[0].x, v[1].x, v[2].x, v[3].x);
                    to[32] = make_uint4(v[0].y, v[1].y, v[2].y, v[3].y);
                    to[64] = make_uint4(v[0].z, v[1].z, v[2].z, v[3].z);
                    to[96] = make_uint4(v[0].w, v[1].w, v[2].w, v[3].w);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (elect_one()) mbar_arrive(&full[st]);
                    if (s + 2 < s_end) load(s + 2);
                }
            }
        }
        if (SPLITS > 1 && tiles.more()) exchange.join();
    } else {
        const int q = warp & 3, part = warp >> 2;          // lanes 32 q .., a quarter of the columns
        uint8_t* stg = sm + C::kOffStg + warp * (kStgRows * kStgPitch);
        const int p = lane & 3, g = lane >> 2;
        const uint32_t first_acc_empty = map_rank(su32(acc_empty), first_rank);
        const uint32_t first_shr_empty = map_rank(su32(shr_empty), first_rank);
        const int part_rows = P.N / Q.parts;
        int use = 0;               // buffers read so far
        bool ok = true;
#pragma unroll 1
        for (Walk at = tiles; at.more(); at.next()) {
            const Tile t = at.tile();
            const int width = t.mma_n() / 4, c0 = part * width;            // this warp's columns of the tile
            const int n0 = t.m0 + rank * kM + 32 * q;                      // first output
            // lane l: row of y (or -1) and row scale of columns c0 + l and c0 + 32 + l, asked for under the MMAs
            int dst[2];
            float scale[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int c = 32 * i + lane, col = c0 + c;
                dst[i] = -1, scale[i] = 0.f;
                if (c < width && col < t.n) {
                    const int src = x_row(P, t.r0 + col);
                    dst[i] = y_row(P, t.r0 + col);
                    if (src >= 0) scale[i] = Q.xr[src];
                }
            }
            float wt[4];                                                   // tensor scales of outputs n0 + 8 i + g
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int n = n0 + 8 * i + g;
                wt[i] = n < P.N ? Q.wt[(size_t)t.e * Q.parts + n / part_rows] : 0.f;
            }
            const int buf = use % C::kBufs;
            const uint32_t lanes = tmem + ((uint32_t)(32 * q) << 16) + buf * C::kBufStep + c0;
            if (ok) ok = wait(&acc_full[buf], (use / C::kBufs) & 1);
            tc_fence_after();
            const auto sums = [&](int c, float (&v)[16]) {
                if (ok) {
                    tmem_ld_frag(lanes + c, v);
                    tmem_wait16(v);
                }
            };
            const auto finish = [&](int c, float (&v)[16]) {
                const int d = c & 32 ? dst[1] : dst[0];
                const float sc = c & 32 ? scale[1] : scale[0];
                float s4[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    s4[i] = __shfl_sync(0xffffffffu, sc, (c & 16) + 8 * (i >> 1) + 2 * p + (i & 1));
#pragma unroll
                for (int i = 0; i < 16; ++i)     // lane group 2 L + u, column 2 j + b of the fragment
                    v[i] *= s4[2 * ((i >> 2) & 1) + (i & 1)] * wt[2 * (i >> 3) + ((i >> 1) & 1)];
                if (*abort_flag)
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(0x7FC00000u);
                store_frag(P, v, __shfl_sync(0xffffffffu, d, (c & 16) + (lane & 15)), n0, stg);
            };
            if constexpr (SPLITS > 1) {
                exchange.send(sums, t, width, c0, part, q);
#pragma unroll
                for (int c = 0; c < C::kCols; c += 16) {
                    if (c >= width || c0 + c >= t.n) break;
                    float v[16];
                    sums(c, v);
                    if (exchange.finish(v, c, width, part, q)) finish(c, v);
                }
            } else {
                // The columns that the next tile's buffer shares come first: the last ones of buffer 0, the first of
                // buffer 1.
                const bool down = C::kOverlap && buf == 0;
                const auto shared_left = [&](int c) {              // chunk c is in, or before, the shared columns
                    return down ? c0 + c + 16 > NT - C::kShared : c0 + c < C::kShared;
                };
                bool told = !C::kOverlap;
                const auto tell = [&](uint32_t bar) {
                    tc_fence_before();
                    __syncwarp();
                    if (ok && elect_one()) arrive_cluster(bar + 8 * buf);
                };
#pragma unroll 1
                for (int i = 0; i < width; i += 16) {
                    const int c = down ? width - 16 - i : i;
                    if (!told && !shared_left(c)) tell(first_shr_empty), told = true;
                    if (c0 + c >= t.n) continue;                    // padding is neither read nor written
                    float v[16];
                    sums(c, v);
                    finish(c, v);
                }
                if (!told) tell(first_shr_empty);
                tell(first_acc_empty);
            }
            ++use;
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

// Sets the kernel up on the current device, once, and says how many of its clusters run there at a time
// (clusters of eight CTAs do not fill every GPC).
template <int NT, int SPLITS>
cudaError_t resident_clusters(const DeviceInfo& dev, int* clusters) {
    using C = Cfg<NT>;
    static std::atomic<int> known[64];           // by device: one more than the clusters
    int n = known[dev.device].load(std::memory_order_acquire) - 1;
    if (n < 0) {
        const auto kernel = rows_fp4_kernel<NT, SPLITS>;
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
        if (e != cudaSuccess) return e;
        cudaLaunchAttribute attr{};
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = 2 * SPLITS;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(2 * SPLITS * dev.num_sms);
        cfg.blockDim = dim3(C::kThreads);
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

// Tiles of NT columns. The estimate (us) takes the rows to be even over the experts.
template <int NT>
cudaError_t plan_tiles(const RowsProduct& P, const DeviceInfo& dev, Plan* best) {
    const int m_tiles = (P.N + 2 * kM - 1) / (2 * kM), nk = (P.K + kStepK - 1) / kStepK;
    const int groups = std::min(P.R, P.E), rows = (P.R + groups - 1) / groups;
    Plan p;
    p.nt = NT;
    // tiles at most: every expert has rows, and its last tile one
    p.tiles = ((P.R - groups) / NT + groups) * (long long)m_tiles;
    // as many pairs to a tile as the device runs at a time, where each has kMinSteps steps
    int c2 = 0, c4 = 0;
    if (nk >= 2 * kMinSteps && 2 * p.tiles <= dev.num_sms / 2)
        if (cudaError_t e = resident_clusters<NT, 2>(dev, &c2); e != cudaSuccess) return e;
    if (nk >= 4 * kMinSteps && 4 * p.tiles <= dev.num_sms / 2)
        if (cudaError_t e = resident_clusters<NT, 4>(dev, &c4); e != cudaSuccess) return e;
    p.splits = p.tiles <= c4 ? 4 : p.tiles <= c2 ? 2 : 1;
    const int parts = (rows + NT - 1) / NT, n = ((rows + parts - 1) / parts + kNRound - 1) / kNRound * kNRound;
    const long long even = (long long)groups * parts * m_tiles, rounds = (even + dev.num_sms / 2 - 1) / (dev.num_sms / 2);
    const float step = 0.08f + 0.0012f * n;
    p.us = rounds * ((nk + p.splits - 1) / p.splits * step + 1.0f + (p.splits > 1 ? 0.5f + 0.009f * n : 0.0f));
    if (p.us < best->us) *best = p;
    return cudaSuccess;
}

template <int NT, int SPLITS>
cudaError_t launch_clusters(const Fp4Product& P, const TcRowMaps& maps, int tiles, WsHeader* hdr,
                            const DeviceInfo& dev, uint64_t wait_limit, cudaStream_t s) {
    int resident = 0;
    if (cudaError_t e = resident_clusters<NT, SPLITS>(dev, &resident); e != cudaSuccess) return e;
    if (resident < 1) return cudaErrorInvalidConfiguration;
    const int clusters = SPLITS > 1 ? tiles : std::min(tiles, resident), m_tiles = (P.r.N + 2 * kM - 1) / (2 * kM);
    return launch_pdl(rows_fp4_kernel<NT, SPLITS>, 2 * SPLITS * clusters, Cfg<NT>::kThreads, Cfg<NT>::kSmem, s, P, maps,
                      m_tiles, tiles, hdr, (unsigned long long)wait_limit);
}

template <int NT>
cudaError_t launch_tiles(const Fp4Product& P, const Plan& plan, WsHeader* hdr, const DeviceInfo& dev,
                         uint64_t wait_limit, cudaStream_t s) {
    using C = Cfg<NT>;
    PFN_cuTensorMapEncodeTiled_v12000 fn = tensor_map_encoder();
    TcRowMaps maps;
    const uint64_t bytes = P.r.K / 2;
    if (fn == nullptr || !encode_rows(fn, &maps.w, P.r.w, true, bytes, (uint64_t)P.r.E * P.r.N, kM)) return cudaErrorInvalidValue;
    for (int i = 0; i < (P.r.gather ? 1 : C::kBoxes); ++i)
        if (!encode_rows(fn, &maps.x[i], P.r.x, true, bytes, P.r.x_rows, P.r.gather ? 1 : (i + 1) * C::kBoxRows))
            return cudaErrorInvalidValue;
    const int tiles = (int)plan.tiles;
    if (plan.splits == 4) return launch_clusters<NT, 4>(P, maps, tiles, hdr, dev, wait_limit, s);
    if (plan.splits == 2) return launch_clusters<NT, 2>(P, maps, tiles, hdr, dev, wait_limit, s);
    return launch_clusters<NT, 1>(P, maps, tiles, hdr, dev, wait_limit, s);
}

}  // namespace

cudaError_t launch_rows_fp4(const Fp4Product& P, WsHeader* hdr, const DeviceInfo& dev, uint64_t wait_limit,
                            cudaStream_t s) {
    Plan plan{};
    plan.us = 3.0e38f;
    const int groups = std::min(P.r.R, P.r.E), rows = (P.r.R + groups - 1) / groups;
    cudaError_t e;
    if (rows <= 64) {
        if ((e = plan_tiles<64>(P.r, dev, &plan)) != cudaSuccess) return e;
    } else {
        if ((e = plan_tiles<128>(P.r, dev, &plan)) != cudaSuccess) return e;
        if ((e = plan_tiles<256>(P.r, dev, &plan)) != cudaSuccess) return e;
    }
    if (plan.tiles > kMaxTiles) return cudaErrorInvalidConfiguration;
    if (plan.nt == 64) return launch_tiles<64>(P, plan, hdr, dev, wait_limit, s);
    if (plan.nt == 128) return launch_tiles<128>(P, plan, hdr, dev, wait_limit, s);
    return launch_tiles<256>(P, plan, hdr, dev, wait_limit, s);
}

}  // namespace nvfp4
