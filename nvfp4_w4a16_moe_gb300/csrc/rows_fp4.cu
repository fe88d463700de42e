// Products of NVFP4 rows with one NVFP4 matrix or with each expert's on the block-scaled tensor cores:
//   y[o(r), n] = xr[i(r)] wt[e, n] sum_b xs[i(r), b] ws[n, b] sum_{k in b} x[i(r), k] w[n, k],  blocks b of 16
//
// tcgen05.mma kind::mxf4nvf4 takes both operands in 4 bits from shared memory and their E4M3 block scales from tensor
// memory, and keeps the running sum in fp32: the block scales cost no arithmetic outside the tensor cores, and the
// epilogue multiplies by the two fp32 scales once.
//
// Tiles, pairs of CTAs, the walk over the experts and the exchange between pairs that share a tile's K are those of
// rows_tc.cu (pair_tc.cuh). What differs:
//   A step is 128 bytes of a row as there, 256 elements: four MMAs of 64 columns, each with 4 scales a row.
//   Block scales. Both operands store them row by row, [rows, K/16], while the tensor cores want, for every 64 columns, 32
//     lines of 16 bytes: line l holds the four scales of rows l, 32 + l, 64 + l and 96 + l. Copies bring 32 bytes of every
//     row, the scales of two steps, and a warp for every 128 rows puts them into line order in place: a lane holds the
//     words of its four rows, which are lines l of the eight MMAs when read across. No second copy of the weights' scales
//     in another order is needed. Rows whose scales are no multiple of 16 bytes
//     (K is none of 256) are no strides of a tensor map; two, four or eight of them together are (OddCopies): 48 bytes of
//     each, out of which the same warp takes its 32. (That warp loading them from global memory: 4096 x 8192 x 2016 in 76
//     us, rows gathered for 256 experts in 190; now 58 and 99.) Behind the end of K the scales are 0, so neither the codes
//     nor NaN scales that lie there count.
//   The MMA thread copies a step's scales from the ring to tensor memory (tcgen05.cp, to all four lane quarters), right
//     before the step's MMAs: the tensor pipe runs copies and MMAs of one thread in the order of issue.
//   Tensor memory holds two sums and the scales of a step: 512 columns take tiles of up to 224 columns. (Tiles of 256
//     whose buffers shared 48 columns, which the epilogue read first, left 1.1 us of every tile without MMAs.)
//   A warp looks up a tile ahead what the epilogue needs of its rows (scales, places of y), so that no epilogue warp waits
//     for a list entry. The epilogue writes past L1.
//
// What bounds it. With many rows the operands on their way into shared memory, 30 KB a step and SM: a step of 224 columns
// takes 0.24 us between K = 1024 and 2048 and 0.30 from 4096 on (at 1.93 GHz 66 and 54 bytes a clock; its MMAs need 240
// clocks); 4096 x 8192 x 8192 takes 91 us, 6 PFLOP/s. Below that also what a tile's epilogue takes beyond the next tile's
// steps: 4096 x 8192 x 2048 takes 33.4 us (4.1 PFLOP/s) for eight rounds of tiles, each 1.9 of steps, some 1.0 of epilogue and
// 0.6 of stores (28.2 without any stores), and 4.5 around them; 4096 x 8192 x 512 takes 22.7, 18.7 without stores, and a
// fill of y 17. With few rows to many experts the weights from memory (64 tokens to eight of 256 experts of 1024 x 2048
// each: 36 us for the 190 MB of some 160 experts), with few rows of one matrix the start of a launch.
#include <atomic>
#include <cmath>
#include <cstring>

#include "common.cuh"
#include "kernels.cuh"
#include "pair_tc.cuh"

namespace nvfp4 {

namespace {

constexpr int kABytes = kM * kStepBytes;
constexpr int kStepK = 2 * kStepBytes;   // elements of a step
constexpr int kMmas = kStepK / 64;       // MMAs of a step
constexpr int kSectorBytes = 32;         // block scales of a row in two steps
constexpr int kOddBytes = 48;            // ... with the 16-byte pieces that they lie in (rows are no multiple of 16 bytes)
constexpr int kRing = 192 * 1024;        // operands and scales
constexpr int kMaxStages = 9;
constexpr int kWidths = 16;
constexpr int kMinSteps = 2;             // steps of each pair that shares a tile's K, at least

// Warps: 16 of epilogue, TMA, MMA, four of gather (which bring OddCopies where no rows are gathered), one that looks up the
// tiles' ends, one for every 128 rows of scales.
constexpr int kEpiWarps = 16, kTmaWarp = 16, kMmaWarp = 17, kGatherWarp0 = 18, kGatherWarps = 4, kEndsWarp = 22;
constexpr int kScaleWarp0 = 23;

// ODD: a row's scales are no multiple of 16 bytes (K is none of 256).
template <int NT, bool ODD>
struct Cfg {
    static constexpr int kNT = NT;
    static constexpr int kRound = NT > 128 ? 32 : kNRound;       // a tile's columns are a multiple of this
    static constexpr int kXBlocks = (NT + 127) / 128, kBlocks = 1 + kXBlocks;     // of 128 rows' scales
    static constexpr int kThreads = 32 * (kScaleWarp0 + kBlocks);
    static constexpr int kBoxRows = NT > 128 ? 56 : 32;          // rows of x of a copy
    static constexpr int kStage = kABytes + NT / 2 * kStepBytes;
    // ring of block scales of two steps: W's 128 rows, then x's NT
    static constexpr int kXRows = std::min(NT, 128);             // rows of x whose scales come together
    static constexpr int kRowBytes = ODD ? kOddBytes : kSectorBytes, kBlkBytes = kM * kRowBytes;
    static constexpr int kSlotBytes = kBlocks * kBlkBytes, kSlots = NT > 128 && !ODD ? 3 : 4;
    static constexpr int kStages = std::min(kMaxStages, (kRing - kSlots * kSlotBytes) / kStage);
    static constexpr int kOffSlots = kStages * kStage;
    // tensor memory: buffers of NT columns, then the scales of a step (two sets of them where there is room)
    static constexpr int kSfCols = 4 * kMmas * kBlocks;
    static constexpr int kBufs = NT > 128 ? 2 : 256 / NT;
    static constexpr int kSf = kBufs * NT, kSfSets = NT > 128 ? 1 : 2;
    static constexpr int kCols = NT / 4;                         // columns of an epilogue warp, at most
    static constexpr int kOffStg = kOffSlots + kSlots * kSlotBytes;
    // what the epilogue needs of a tile: address of the row of y (0: none) and row scale of its columns, tensor scale of
    // the CTA's outputs, its rows and first output
    static constexpr int kEndsBytes = NT * 12 + kM * 4 + 16, kEnds = 3;
    static constexpr int kOffEnds = kOffStg + kEpiWarps * kStgRows * kStgPitch;
    static constexpr int kOffBars = kOffEnds + kEnds * kEndsBytes;
    static constexpr int kNumBars = 2 * kStages + 2 * kBufs + 3 * kSlots + 2 * kEnds + 1;
    static constexpr int kOffWidths = kOffBars + kNumBars * 8 + 16;  // MMA columns of the latest tiles [kWidths]
    static constexpr int kOffTab = kOffWidths + kWidths * 4;     // tile prefix [E + 1], first position [E], rows [E]
    static constexpr int kSmem = 1024 + kOffTab + (3 * NVFP4_MAX_EXPERTS + 1) * 4;
    static_assert(NT % kRound == 0 && NT <= 256 && kStage % 1024 == 0 && NT / 2 % kBoxRows == 0, "swizzle atoms, copies");
    static_assert(kSmem <= 227 * 1024 && kStages < kWidths, "shared memory");
    static_assert(4 * NT / 16 * 2048 <= kOffStg, "exchanged sums fit in the ring");
    static_assert(kSf + kSfSets * kSfCols <= 512, "tensor memory");
};

struct Fp4Maps {
    CUtensorMap w, x;      // x: boxes of kBoxRows rows, or of one to gather
    CUtensorMap ws, xs;    // block scales of two steps (encode_scales, encode_odd_scales); xs is not read to gather
};

// D (256 x N over both CTAs) = A B^T of 64 columns, scaled by 4 E4M3 scales a row, plus D where accumulate.
__device__ __forceinline__ void mma_nvfp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n}"
        :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate) : "memory");
}
// tma_load_2d with a cache policy: what leaves the L2 first, or as usual.
__device__ __forceinline__ uint64_t l2_policy(bool first) {
    uint64_t f, n;
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(f));
    asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(n));
    return first ? f : n;
}
__device__ __forceinline__ void tma_load_2d_policy(uint32_t dst, const CUtensorMap* map, int x, int y, uint64_t* bar,
                                                   uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint "
        "[%0], [%1, {%2, %3}], [%4], %5;"
        :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(su32(bar)), "l"(policy) : "memory");
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

// A warp that puts the scales of 128 rows (blk 0: of W, then of x) of two steps after two steps into line order, in place,
// from the sectors that copies brought, row after row. ready: barriers of the pair's first CTA, whose copies into tensor
// memory read both CTAs' lines.
template <typename C>
__device__ __forceinline__ void scale_warp(int count, int blk, uint8_t* slots, uint64_t* raw, uint32_t ready,
                                           const Waiter& wait) {
    const int lane = threadIdx.x & 31;
    int slot = 0;
    uint32_t par = 0;
#pragma unroll 1
    for (int j = 0; j < count; ++j) {
        uint8_t* blkp = slots + slot * C::kSlotBytes + blk * C::kBlkBytes;
        uint4* to = reinterpret_cast<uint4*>(blkp) + lane;
        if (!wait(&raw[slot], par)) return;
        uint32_t w[4][8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // the halves of rows 4 .. 7 of every eight have changed places (32-byte swizzle): no bank is read twice
            const uint8_t* p = blkp + (32 * i + lane) * kSectorBytes;
            const int odd = (lane >> 2) & 1;
            const uint4 a = *reinterpret_cast<const uint4*>(p + 16 * odd);
            const uint4 b = *reinterpret_cast<const uint4*>(p + 16 * (odd ^ 1));
            w[i][0] = a.x, w[i][1] = a.y, w[i][2] = a.z, w[i][3] = a.w;
            w[i][4] = b.x, w[i][5] = b.y, w[i][6] = b.z, w[i][7] = b.w;
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 8; ++k) to[32 * k] = make_uint4(w[0][k], w[1][k], w[2][k], w[3][k]);
        fence_proxy_async_smem();
        __syncwarp();
        if (elect_one()) arrive_cluster_release_smem(ready + 8 * slot);
        if (++slot == C::kSlots) slot = 0, par ^= 1u;
    }
}

// Rows of KB scales, a multiple of 2 but not of 16, are no strides of a tensor map; 2^lg(KB) rows together are. One copy
// then brings every 2^lg-th row: of each the three 16-byte pieces that 32 bytes may lie in, from byte (row KB) mod 16 on.
// Row l of the 128 is row l >> lg of copy l mod 2^lg.
__host__ __device__ __forceinline__ int strided_lg(int KB) { return KB & 2 ? 3 : KB & 4 ? 2 : 1; }
__device__ __forceinline__ int odd_place(int l, int lg) { return (((l & ((1 << lg) - 1)) << (7 - lg)) + (l >> lg)) * kOddBytes; }

struct OddCopies {
    int lg, x[8], y[8];
    __device__ __forceinline__ void rows(int first, int KB) {
        lg = strided_lg(KB);
#pragma unroll
        for (int c = 0; c < 8; ++c) x[c] = ((first + c) & ((1 << lg) - 1)) * KB & ~15, y[c] = (first + c) >> lg;
    }
    __device__ __forceinline__ void bring(uint32_t to, const CUtensorMap* map, int byte, uint64_t* bar) const {
#pragma unroll
        for (int c = 0; c < 8; ++c)
            if (c < 1 << lg) tma_load_2d(to + c * ((kM >> lg) * kOddBytes), map, x[c] + byte, y[c], bar);
    }
};

// The same for rows of KB scales that OddCopies, or the gather warps in their order, brought. The array's last rows, where
// they make no 2^lg, lie behind the map's end (zeros): the warp loads them itself.
template <typename C>
__device__ __forceinline__ void odd_scale_warp(const Fp4Product& Q, WalkOf<C::kRound> at, int pairs, int m_begin, int blk,
                                               int rank, uint8_t* slots, uint64_t* raw, uint32_t ready, const Waiter& wait) {
    const RowsProduct& P = Q.r;
    const int lane = threadIdx.x & 31, KB = P.K / 16, l0 = (blk - 1) * 128;
    const uint8_t* base = blk == 0 ? Q.ws : Q.xs;
    const int lg = strided_lg(KB), rows = blk == 0 ? P.E * P.N : P.x_rows, whole = rows >> lg ? rows >> lg << lg : rows;
    const bool listed = blk != 0 && P.gather;
    TileOf<C::kRound> t{};
    int entry[4] = {};
    const auto ask = [&] {
        t = at.tile();
        if (!listed) return;
#pragma unroll
        for (int i = 0; i < 4; ++i) entry[i] = P.list[t.r0 + min(l0 + 32 * i + lane, t.n - 1)];
    };
    if (at.more()) ask();
    int slot = 0;
    uint32_t par = 0;
#pragma unroll 1
    while (at.more()) {
        const int first = blk == 0 ? t.e * P.N + t.m0 + rank * kM : t.r0 + l0;
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = !listed ? first + 32 * i + lane : (unsigned)entry[i] < (unsigned)P.R ? entry[i] / P.k : 0;
            o[i] = (uint32_t)row * KB & 15u;
        }
        // rows the copies leave out, four lanes each
        const int spare0 = max(first, whole), spares = listed ? 0 : min(rows, first + 128) - spare0, spare = spare0 + (lane >> 2);
        at.next();
        if (at.more()) ask();
#pragma unroll 1
        for (int j = 0; j < pairs; ++j) {
            const int byte = kSectorBytes * (m_begin + j);
            uint8_t* blkp = slots + slot * C::kSlotBytes + blk * C::kBlkBytes;
            uint16_t late[4];
            if (spares > 0) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int b = byte + 8 * (lane & 3) + 2 * k;
                    late[k] = *reinterpret_cast<const uint16_t*>(base + (size_t)min(spare, rows - 1) * KB + min(b, KB - 2));
                }
            }
            if (!wait(&raw[slot], par)) return;
            if (spares > 0) {
                const int l = spare - first;
                uint8_t* p = blkp + odd_place(l, lg) + ((uint32_t)spare * KB & 15u) + 8 * (lane & 3);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (lane >> 2 < spares) *reinterpret_cast<uint16_t*>(p + 2 * k) = late[k];
                __syncwarp();
            }
            uint32_t w[4][8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t* p = reinterpret_cast<const uint32_t*>(
                    blkp + odd_place(32 * i + lane, lg) + (o[i] & 12u));
                uint32_t r[9];
#pragma unroll
                for (int k = 0; k < 9; ++k) r[k] = p[k];
#pragma unroll
                for (int k = 0; k < 8; ++k) w[i][k] = __funnelshift_r(r[k], r[k + 1], 8 * (o[i] & 2u));
            }
            if (KB < byte + kSectorBytes) {            // the row ends in these steps
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int left = KB - (byte + 4 * k);
                    const uint32_t keep = left >= 4 ? 0xFFFFFFFFu : left > 0 ? 0xFFFFu : 0u;
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[i][k] &= keep;
                }
            }
            __syncwarp();
            uint4* to = reinterpret_cast<uint4*>(blkp) + lane;
#pragma unroll
            for (int k = 0; k < 8; ++k) to[32 * k] = make_uint4(w[0][k], w[1][k], w[2][k], w[3][k]);
            fence_proxy_async_smem();
            __syncwarp();
            if (elect_one()) arrive_cluster_release_smem(ready + 8 * slot);
            if (++slot == C::kSlots) slot = 0, par ^= 1u;
        }
    }
}

// The warp that looks up what the epilogue needs of a tile: for its columns row scale and address of the row of y, for the
// CTA's outputs the tensor scale. The list entries of the next tile are asked for with this one's scales.
template <typename C>
__device__ __forceinline__ void ends_warp(const Fp4Product& Q, WalkOf<C::kRound> at, int rank, uint8_t* ends,
                                          uint64_t* ends_full, uint64_t* ends_empty, const Waiter& wait) {
    constexpr int kPer = C::kNT / 32;
    const RowsProduct& P = Q.r;
    const int lane = threadIdx.x & 31, part_rows = P.N / Q.parts;
    const bool listed = P.gather || P.scatter;
    if (!at.more()) return;
    auto t = at.tile();
    int entry[kPer];
    const auto ask = [&] {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int r = t.r0 + min(32 * i + lane, t.n - 1);
            entry[i] = listed ? P.list[r] : r;
        }
    };
    ask();
    int end = 0;
    uint32_t par = 0;
#pragma unroll 1
    for (bool more = true; more;) {
        const auto now = t;
        int src[kPer], d[kPer];
        float f[kPer], w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = Q.wt[(size_t)now.e * Q.parts + min(now.m0 + rank * kM + 32 * i + lane, P.N - 1) / part_rows];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int col = 32 * i + lane, r = now.r0 + min(col, now.n - 1);
            const bool good = (unsigned)entry[i] < (unsigned)P.R;
            src[i] = P.gather ? (good ? entry[i] / P.k : -1) : r;
            d[i] = col < now.n ? (P.scatter ? (good ? entry[i] : -1) : r) : -1;
            f[i] = Q.xr[max(src[i], 0)];
        }
        at.next();
        more = at.more();
        if (more) t = at.tile(), ask();
        if (!wait(&ends_empty[end], par ^ 1u)) return;
        unsigned long long* to = reinterpret_cast<unsigned long long*>(ends + end * C::kEndsBytes);
        float* scale = reinterpret_cast<float*>(to + C::kNT);
        float* tensor = scale + C::kNT;
        int* tile = reinterpret_cast<int*>(tensor + kM);
#pragma unroll
        for (int i = 0; i < 4; ++i) tensor[32 * i + lane] = w[i];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            scale[32 * i + lane] = src[i] < 0 ? 0.f : f[i];
            to[32 * i + lane] = d[i] < 0 ? 0ull : (unsigned long long)P.y + ((unsigned long long)d[i] * P.N << (P.y_f32 ? 2 : 1));
        }
        if (lane == 0) tile[0] = now.n, tile[1] = now.m0;
        __syncwarp();
        if (elect_one()) mbar_arrive(&ends_full[end]);
        if (++end == C::kEnds) end = 0, par ^= 1u;
    }
}

// Past L1, which keeps room for the scales and lists (4096 x 8192 x 2048: 33.9 us, with plain stores 35.1).
__device__ __forceinline__ void store_once(unsigned long long at, const uint4 v) {
    asm volatile("st.global.L1::no_allocate.v4.u32 [%0], {%1, %2, %3, %4};"
                 :: "l"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// (a, b) *= s * t, each product rounded: the packed fp32 pipe.
__device__ __forceinline__ void scale2(float& a, float& b, const float2 s, float t) {
    asm("{\n .reg .b64 v, s, t;\n mov.b64 v, {%0, %1};\n mov.b64 s, {%2, %3};\n mov.b64 t, {%4, %4};\n"
        " mul.rn.f32x2 s, s, t;\n mul.rn.f32x2 v, v, s;\n mov.b64 {%0, %1}, v;\n}"
        : "+f"(a), "+f"(b) : "f"(s.x), "f"(s.y), "f"(t));
}

// SPLITS: pairs of a cluster, which share a tile's K.
template <int NT, bool ODD, int SPLITS>
__global__ void __cluster_dims__(2 * SPLITS, 1, 1) __launch_bounds__(Cfg<NT, ODD>::kThreads, 1)
rows_fp4_kernel(const Fp4Product Q, const __grid_constant__ Fp4Maps maps, int m_tiles, int max_tiles, WsHeader* hdr,
                unsigned long long wait_limit) {
    using C = Cfg<NT, ODD>;
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
    uint64_t* sf_raw = acc_empty + C::kBufs;                           // scales of two steps landed
    uint64_t* sf_ready = sf_raw + C::kSlots;                           // first CTA: ... and are in line order in both
    uint64_t* sf_empty = sf_ready + C::kSlots;                         // ... and copied to tensor memory
    uint64_t* ends_full = sf_empty + C::kSlots;                        // scales and rows of a tile's outputs
    uint64_t* ends_empty = ends_full + C::kEnds;                       // ... and read
    uint64_t* done = ends_empty + C::kEnds;                            // every MMA of the pair
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* tab = reinterpret_cast<int*>(sm + C::kOffTab);
    volatile int* widths = reinterpret_cast<volatile int*>(sm + C::kOffWidths);

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
            for (int i = 0; i < C::kSlots; ++i) {
                mbar_init(&sf_raw[i], P.gather ? 1 + 32 * kGatherWarps : ODD ? C::kBlocks : 1);
                mbar_init(&sf_ready[i], 2 * C::kBlocks);
                mbar_init(&sf_empty[i], 1);
            }
            for (int i = 0; i < C::kEnds; ++i) {
                mbar_init(&ends_full[i], 1);
                mbar_init(&ends_empty[i], kEpiWarps);
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
    // scales come for steps 2 m and 2 m + 1 together, by TMA where their rows can be strides of a tensor map
    const int m_begin = s_begin >> 1, m_pairs = ((s_end - 1) >> 1) - m_begin + 1, KB = P.K / 16;
    using Walk = WalkOf<C::kRound>;
    using Tile = TileOf<C::kRound>;
    const Walk tiles(tab, P.E, m_tiles, blockIdx.x / kCluster, gridDim.x / kCluster, total);
    const int tiles_here = tiles.more() ? (total - 1 - tiles.i) / tiles.step + 1 : 0;
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
    auto drain_scales = [&](int m) {
        for (int i = max(0, m - C::kSlots); i < m; ++i)
            mbar_wait_bounded(&sf_raw[i % C::kSlots], (i / C::kSlots) & 1, kCopyDrainNs);
    };

    if (warp >= kEpiWarps) {
        if (warp == kTmaWarp) {
            int step = 0, two = 0, i_tile = 0;                                  // steps, pairs of steps and tiles so far
            // Weights that are read about once leave the L2 first (us, 256 experts: 64 tokens gate/up 39.7 / 36.0, down 23.4 /
            // 21.6, 512 tokens down 35.5 / 32.0; 248320 x 2048, one row 62.3 / 59.3). Others stay (4096 x 8192 x 8192
            // 90 / 100).
            const uint64_t w_policy = l2_policy(P.R <= P.E * NT);
            bool ok = true;
#pragma unroll 1
            for (Walk at = tiles; at.more() && ok; at.next(), ++i_tile) {
                const Tile t = at.tile();
                const int share = t.mma_n() / 2;                                // rows of x here
                const int wy = t.e * P.N + t.m0 + rank * kM;
                const int boxes = P.gather ? 0 : (share + C::kBoxRows - 1) / C::kBoxRows;
                const uint32_t bytes = kABytes + boxes * (C::kBoxRows * kStepBytes);
                OddCopies odd;
                if constexpr (ODD) odd.rows(wy, KB);
#pragma unroll 1
                for (int s = s_begin; s < s_end; ++s, ++step) {
                    if ((!ODD || P.gather) && (s == s_begin || (s & 1) == 0)) {
                        const int sl = two % C::kSlots, u = two / C::kSlots;
                        if (u > 0) ok = wait(&sf_empty[sl], (u - 1) & 1);
                        if (!ok) break;
                        const uint32_t to = sm_base + C::kOffSlots + sl * C::kSlotBytes;
                        if constexpr (ODD) {
                            if (elect_one()) {
                                mbar_arrive_expect_tx(&sf_raw[sl], kM * kOddBytes);
                                odd.bring(to, &maps.ws, (s >> 1) * kSectorBytes, &sf_raw[sl]);
                            }
                        } else if (elect_one()) {
                            mbar_arrive_expect_tx(&sf_raw[sl], C::kBlkBytes + (P.gather ? 0 : NT * kSectorBytes));
                            tma_load_2d(to, &maps.ws, (s >> 1) * kSectorBytes, wy, &sf_raw[sl]);
                            if (!P.gather) tma_load_2d(to + C::kBlkBytes, &maps.xs, (s >> 1) * kSectorBytes, t.r0, &sf_raw[sl]);
                        }
                        ++two;
                    }
                    const int st = step % C::kStages, u = step / C::kStages;
                    if (u > 0) ok = wait(&empty[st], (u - 1) & 1);
                    if (!ok) break;
                    const uint32_t a = sm_base + st * C::kStage, b = a + kABytes;
                    if (elect_one()) {
                        if (s == s_begin) widths[i_tile % kWidths] = 2 * share;  // for the MMA thread, with the arrival
                        mbar_arrive_expect_tx(&full[st], bytes);
                        tma_load_2d_policy(a, &maps.w, s * kStepBytes, wy, &full[st], w_policy);
                        for (int i = 0; i < boxes; ++i)
                            tma_load_2d(b + i * (C::kBoxRows * kStepBytes), &maps.x, s * kStepBytes,
                                        t.r0 + rank * share + i * C::kBoxRows, &full[st]);
                    }
                }
            }
            if (lane == 0) {
                drain(step);
                drain_scales(two);
            }
        } else if (warp == kMmaWarp) {
            // One thread: in a loop of the whole warp with votes at every wait the waits that did not have to wait took as
            // long as a third of the MMAs.
            if (elect_one()) {
                int st = 0, buf = 0, sl = 0;
                uint32_t st_par = 0, sl_par = 0, buf_par = 1;      // an unused buffer's "empty" phase counts as over
                bool ok = true;
                const uint64_t stage0 = sw128_desc(sm_base), scales0 = lines_desc(sm_base + C::kOffSlots);
#pragma unroll 1
                for (int i = 0; i < tiles_here && ok; ++i) {
                    uint32_t idesc = 0;
#pragma unroll 1
                    for (int s = s_begin; s < s_end; ++s) {
                        if (rank == 0 && (s == s_begin || (s & 1) == 0)) ok = wait.one<true>(&sf_ready[sl], sl_par);
                        if (ok) ok = wait.one(&full[st], st_par);
                        if (!ok) break;
                        const bool sl_done = (s & 1) != 0 || s == s_end - 1;
                        if (rank != 0) {
                            arrive_cluster(map_rank(su32(&full[st]), first_rank));
                        } else {
                            if (s == s_begin) {
                                ok = wait.one(&acc_empty[buf], buf_par);
                                idesc = nvfp4_idesc(widths[i % kWidths]);
                            }
                            if (!ok) break;
                            tc_fence_after();
                            const uint64_t a = stage0 + st * (C::kStage / 16), b = a + kABytes / 16;
                            const uint64_t sf = scales0 + (sl * C::kSlotBytes + (s & 1) * (16 * kM)) / 16;
                            const uint32_t tsf = tmem + C::kSf + (C::kSfSets > 1 ? (s & 1) * C::kSfCols : 0);
                            // columns: 4 for each MMA's scales of W, then 4 kXBlocks for each MMA's of x
#pragma unroll
                            for (int j = 0; j < kMmas; ++j) {
                                copy_scales(tsf + 4 * j, sf + j * (512 / 16));
#pragma unroll
                                for (int k = 0; k < C::kXBlocks; ++k)
                                    copy_scales(tsf + 4 * kMmas + 4 * (C::kXBlocks * j + k),
                                                sf + ((1 + k) * C::kBlkBytes + j * 512) / 16);
                            }
#pragma unroll
                            for (int j = 0; j < kMmas; ++j)      // 32 bytes of K an MMA: 2 address units
                                mma_nvfp4(tmem + buf * NT, a + 2 * j, b + 2 * j, idesc, tsf + 4 * j,
                                          tsf + 4 * kMmas + 4 * C::kXBlocks * j, s != s_begin || j != 0);
                            commit_pair(&empty[st], pair_mask);
                            if (sl_done) commit_pair(&sf_empty[sl], pair_mask);
                            if (s == s_end - 1) {
                                commit_pair(&acc_full[buf], pair_mask);
                                if (++buf == C::kBufs) buf = 0, buf_par ^= 1;
                            }
                        }
                        if (++st == C::kStages) st = 0, st_par ^= 1;
                        if (sl_done && ++sl == C::kSlots) sl = 0, sl_par ^= 1;
                    }
                }
                // no MMA still reads or writes either CTA's memory, nor has an arrival on the way to it, when it is freed
                if (rank == 0) commit_pair(done, pair_mask);
                drain_wait(done, 0);
            }
            __syncwarp();
        } else if (warp == kEndsWarp) {
            ends_warp<C>(Q, tiles, rank, sm + C::kOffEnds, ends_full, ends_empty, wait);
        } else if (warp < kEndsWarp) {
            if (P.gather) {
                // copies of four rows, in turn over the warps: at most kPer a warp and step; lane 4 j + r has
                // row r of this warp's copy j
                constexpr int kPer = (NT / 2 / 4 + kGatherWarps - 1) / kGatherWarps;
                const int w = warp - kGatherWarp0;
                // and the scales of all columns, 16 bytes a lane, neighbours first the pieces of a row (by copies of four rows, 32
                // bytes of each, they cost as much as rows of 128)
                constexpr int kPieces = C::kRowBytes / 16, kSfPer = (NT * kPieces + 127) / 128;
                const auto sf_row = [&](int i) { return (32 * w + lane + 128 * i) / kPieces; };
                const auto sf_piece = [&](int i) { return (32 * w + lane + 128 * i) % kPieces; };
                const size_t sf_bytes = (size_t)P.x_rows * KB;
                const int lg = strided_lg(KB);
                int step = 0, two = 0;
                bool ok = true;
                Walk at = tiles;
                Tile t{};
                // list entries of this lane's rows, asked for a tile ahead: of x, then of the scales
                int entry[1 + kSfPer];
                const int l = 4 * (w + kGatherWarps * (lane >> 2)) + (lane & 3);
                const auto ask = [&] {
                    t = at.tile();
                    const int col = rank * (t.mma_n() / 2) + l;
                    entry[0] = P.list[t.r0 + min(col, t.n - 1)];
#pragma unroll
                    for (int i = 0; i < kSfPer; ++i) entry[1 + i] = P.list[t.r0 + min(sf_row(i), t.n - 1)];
                };
                if (at.more()) ask();
#pragma unroll 1
                while (at.more() && ok) {
                    const int share = t.mma_n() / 2, copies = share / 4, n = t.n;
                    const auto row_of = [&](int e, int col) { return col < n && (unsigned)e < (unsigned)P.R ? e / P.k : -1; };
                    int src = row_of(entry[0], l < share ? rank * share + l : n);
                    if (src < 0) src = P.x_rows;                     // past the last row: zeros
                    int sf_src[kSfPer];
#pragma unroll
                    for (int i = 0; i < kSfPer; ++i) sf_src[i] = row_of(entry[1 + i], sf_row(i));
                    at.next();
                    if (at.more()) ask();
                    const int mine = (copies - w + kGatherWarps - 1) / kGatherWarps;
                    int rows4[kPer][4];
#pragma unroll
                    for (int j = 0; j < kPer; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i) rows4[j][i] = __shfl_sync(0xffffffffu, src, 4 * j + i);
#pragma unroll 1
                    for (int s = s_begin; s < s_end; ++s, ++step) {
                        if (s == s_begin || (s & 1) == 0) {
                            const int sl = two % C::kSlots, u = two / C::kSlots;
                            if (u > 0) ok = wait(&sf_empty[sl], (u - 1) & 1);
                            if (!ok) break;
                            const uint32_t to = sm_base + C::kOffSlots + sl * C::kSlotBytes + C::kBlkBytes;
#pragma unroll
                            for (int i = 0; i < kSfPer; ++i) {
                                const int l = sf_row(i), piece = sf_piece(i), byte = (s >> 1) * kSectorBytes + 16 * piece;
                                if (l >= NT) break;
                                size_t from = (size_t)max(sf_src[i], 0) * KB;
                                if constexpr (ODD) {           // as odd_scale_warp wants them; the array may end in a piece
                                    from = (from & ~(size_t)15) + byte;
                                    const int left = from < sf_bytes ? (int)min(sf_bytes - from, (size_t)16) : 0;
                                    const int there = sf_src[i] >= 0 ? left : 0;
                                    cp_async16_zfill(to + (l >> 7) * C::kBlkBytes + odd_place(l & 127, lg) + 16 * piece,
                                                     Q.xs + (there > 0 ? from : 0), there);
                                } else {                       // in the order of the 32-byte swizzle (scale_warp)
                                    const bool there = sf_src[i] >= 0 && byte < KB;
                                    cp_async16_zfill(to + l * kSectorBytes + 16 * (piece ^ ((l >> 2) & 1)),
                                                     Q.xs + (there ? from + byte : 0), there ? 16 : 0);
                                }
                            }
                            cp_async_arrive_noinc(&sf_raw[sl]);
                            ++two;
                        }
                        const int st = step % C::kStages, u = step / C::kStages;
                        if (u > 0) ok = wait(&empty[st], (u - 1) & 1);
                        if (!ok) break;
                        const uint32_t b = sm_base + st * C::kStage + kABytes + w * 4 * kStepBytes;
                        if (elect_one()) mbar_arrive_expect_tx(&full[st], mine * 4 * kStepBytes);
#pragma unroll
                        for (int j = 0; j < kPer; ++j) {
                            if (j >= mine) break;
                            if (elect_one())
                                tma_gather4(b + j * (kGatherWarps * 4 * kStepBytes), &maps.x, s * kStepBytes,
                                            rows4[j][0], rows4[j][1], rows4[j][2], rows4[j][3], &full[st]);
                        }
                    }
                }
                asm volatile("cp.async.wait_all;" ::: "memory");
                if (lane == 0) {
                    drain(step);
                    drain_scales(two);
                }
            } else if (const int blk = warp - kGatherWarp0; ODD && blk < C::kBlocks) {
                // these warps bring the scales (24 copies of the TMA warp's, in one go, held up those of its operands)
                int two = 0;
                bool ok = true;
#pragma unroll 1
                for (Walk at = tiles; at.more() && ok; at.next()) {
                    const Tile t = at.tile();
                    OddCopies odd;
                    odd.rows(blk == 0 ? t.e * P.N + t.m0 + rank * kM : t.r0 + 128 * (blk - 1), KB);
#pragma unroll 1
                    for (int j = 0; j < m_pairs; ++j, ++two) {
                        const int sl = two % C::kSlots, u = two / C::kSlots;
                        if (u > 0) ok = wait(&sf_empty[sl], (u - 1) & 1);
                        if (!ok) break;
                        if (elect_one()) {
                            mbar_arrive_expect_tx(&sf_raw[sl], (blk == 0 ? kM : C::kXRows) * kOddBytes);
                            odd.bring(sm_base + C::kOffSlots + sl * C::kSlotBytes + blk * C::kBlkBytes,
                                      blk == 0 ? &maps.ws : &maps.xs, (m_begin + j) * kSectorBytes, &sf_raw[sl]);
                        }
                    }
                }
                if (lane == 0) drain_scales(two);
            }
        } else {
            const int blk = warp - kScaleWarp0;
            uint8_t* slots = sm + C::kOffSlots;
            const uint32_t ready = map_rank(su32(sf_ready), first_rank);
            if constexpr (ODD) odd_scale_warp<C>(Q, tiles, m_pairs, m_begin, blk, rank, slots, sf_raw, ready, wait);
            else scale_warp<C>(tiles_here * m_pairs, blk, slots, sf_raw, ready, wait);
        }
        if (SPLITS > 1 && tiles.more()) exchange.join();
    } else {
        const int q = warp & 3, part = warp >> 2;          // lanes 32 q .., a quarter of the columns
        uint8_t* stg = sm + C::kOffStg + warp * (kStgRows * kStgPitch);
        const int p = lane & 3, g = lane >> 2;
        const uint32_t first_acc_empty = map_rank(su32(acc_empty), first_rank);
        int end = 0;
        uint32_t end_par = 0;
        bool ok = true;
#pragma unroll 1
        for (int use = 0; use < tiles_here; ++use) {
            const int buf = use % C::kBufs;
            const uint32_t lanes = tmem + ((uint32_t)(32 * q) << 16) + buf * NT;
            if (ok) ok = wait(&ends_full[end], end_par);
            const unsigned long long* to = reinterpret_cast<const unsigned long long*>(sm + C::kOffEnds + end * C::kEndsBytes);
            const float* scale = reinterpret_cast<const float*>(to + NT);
            const float* tensor = scale + NT;
            int rows = reinterpret_cast<const int*>(tensor + kM)[0], m0 = reinterpret_cast<const int*>(tensor + kM)[1], r0 = 0;
            float wt[4];                                                   // tensor scales of outputs n0 + 8 i + g
#pragma unroll
            for (int i = 0; i < 4; ++i) wt[i] = tensor[32 * q + 8 * i + g];
            if (ok) ok = wait(&acc_full[buf], (use / C::kBufs) & 1);
            if (!ok) {                                                     // an abandoned call: nobody looked this tile up
                Walk at = tiles;
                for (int i = 0; i < use; ++i) at.next();
                const Tile t = at.tile();
                rows = t.n, m0 = t.m0, r0 = t.r0;
            }
            tc_fence_after();
            const int n0 = m0 + rank * kM + 32 * q;                        // first output
            const int width = ((rows + C::kRound - 1) & ~(C::kRound - 1)) / 4;
            const auto hand_back = [&] {
                tc_fence_before();
                __syncwarp();
                if (ok && elect_one()) arrive_cluster(first_acc_empty + 8 * buf);
            };
            // sums of columns c .. c + 15 times their two scales; v[8 L + 4 j + 2 u + b]: output 16 L + 8 u + g, column
            // 8 j + 2 p + b
            const auto scaled = [&](int c, float (&v)[16]) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float2 s = *reinterpret_cast<const float2*>(scale + c + 8 * j + 2 * p);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int k = 8 * (i >> 1) + 4 * j + 2 * (i & 1);
                        scale2(v[k], v[k + 1], s, wt[i]);
                    }
                }
                if (!ok)
#pragma unroll
                    for (int k = 0; k < 16; ++k) v[k] = __uint_as_float(0x7FC00000u);
            };
            // rows of y that are no multiple of 16 bytes, fp32, and abandoned calls
            const auto store_any = [&](int c, const float (&v)[16]) {
                const int col = c + (lane & 15);
                int d = -1;
                if (col < rows) {
                    if (ok) {
                        const unsigned long long a = to[col];
                        if (a != 0) d = (int)((a - (unsigned long long)P.y >> (P.y_f32 ? 2 : 1)) / (unsigned long long)P.N);
                    } else {
                        d = y_row(P, r0 + col);
                    }
                }
                store_frag(P, v, d, n0, stg);
            };
            // bf16 with rows of whole 16-byte pieces: 16 rows of 32 outputs through shared memory. Piece m of row r lies at
            // 64 r + 16 (m ^ (r >> 1) % 4): neither eight rows of a piece nor two whole rows meet on a bank.
            const uint32_t st_to = su32(stg) + (lane & 7) * 64 + 16 * ((lane >> 3) ^ ((lane >> 1) & 3));
            const uint8_t* st_from = stg + g * 64 + 16 * (p ^ ((g >> 1) & 3));
            const bool piece = n0 + 8 * p < P.N;
            const auto store16 = [&](int c, const uint32_t (&w)[8]) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};"
                                 :: "r"(st_to + 512 * j), "r"(w[4 * j]), "r"(w[4 * j + 1]), "r"(w[4 * j + 2]), "r"(w[4 * j + 3])
                                 : "memory");
                const unsigned long long a0 = to[c + g], a1 = to[c + 8 + g];
                __syncwarp();
                const uint4 u0 = *reinterpret_cast<const uint4*>(st_from), u1 = *reinterpret_cast<const uint4*>(st_from + 512);
                const unsigned long long o = 2ull * (unsigned)(n0 + 8 * p);
                if (a0 != 0 && piece) store_once(a0 + o, u0);
                if (a1 != 0 && piece) store_once(a1 + o, u1);
                __syncwarp();
            };
            const auto packed = [&](const float (&v)[16], uint32_t (&w)[8]) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int k = 8 * (i >> 1) + 4 * j + 2 * (i & 1);
                        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[4 * j + i]) : "f"(v[k + 1]), "f"(v[k]));
                    }
            };
            const bool plain = ok && !P.y_f32 && (P.N & 7) == 0;
            if constexpr (SPLITS > 1) {
                const int c0 = part * width;                               // this warp's columns of the tile
                const auto sums = [&](int c, float (&v)[16]) {
                    if (ok) {
                        tmem_ld_frag(lanes + c0 + c, v);
                        tmem_wait16(v);
                    } else {
#pragma unroll
                        for (int k = 0; k < 16; ++k) v[k] = __uint_as_float(0x7FC00000u);
                    }
                };
                Tile t{};
                t.n = rows;
                exchange.send(sums, t, width, c0, part, q);
#pragma unroll
                for (int c = 0; c < C::kCols; c += 16) {
                    if (c >= width || c0 + c >= rows) break;
                    float v[16];
                    sums(c, v);
                    if (!exchange.finish(v, c, width, part, q)) continue;
                    scaled(c0 + c, v);
                    if (plain) {
                        uint32_t w[8];
                        packed(v, w);
                        store16(c0 + c, w);
                    } else {
                        store_any(c0 + c, v);
                    }
                }
            } else {
                // Chunks of 16 columns go round the warps; the next is asked for before this one is written. A buffer is
                // handed back when its last chunk is in registers.
                const int chunks = (rows - 16 * part + 63) / 64;           // none where it is not positive
                float v[16];
                if (chunks <= 0) hand_back();
                if (plain) {
                    if (chunks > 0) tmem_ld_frag(lanes + 16 * part, v);
#pragma unroll 1
                    for (int i = 0; i < chunks; ++i) {
                        const int c = 64 * i + 16 * part;
                        tmem_wait16(v);
                        if (i == chunks - 1) hand_back();
                        scaled(c, v);
                        uint32_t w[8];
                        packed(v, w);
                        if (i + 1 < chunks) tmem_ld_frag(lanes + c + 64, v);
                        store16(c, w);
                    }
                } else {
#pragma unroll 1
                    for (int i = 0; i < chunks; ++i) {
                        const int c = 64 * i + 16 * part;
                        if (ok) {
                            tmem_ld_frag(lanes + c, v);
                            tmem_wait16(v);
                        }
                        if (i == chunks - 1) hand_back();
                        scaled(c, v);
                        store_any(c, v);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&ends_empty[end]);
            if (++end == C::kEnds) end = 0, end_par ^= 1u;
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
template <int NT, bool ODD, int SPLITS>
cudaError_t resident_clusters(const DeviceInfo& dev, int* clusters) {
    using C = Cfg<NT, ODD>;
    static std::atomic<int> known[64];           // by device: one more than the clusters
    int n = known[dev.device].load(std::memory_order_acquire) - 1;
    if (n < 0) {
        const auto kernel = rows_fp4_kernel<NT, ODD, SPLITS>;
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

// Tiles of NT columns with one, two or four pairs each, if the estimate makes them the best so far.
//
// The estimate (us) is a launch, then for every round of tiles its steps and the part of its epilogue that the next tile's
// steps do not hide; tiles that pairs share add the exchange of their sums. Its constants are fitted to the times of all
// seven forms at 33 .. 4096 rows, 2048 and 8192 outputs and K of 512, 2048 and 4096; there the form that it takes is at
// most 6% (0.4% on average) slower than the best; over 2 to 256 experts, whose rows it does not know, at most 16% (1.7%).
//     4096 x 8192 x 2048   64 columns 68.6, 128: 41.8, 224: 33.5        128 x 8192 x 2048   64: 6.7, 128: 7.0, 224: 7.6
//      512 x 8192 x 2048   64 columns 13.3, 128: 10.0, 224: 11.3        256 x 2048 x 512    64: 5.3, 128: 5.7, 224: 6.1
//     33 x 2048 x 4096     64 columns, one pair 7.8, two 7.2, four 6.7  33 x 2048 x 2048    one 6.2, two 6.4, four 6.3
// The host does not know how rows spread over experts: an expert is taken to have half a tile more than its even share.
template <int NT, bool ODD>
cudaError_t plan_tiles(const RowsProduct& P, const DeviceInfo& dev, Plan* best) {
    const int m_tiles = (P.N + 2 * kM - 1) / (2 * kM), nk = (P.K + kStepK - 1) / kStepK;
    const int groups = std::min(P.R, P.E), rows = (P.R + groups - 1) / groups, pairs = dev.num_sms / 2;
    // tiles at most: every expert has rows, and its last tile one
    const long long tiles = ((P.R - groups) / NT + groups) * (long long)m_tiles;
    float parts, n, rounds;                  // tiles of an expert's rows, their rows (in 16s), tiles of a pair
    if (groups == 1) {
        const int p = (rows + NT - 1) / NT;
        parts = (float)p;
        n = (float)(((rows + p - 1) / p + 15) / 16 * 16);
        rounds = (float)(((long long)p * m_tiles + pairs - 1) / pairs);
    } else {
        parts = std::max(1.0f, (float)rows / NT + 0.5f);
        n = std::max(std::min((float)NT, rows / parts + 8), NT / 4.0f);
        rounds = std::max(1.0f, std::ceil(groups * parts * m_tiles / pairs - 0.25f));
    }
    for (int splits = 1; splits <= (NT <= 128 ? 4 : 1); splits *= 2) {
        if (splits > 1) {
            // no more tiles than clusters that run at a time, and kMinSteps steps for each pair
            if (nk < kMinSteps * splits || tiles * splits > pairs) break;
            int clusters = 0;
            if constexpr (NT <= 128) {
                const cudaError_t e = splits == 2 ? resident_clusters<NT, ODD, 2>(dev, &clusters)
                                                  : resident_clusters<NT, ODD, 4>(dev, &clusters);
                if (e != cudaSuccess) return e;
            }
            if (tiles > clusters) break;
        }
        const float joined = splits == 1 ? 0.0f : splits == 2 ? 0.5f + 0.0095f * n : 0.5f + 0.0165f * n;
        const float us = 4.2f + rounds * ((nk + splits - 1) / splits * (0.21f + 0.00025f * n) + 0.0074f * n) + joined;
        if (us < best->us) *best = Plan{NT, splits, tiles, us};
    }
    return cudaSuccess;
}

template <int NT, bool ODD, int SPLITS>
cudaError_t launch_clusters(const Fp4Product& P, const Fp4Maps& maps, int tiles, WsHeader* hdr,
                            const DeviceInfo& dev, uint64_t wait_limit, cudaStream_t s) {
    int resident = 0;
    if (cudaError_t e = resident_clusters<NT, ODD, SPLITS>(dev, &resident); e != cudaSuccess) return e;
    if (resident < 1) return cudaErrorInvalidConfiguration;
    const int clusters = SPLITS > 1 ? tiles : std::min(tiles, resident), m_tiles = (P.r.N + 2 * kM - 1) / (2 * kM);
    return launch_pdl(rows_fp4_kernel<NT, ODD, SPLITS>, 2 * SPLITS * clusters, Cfg<NT, ODD>::kThreads, Cfg<NT, ODD>::kSmem, s, P, maps,
                      m_tiles, tiles, hdr, (unsigned long long)wait_limit);
}

// [rows, KB] block scales, read as box_rows x 32 bytes, 32-byte swizzled in shared memory.
bool encode_scales(PFN_cuTensorMapEncodeTiled_v12000 fn, CUtensorMap* m, const void* base, uint64_t KB, uint64_t rows,
                   uint32_t box_rows) {
    const cuuint64_t dims[2] = {KB, rows};
    const cuuint64_t strides[1] = {KB};
    const cuuint32_t box[2] = {kSectorBytes, box_rows};
    const cuuint32_t one[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, one,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_32B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The same for OddCopies of box_rows rows together: 2^lg rows are one of the map. Where there are fewer, these are its one.
bool encode_odd_scales(PFN_cuTensorMapEncodeTiled_v12000 fn, CUtensorMap* m, const void* base, uint64_t KB, uint64_t rows,
                       uint32_t box_rows) {
    const int lg = strided_lg((int)KB);
    const cuuint64_t dims[2] = {KB * std::min<uint64_t>(rows, 1u << lg), std::max<uint64_t>(rows >> lg, 1)};
    const cuuint64_t strides[1] = {KB << lg};
    const cuuint32_t box[2] = {kOddBytes, box_rows >> lg};
    const cuuint32_t one[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, one,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NT, bool ODD>
cudaError_t launch_tiles(const Fp4Product& P, const Plan& plan, WsHeader* hdr, const DeviceInfo& dev,
                         uint64_t wait_limit, cudaStream_t s) {
    PFN_cuTensorMapEncodeTiled_v12000 fn = tensor_map_encoder();
    Fp4Maps maps;
    const uint64_t bytes = P.r.K / 2;
    if (fn == nullptr || !encode_rows(fn, &maps.w, P.r.w, true, bytes, (uint64_t)P.r.E * P.r.N, kM)) return cudaErrorInvalidValue;
    if (!encode_rows(fn, &maps.x, P.r.x, true, bytes, P.r.x_rows, P.r.gather ? 1 : Cfg<NT, ODD>::kBoxRows)) return cudaErrorInvalidValue;
    const uint64_t KB = P.r.K / 16, w_rows = (uint64_t)P.r.E * P.r.N;
    if (ODD ? !encode_odd_scales(fn, &maps.ws, P.ws, KB, w_rows, kM) ||
                  !encode_odd_scales(fn, &maps.xs, P.xs, KB, P.r.x_rows, Cfg<NT, ODD>::kXRows)
            : !encode_scales(fn, &maps.ws, P.ws, KB, w_rows, kM) ||
              !encode_scales(fn, &maps.xs, P.xs, KB, P.r.x_rows, P.r.gather ? 1 : NT))
        return cudaErrorInvalidValue;
    const int tiles = (int)plan.tiles;
    if constexpr (NT <= 128) {
        if (plan.splits == 4) return launch_clusters<NT, ODD, 4>(P, maps, tiles, hdr, dev, wait_limit, s);
        if (plan.splits == 2) return launch_clusters<NT, ODD, 2>(P, maps, tiles, hdr, dev, wait_limit, s);
    }
    return launch_clusters<NT, ODD, 1>(P, maps, tiles, hdr, dev, wait_limit, s);
}

template <bool ODD>
cudaError_t launch(const Fp4Product& P, WsHeader* hdr, const DeviceInfo& dev, uint64_t wait_limit, cudaStream_t s) {
    Plan plan{};
    plan.us = 3.0e38f;
    const int groups = std::min(P.r.R, P.r.E), rows = (P.r.R + groups - 1) / groups;
    cudaError_t e;
    if ((e = plan_tiles<64, ODD>(P.r, dev, &plan)) != cudaSuccess) return e;
    if ((e = plan_tiles<128, ODD>(P.r, dev, &plan)) != cudaSuccess) return e;
    // Gathered rows cost the widest tiles more, all of whose scales come in pieces, unless an expert has many (us, 128 / 224
    // columns, 1024 outputs: K = 2048, 94 rows to an expert 61 / 69, 256: 62 / 68, 512: 57 / 59, 4096: 51 / 48; K = 2016,
    // 94 rows 71 / 88, 256: 86 / 91, 512: 79 / 77, 4096: 74 / 64).
    if ((!P.r.gather || rows >= 512) && (e = plan_tiles<224, ODD>(P.r, dev, &plan)) != cudaSuccess) return e;
    if (plan.tiles > kMaxTiles) return cudaErrorInvalidConfiguration;
    if (plan.nt == 64) return launch_tiles<64, ODD>(P, plan, hdr, dev, wait_limit, s);
    if (plan.nt == 128) return launch_tiles<128, ODD>(P, plan, hdr, dev, wait_limit, s);
    return launch_tiles<224, ODD>(P, plan, hdr, dev, wait_limit, s);
}

}  // namespace

cudaError_t launch_rows_fp4(const Fp4Product& P, WsHeader* hdr, const DeviceInfo& dev, uint64_t wait_limit,
                            cudaStream_t s) {
    return P.r.K % kStepK == 0 ? launch<false>(P, hdr, dev, wait_limit, s) : launch<true>(P, hdr, dev, wait_limit, s);
}

}  // namespace nvfp4
