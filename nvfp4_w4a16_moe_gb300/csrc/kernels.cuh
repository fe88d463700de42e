// Launchers of the sm_103a kernels (internal; the C ABI in api.cu validates
// arguments and calls these).
#pragma once

#include <algorithm>

#include "common.cuh"

namespace nvfp4 {

struct DeviceInfo {
    int device;
    int num_sms;
    int cc_major, cc_minor;
    size_t smem_optin;
};

cudaError_t launch_pack(const float* w, int N, int K, int kind, uint8_t* packed, void* scales,
                        float* tensor_scale, WsHeader* ws, int num_sms, cudaStream_t s);

// hdr (nullable): where a bounded wait that ran out is recorded
cudaError_t launch_gemv(const nvfp4_weight& W, const uint16_t* x, int T, uint16_t* y, WsHeader* hdr,
                        const DeviceInfo& dev, uint64_t wait_limit, cudaStream_t s);

cudaError_t launch_route_topk(const float* logits, int T, int E, int k, int32_t* ids, float* w,
                              cudaStream_t s);
cudaError_t launch_route_lists(const int32_t* ids, int total, int E, int32_t* offsets,
                               int32_t* token_list, int32_t* active, cudaStream_t s);
cudaError_t launch_route(const float* logits, int T, int E, int k, int32_t* ids, float* w,
                         int32_t* offsets, int32_t* token_list, cudaStream_t s);

// Exchange words of the one-launch single-token kernel: kWordReplicas copies of the E + 1
// logits (8-byte words, each copy padded to 16 words) and of the k*I + Is SwiGLU values
// (4-byte words, each copy padded to 32 words); in 8-byte units.
constexpr int kWordReplicas = 8;
__host__ __device__ inline size_t t1_logit_stride(const moe_layer_desc& d) { return ((size_t)d.E + 1 + 15) & ~size_t(15); }
__host__ __device__ inline size_t t1_h_stride(const moe_layer_desc& d) { return ((size_t)d.k * d.I + d.Is + 31) & ~size_t(31); }
// Exchange area of the cluster form, in 8-byte units: kWordReplicas copies of the Is shared
// values (4-byte tagged words, each copy padded to 32 words), then k * H tagged partial
// outputs (8-byte words).
__host__ __device__ inline size_t t1c_words(const moe_layer_desc& d) {
    return (size_t)kWordReplicas * ((((size_t)d.Is + 31) & ~size_t(31)) / 2) + (size_t)d.k * d.H;
}
__host__ __device__ inline size_t t1_words(const moe_layer_desc& d) {
    const size_t grid = (size_t)kWordReplicas * (t1_logit_stride(d) + t1_h_stride(d) / 2);
    const size_t cl = t1c_words(d);
    return grid > cl ? grid : cl;
}

// Workspace of one layer call (device scratch carved from the caller's buffer).
struct LayerWs {
    WsHeader* hdr;
    float* logits;        // [T, E]
    float* gate_logit;    // [T]        shared-expert sigmoid gate pre-activation
    int32_t* ids;         // [T, k]
    float* w;             // [T, k]
    int32_t* offsets;     // [E + 1]
    int32_t* token_list;  // [T * k]
    int32_t* active;      // [E + 1]    active[0] = A, active[1..A] = expert ids ascending
    float* h;             // [T * k, I] routed SwiGLU intermediates (entry-major)
    float* hs;            // [T, Is]    shared intermediates
    unsigned long long* words;  // [t1_words(d)] (launch tag, value) words of the one-launch kernel
    int32_t* pass_map;    // [E + T*k + 2]  pass_map[0] = P, then (active slot << 8) | pass
    float* part;          // [T*k + T, H]  weighted routed rows, then the shared rows
    uint32_t* amax;       // [T + T*k + T] max |x| of each token, then max |h| of each h row (fp32 bits)
    size_t bytes;
};

LayerWs carve_layer_ws(void* base, const moe_layer_desc& d, int T);
size_t layer_ws_bytes(const moe_layer_desc& d, int T);

// resid (nullable, bf16 [T, H]): added to every output element before its one rounding
cudaError_t launch_moe_decode(const moe_layer_desc& d, const uint16_t* x, int T, uint16_t* y,
                              int32_t* ids_out, float* w_out, const LayerWs& ws,
                              const DeviceInfo& dev, uint64_t wait_limit, cudaStream_t s,
                              const uint16_t* resid = nullptr);

// Multi-token decode on mma.sync (E4M3 scales, H, I, Is multiples of 256, <= 4096).
bool decode_mma_supported(const moe_layer_desc& d, int T);
cudaError_t launch_moe_decode_mma(const moe_layer_desc& d, const uint16_t* x, int T, uint16_t* y,
                                  int32_t* ids_out, float* w_out, const LayerWs& ws, const DeviceInfo& dev,
                                  cudaStream_t s, const uint16_t* resid = nullptr);

// Launch tags of the single-token kernels: every launch adds tag_period(dev) to the
// workspace counter (each of its CTAs adds tag_period / grid size), so the counter is a
// multiple of the period between launches of either form, and a launch's tag is
// counter / period + 1 at any of its CTAs.
unsigned long long t1_tag_period(const DeviceInfo& dev);

// Single-token decode in one launch: the persistent-grid form, or on request the cluster
// form (k clusters of 8 to 16 CTAs) where the shape and the device allow it. form: 0 =
// automatic (the grid form), 1 = grid form, 2 = cluster form (unsupported -> grid form).
void set_t1_form(int form);
bool t1c_supported(const moe_layer_desc& d, int T, const DeviceInfo& dev);
cudaError_t launch_moe_decode_t1c(const moe_layer_desc& d, const uint16_t* x, uint16_t* y, int32_t* ids_out,
                                  float* w_out, const LayerWs& ws, const DeviceInfo& dev, uint64_t wait_limit,
                                  cudaStream_t s, const uint16_t* norm_w, float eps, const uint16_t* resid);
bool fused_decode_supported(const moe_layer_desc& d, int T, const DeviceInfo& dev);
// 2: the cluster form runs this call, 1: the grid form, 0: neither (T != 1 or the shape)
int single_token_form_of(const moe_layer_desc& d, int T, const DeviceInfo& dev);
// resident 16-CTA clusters of the cluster form for this layer (0 when the shape has none)
int t1c_cluster_capacity(const moe_layer_desc& d, const DeviceInfo& dev);
cudaError_t launch_moe_decode_fused(const moe_layer_desc& d, const uint16_t* x, uint16_t* y,
                                    int32_t* ids_out, float* w_out, const LayerWs& ws,
                                    const DeviceInfo& dev, uint64_t wait_limit, cudaStream_t s,
                                    const uint16_t* norm_w = nullptr, float eps = 0.f,
                                    const uint16_t* resid = nullptr);

// Pre-MoE RMSNorm, (1 + w) form: out[t] = bf16(h[t] / sqrt(mean(h[t]^2) + eps) * (1 + w)).
cudaError_t launch_rmsnorm(const uint16_t* h, int T, int H, const uint16_t* w, float eps, uint16_t* out,
                           cudaStream_t s);

// Prefill path (T > 64 tokens, E4M3 scales): grouped tensor-core GEMMs.
constexpr int kTokTile = 256;   // token rows per grouped-GEMM tile

// Everything the two grouped GEMMs read. Slots 0..E-1 are the routed experts
// (rows = their entries in token_list order), slot E the shared expert (rows =
// tokens 0..T-1). tile_prefix[s] is the first kTokTile-row tile of slot s.
struct GroupedParams {
    const uint16_t* x;
    int T, H, E, k, I, Is;
    const uint8_t* gu_packed; const uint8_t* gu_scales; const float* gu_tscale;
    const uint8_t* dn_packed; const uint8_t* dn_scales; const float* dn_tscale;
    const uint8_t* sh_gu_packed; const uint8_t* sh_gu_scales; const float* sh_gu_tscale;
    const uint8_t* sh_dn_packed; const uint8_t* sh_dn_scales; const float* sh_dn_tscale;
    const int32_t* offsets;     // [E + 1]
    const int32_t* token_list;  // [T * k] entries t*k + j grouped by expert
    const int32_t* tile_prefix; // [E + 2]
    const float* w;             // [T, k] routing weights
    const float* gate;          // [T] shared gate pre-activation
    uint16_t* h;                // [T * k, I] bf16, rows in token_list order
    uint16_t* hs;               // [T, Is] bf16
    float* Y;                   // [T, k + 1, H] fp32 scaled expert outputs
};


struct PrefillWs {
    WsHeader* hdr;
    float* logits;        // [T, E]
    float* gate;          // [T]
    int32_t* ids;         // [T, k]
    float* w;             // [T, k]
    int32_t* bcount;      // [ceil(T*k / 1024), E]  per-block counts, then bases
    int32_t* offsets;     // [E + 1]
    int32_t* tile_prefix; // [E + 2]  first kTokTile-row tile of each slot (E = shared)
    int32_t* token_list;  // [T * k]
    uint16_t* h;          // [T * k, I]  bf16 SwiGLU intermediates, token_list order
    uint16_t* hs;         // [T, Is]     bf16 shared intermediates
    float* Y;             // [T, k + 1, H] weighted expert outputs
    size_t bytes;
};

bool prefill_supported(const moe_layer_desc& d, int T);
size_t prefill_ws_bytes(const moe_layer_desc& d, int T);
PrefillWs carve_prefill_ws(void* base, const moe_layer_desc& d, int T);
int prefill_launch_count(const moe_layer_desc& d, int T);
cudaError_t launch_moe_prefill(const moe_layer_desc& d, const uint16_t* x, int T, uint16_t* y,
                               int32_t* ids_out, float* w_out, const PrefillWs& ws, uint64_t wait_limit,
                               cudaStream_t s,
                               const uint16_t* resid = nullptr);
// Grouped tcgen05 GEMM over the token tiles of every slot: mode 0 = gate/up with the
// SwiGLU epilogue (x -> h, hs), mode 1 = down with the weighted epilogue (h, hs -> Y).
cudaError_t launch_grouped_tc(const GroupedParams& P, int mode, int tiles_max, WsHeader* hdr,
                              uint64_t wait_limit, cudaStream_t s);

// Data read once (weights, the quantiser's input): past L1.
__device__ __forceinline__ uint4 ld_once_v4(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// The 8-bit and grouped products and the quantiser are launched with programmatic stream serialisation, which
// takes 1.6 to 2.7 us off a call in a row of calls (one token through 8192 x 2048 8.2 -> 6.6, quantising 4096 x 2048
// 8.2 -> 5.5). Every thread first waits until the kernel before this one is complete and its writes are
// visible (nothing in global memory is touched before, and data is read with plain loads, not through the
// non-coherent path). Only then may the next kernel start: one that reads its weights before its own wait (the
// NVFP4 kernels do) sees all that was enqueued before this kernel, though not this kernel's own outputs: the
// header forbids those as its weights. Releasing it only after a fence behind the last store would allow them, and
// costs 0.3 to 0.8 us a call (one token's gate/up over bf16 experts 7.5 -> 8.3, quantising 4096 x 2048 5.0 -> 5.8).
// Letting it start before the wait measured the same.
__device__ __forceinline__ void pdl_wait_then_trigger() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
template <typename... Params, typename... Args>
cudaError_t launch_pdl(void (*kernel)(Params...), unsigned grid, unsigned threads, size_t smem, cudaStream_t s,
                       Args&&... args) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

// bf16 [B, R, K] -> E4M3 codes and fp32 scales of 1 x 128 (block_rows 1) or 128 x 128 blocks.
cudaError_t launch_fp8_quantize(const uint16_t* x, int B, int R, int K, int block_rows, uint8_t* q, float* scales,
                                cudaStream_t s);

// Rows [R, K] as nvfp4_rows: quantised bf16 rows (kind NVFP4), normed rows, SwiGLU rows.
cudaError_t launch_quantize_rows(const uint16_t* x, int R, int K, const nvfp4_rows& out, cudaStream_t s);
cudaError_t launch_norm_rows(const uint16_t* h, const uint16_t* delta, const uint16_t* w, float eps, int T, int H,
                             uint16_t* h_out, const nvfp4_rows& out, cudaStream_t s);
cudaError_t launch_swiglu_rows(const void* gu, bool f32, int R, int I, const nvfp4_rows& out, cudaStream_t s);
cudaError_t launch_dequantize_rows(const uint8_t* packed, const uint8_t* scales, const float* scale, int scale_rows,
                                   int R, int K, void* y, bool f32, cudaStream_t s);

// Rows sorted by expert and back.
cudaError_t launch_permute(const void* x, bool f32, const int32_t* list, int T, int k, int N, void* rows,
                           int32_t* positions, cudaStream_t s);
cudaError_t launch_combine(const void* rows, bool rows_f32, const float* w, const int32_t* positions,
                           const uint16_t* add, int T, int k, int N, void* y, bool y_f32, cudaStream_t s);
cudaError_t launch_combine_backward(const void* dy, bool dy_f32, const void* rows, bool rows_f32, const float* w,
                                    const int32_t* positions, int T, int k, int N, void* d_rows, float* d_w,
                                    cudaStream_t s);

// Products of rows of x with one matrix (offsets NULL) or with each expert's:
// y[o(r)] = W[e(r)] x[i(r)] for the list positions r of every expert. xs NULL: bf16 operands;
// otherwise E4M3 codes with the scales xs [x_rows, ceil(K/128)], ws [E, ceil(N/128), ceil(K/128)].
struct RowsProduct {
    const void* x;           // [x_rows, K]
    const float* xs;
    const void* w;           // [E, N, K]
    const float* ws;
    void* y;                 // [R, N] bf16, or fp32 where y_f32
    const int32_t* offsets;  // [E + 1] or NULL
    const int32_t* list;     // [R] entries t*k + j, or NULL
    int R, x_rows, E, N, K, k;
    int gather, scatter, y_f32;
};

// The same of NVFP4 rows and matrices: x [x_rows, K/2] with xs [x_rows, K/16] and xr [x_rows], w [E, N, K/2] with
// ws [E, N, K/16] and wt [E, parts].
struct Fp4Product {
    RowsProduct r;           // its xs and ws unused
    const uint8_t* xs;
    const float* xr;
    const uint8_t* ws;
    const float* wt;
    int parts;
};
// Up to kStreamRows rows in all, of up to kStreamBytes4 of codes: weights streamed through warp-level MMAs; otherwise
// tcgen05 tiles. Device us, stream / tiles, weights that are not in the L2: one row of 8192 x 2048 (8 MiB) 5.1 / 7.7,
// 2048 x 8192 6.3 / 7.9, 1024 x 512 3.2 / 4.8; 8 rows of 8192 x 2048 5.8 / 7.5; 8 experts of 1024 x 2048 with a row each
// 6.2 / 8.3; but 16384 x 2048 (16 MiB) with one row 9.2 / 9.2, with eight 9.5 / 8.1, and one row of 248320 x 2048
// (243 MiB) 80 / 59: expanding codes to f16 costs the streaming kernel 3.6 TB/s.
constexpr long long kStreamBytes4 = 12ll << 20;
cudaError_t launch_fp4_stream(const Fp4Product& P, const DeviceInfo& dev, cudaStream_t s);
cudaError_t launch_rows_fp4(const Fp4Product& P, WsHeader* hdr, const DeviceInfo& dev, uint64_t wait_limit,
                            cudaStream_t s);

// Row of x and of y of list position r; -1 for an entry outside [0, R).
__device__ __forceinline__ int x_row(const RowsProduct& P, int r) {
    if (!P.gather) return r;
    const int entry = P.list[r];
    return (unsigned)entry < (unsigned)P.R ? entry / P.k : -1;
}
__device__ __forceinline__ int y_row(const RowsProduct& P, int r) {
    if (!P.scatter) return r;
    const int entry = P.list[r];
    return (unsigned)entry < (unsigned)P.R ? entry : -1;
}

// Up to kStreamRows rows in all: weights streamed through warp-level MMAs; more: tcgen05 tiles. Measured on
// a GB300 with weights that are not in the L2 (us on the device, stream / tiles): 8192 x 2048 in 8 bits at 8 rows
// 5.8 / 8.3, at 16 rows (two blocks of columns in the streaming kernel) 9.4 / 8.4; 2048 x 8192 at 8 rows 7.2 / 9.6,
// at 16 rows 10.2 / 9.6; 8 bf16 experts of 1024 x 2048 with a row each 8.1 / 10.3, 8192 x 2048 in bf16 at 16 rows
// 12.5 / 10.4.
// Large 8-bit matrices go to the tiles even so, because the streaming kernel's conversions bound it (one row
// of K = 2048: 33 MB of W 9.1 / 9.8, 67 MB 15.2 / 14.7, 508 MB 93 / 80).
constexpr int kStreamRows = 8;
constexpr long long kStreamBytes8 = 48ll << 20;
cudaError_t launch_rows_stream(const RowsProduct& P, const DeviceInfo& dev, cudaStream_t s);
cudaError_t launch_rows_tc(const RowsProduct& P, WsHeader* hdr, const DeviceInfo& dev, uint64_t wait_limit,
                           cudaStream_t s);

}  // namespace nvfp4
