// internal.h -- launchers shared between the C-ABI layer (api.cu) and the
// kernel files. Every launcher enqueues on `stream` and returns the CUDA
// error of the launch (cudaSuccess when nothing was launched).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "lora.h"

namespace lora {

// Kernel files expose these; arguments are validated by api.cu.
cudaError_t launch_build_segments(const int32_t* ids, int T, int n_adapters,
                                  const lora_segments_t& seg, cudaStream_t stream);

enum SgmvMode { SGMV_SHRINK = 0, SGMV_EXPAND = 1, SGMV_APPLY = 2 };

// x, v, y may be NULL where the mode does not use them. order: NULL, or
// sgmv_order_bytes(T, n_adapters) bytes of device memory (16-byte aligned) into which
// a small kernel first writes the tile rows in descending cost, which the SGMV
// kernel then walks (long rows first, no tail of a few long CTAs).
cudaError_t launch_sgmv(int mode, const void* x, int64_t x_slice_stride, const lora_pool_t& pool,
                        const lora_segments_t& seg, float* v, void* y, cudaStream_t stream,
                        bool pdl_trigger, void* order = nullptr);
size_t sgmv_order_bytes(int T, int n_adapters);
// The expand on the tcgen05 tensor cores (sgmv_tc.cu) for batches of long segments:
// whether a batch qualifies, and the launch (v fp32 [n_slices][T][r_max], y in place).
// v may come as v_parts planes of [n_slices][T][r_max] (the shrink below) that the
// expand sums in plane order.
bool sgmv_expand_tc_eligible(int T, const lora_pool_t& pool);
cudaError_t launch_sgmv_expand_tc(const float* v, int v_parts, const lora_pool_t& pool, const lora_segments_t& seg,
                                  void* y, cudaStream_t stream);
// The shrink on the tensor cores for the same batches, into `parts` planes of v (at most
// sgmv_shrink_tc_parts(pool)); cudaErrorInvalidValue if the pool's tensor map is refused.
int sgmv_shrink_tc_parts(const lora_pool_t& pool);
cudaError_t launch_sgmv_shrink_tc(const void* x, int64_t x_slice_stride, const lora_pool_t& pool,
                                  const lora_segments_t& seg, float* v, int parts, cudaStream_t stream);

// Token-wise merge of the selected adapters into the backbone (merge.cu).
cudaError_t launch_lora_switch_merge(const void* W, int N, int K, const lora_pool_t& pool, const int32_t* sel,
                                     const float* gates, int n_sel, void* W_out, cudaStream_t stream);

// Adapter gradients (grad.cu): the transposed pool (A'_a = B_a^T [N][r_max],
// B'_a = A_a^T [r_max][K]) of the active adapters, and the segmented outer
// products dA_a = s_a x_a^T u_a ([K][r_max], row_major_long) or
// dB_a = s_a v_a^T dY_a ([r_max][N]) of the active adapters.
cudaError_t launch_transpose_pool(const lora_pool_t& pool, const lora_segments_t& seg, void* At, void* Bt,
                                  cudaStream_t stream);
// u[perm[pos]][j] = sum over the v_rep copies of vg[c][pos][j] (the fused GEMM's
// down-projection, segment order) for every position with an adapter (grad.cu).
cudaError_t launch_gather_u(const float* vg, int v_rep, const lora_segments_t& seg, int M, int r_max, float* u,
                            cudaStream_t stream);
cudaError_t launch_grad_outer(bool row_major_long, const void* lng, const float* shrt, int L,
                              const lora_pool_t& pool, const lora_segments_t& seg, float* out, cudaStream_t stream);

// Per-row E4M3 quantisation; row p of the output is row perm[p] of x
// (perm == NULL: identity). The kernel also zeroes zero_words 32-bit words at
// `zero` (may be NULL) and lets a programmatic dependent launch start early.
// copy_bf16: the rows are copied as bf16 instead (xq holds M * K bf16) and sx = 1.
cudaError_t launch_quantize_rows(const void* x, const int32_t* perm, int M, int K, uint8_t* xq,
                                 float* sx, void* zero, size_t zero_words, cudaStream_t stream,
                                 bool copy_bf16 = false);

// OCP MX FP4 quantisation of W bf16 [N][K] (K % 64 == 0): Wp [N][K / 2] packed
// E2M1 codes (element 2i in the low nibble), Wsc E8M0 [ceil(N / 128)][K / 32][128].
cudaError_t launch_mxfp4_quantize(const void* W, int N, int K, uint8_t* Wp, uint8_t* Wsc, cudaStream_t stream);

// 8-bit activation checkpoints (act8.cu): M rows of N bf16 compressed and expanded again.
cudaError_t launch_act8_compress(const void* x, int M, int N, const lora_act8_t& out, cudaStream_t stream);
cudaError_t launch_act8_expand(const lora_act8_t& in, int M, int N, void* x, cudaStream_t stream);

// The gated feed-forward block's GEMM for given sizes: its tiles, and whether its rows are the tokens in the
// segments' order (with a pool; gated.cu says when).
struct GatedPlan {
    bool pair, by_adapter;
    int cols, mt, tiles, units;
    int split;  // pieces of the last round's tiles, 1: they stay whole
    int whole() const { return split > 1 ? tiles / units * units : tiles; }  // tiles before the shared ones
};
GatedPlan gated_plan(bool backward, int M, int K, int F, bool save, const lora_pool_t* pool);
// launch_gated_operands turns the planes of v [2][M][r_max] of each side into the bf16 operands of s_a v (backward:
// gated_operand_bytes, [2][M][hi r16 | lo r16]; forward, one side: gated_expand_bytes, the GEMM's steps, see
// expand_kernel) and lists the rank blocks of each token tile of the GEMM that follows (gated_list_bytes).
// With adapters the launches right before launch_gated_gemm are a shrink that waits for its predecessors
// before it lets its dependents start, then launch_gated_operands (gated.cu says why).
// launch_gated_shrink, for each of n sides: gated_shrink_planes planes of v[s][t][j] = sum_l
// lng[s][t][l] w, w = pool.A[s][a][l][j] (down: x.A) or pool.B[s][a][j][l] (else: d.B^T), lng_slice
// 0: both slices read one lng (gated_grad.cu).
struct GatedSide {
    bool down;
    const void* lng;
    int64_t lng_slice;
    bool by_adapter;  // lng's rows are in the segments' order
    float* v;
    void* ops;  // where launch_gated_operands puts the side's operands
};
int gated_shrink_planes(int M, int L, int n_adapters);
// Also marks the adapters whose matrix in the GEMM to come (forward B, backward A) holds a
// non-finite value: bad[slice][adapter][part], gated_scan_parts parts (gated_bad_bytes).
constexpr int kGatedScanMax = 32;
int gated_scan_parts(bool down, int M, const lora_pool_t& pool);
size_t gated_bad_bytes(const lora_pool_t& pool);
cudaError_t launch_gated_shrink(const GatedSide* sides, int n, int M, const lora_pool_t& pool, const lora_segments_t& seg,
                                uint8_t* bad, cudaStream_t stream);
// Forward: the rows of x that the GEMM reads in the segments' order (gated.cu), before the shrink.
size_t gated_gather_bytes(int M, int K);
cudaError_t launch_gated_gather(const GatedPlan& plan, const void* x, int M, int K, const lora_segments_t& seg, void* out,
                                cudaStream_t stream);
size_t gated_operand_bytes(int M, int r_max);
size_t gated_expand_bytes(int M, int n_adapters, int r_max);
size_t gated_list_bytes(int M);
size_t gated_part_bytes();
size_t gated_count_bytes();
cudaError_t launch_gated_operands(const GatedPlan& plan, const GatedSide* sides, int n, int M, const lora_pool_t& pool,
                                  const lora_segments_t& seg, const uint8_t* bad, bool backward, void* lists, cudaStream_t stream);
struct GatedGemmArgs {
    bool backward;
    int M, K, F, act;
    const void* a[2];       // forward: x, with adapters launch_gated_gather's rows; backward: dg, du [M][F]
    const void* W[2];       // Wg, Wu [F][K]
    void* out;              // h [M][F]; backward: dX [M][K]
    const lora_act8_t* g8;  // forward: both or neither
    const lora_act8_t* u8;
    uint32_t* status;
    float* part;            // backward: gated_part_bytes
    int* count;             // backward: gated_count_bytes, zeroed by launch_gated_point
    bool lora;
    const void* ops;
    const void* lists;
    const void* B;          // the pool's B, backward: its A
    const int32_t *tok_adapter, *order;  // the segments' tok_adapter and perm
    int n_adapters, r_max;
};
// cudaErrorInvalidValue if an operand's tensor map is refused.
cudaError_t launch_gated_gemm(const GatedPlan& plan, const GatedGemmArgs& a, cudaStream_t stream);
// dg, du (and h, may be NULL) from dh and the checkpoints of g and u (gated_grad.cu). Also zeroes `count`
// (gated_count_bytes). order: NULL, or the tokens of dg's and du's rows.
cudaError_t launch_gated_point(const void* dh, int M, int F, int act, const lora_act8_t& g8, const lora_act8_t& u8,
                               const int32_t* order, void* dg, void* du, void* h, int* count, cudaStream_t stream);
// Gradients of both slices, bf16: dA[s][a][k][j] = sum_t x[t][k] op_u[s][t][j] and dB[s][a][j][f] =
// sum_t op_v[s][t][j] d[s][t][f] over the adapter's tokens. by_adapter: the plan's (the rows of d and of the
// operands).
cudaError_t launch_gated_outer(const void* x, const void* ops_u, void* dA, const void* d, const void* ops_v, void* dB, int M,
                               const lora_pool_t& pool, const lora_segments_t& seg, bool by_adapter, cudaStream_t stream);

struct Fp8GemmArgs {
    int M, N, K;
    int esz;             // operand element bytes: 1 = E4M3 (kind::f8f6f4), 2 = bf16 (kind::f16)
    const uint8_t* xq;   // e4m3 (or bf16) [M][K], rows in perm order
    const float* sx;     // [M], perm order (1 for bf16 operands)
    const uint8_t* Wq;   // e4m3 (or bf16) [N][K]
    const float* sw;     // [N]; NULL = 1 (bf16 weights carry no scale)
    const uint8_t* wsc;  // MX FP4 weights (esz 2): Wq holds the packed E2M1 codes
                         // [N][K / 2] and wsc the E8M0 scales [ceil(N / 128)][K / 32][128]
    bool w_e4m3;         // esz 2 with E4M3 weight codes (W8A16): converted to bf16 on chip
    uint16_t* y;         // bf16 [M][N]
    uint32_t* status;    // device status word
    float* partials;     // fp32 [SMs][128][fp8_gemm_tile_n(M)] stream-K partials
    int* flags;          // [SMs], zero on entry
    int* v_done;         // zero on entry
    // LoRA epilogue (lora == false: base only)
    bool lora;
    const uint16_t* x;          // bf16 [M][K], by token index (the down-projection's input)
    const uint16_t* A;          // bf16 [n_adapters][K][r_max]
    const int32_t* perm;        // [M]
    const int32_t* tok_adapter; // [M]
    const int32_t* indptr;      // [n_adapters+1]
    const int32_t* active;      // [n_adapters]
    const int32_t* counts;      // [4]
    float* v;                   // fp32 [M][r_max], segment order, zero on entry
    const uint16_t* B;          // bf16 [n_adapters][r_max][N]
    const int32_t* ranks;
    const float* scales;
    int n_adapters, r_max;
};
// Launched as a programmatic dependent of the previous kernel (the quantiser).
cudaError_t launch_fp8_gemm(const Fp8GemmArgs& a, cudaStream_t stream);
// Token columns of a GEMM tile for M tokens, and the bytes of partial sums.
int fp8_gemm_tile_n(int M);
size_t fp8_gemm_partial_bytes(int M);
// copies of the down-projection v the fused GEMM spreads its atomics over (a power of two)
int fp8_gemm_v_copies(int M);

int device_sm_count();

// Limit of the kernels' bounded waits (2 s unless a test lowered it with
// lora_debug_set_wait_limit) and the test hook that makes one CTA wait on a
// barrier that nothing completes.
unsigned long long debug_wait_limit_ns();
int debug_inject_stall();

// Rows of lora_segments_t.tiles for T tokens over n_adapters.
int max_tiles_for(int T, int n_adapters);
// tokens per tile for a batch (LORA_DECODE_TILE_TOKENS for decode-like batches)
int tile_tokens_for(int T, int n_adapters);

// 2-D tiled tensor map (inner dimension contiguous); false on failure.
bool encode_tmap_2d(CUtensorMap* m, CUtensorMapDataType dt, const void* base, uint64_t inner,
                    uint64_t outer, uint64_t row_stride_bytes, uint32_t box_inner,
                    uint32_t box_outer, CUtensorMapSwizzle swz);

// 3-D tiled tensor map: dims innermost first, strides (bytes) of dims 1 and 2;
// out-of-range box elements are filled with zeros. false on failure.
bool encode_tmap_3d(CUtensorMap* m, CUtensorMapDataType dt, const void* base, const uint64_t dims[3],
                    const uint64_t strides_bytes[2], const uint32_t box[3], CUtensorMapSwizzle swz);

// fp8_gemm_lora_epilogue's argument checks, workspace aside (a lora_status_t).
int fp8_gemm_check_args(const void* x, int M, int K, int N, const uint8_t* Wq, const float* w_scale,
                        const lora_pool_t* pool, const lora_segments_t* seg, const void* y);

// Slot of the device status word in lora_segments_t.counts.
constexpr int kSegStatusSlot = 4;
// status bit: a tile held more tokens than the segments' tile size allows
constexpr int kSegTooLarge = 0x1000;

}  // namespace lora
