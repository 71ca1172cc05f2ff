// gated_grad.cu -- the gated feed-forward block around its matrix products (gated.cu): the
// backward's element-wise part, read from the 8-bit checkpoints, the shrinks of both directions
// and the adapters' gradients.
//
//   dg = dh u act'(g),  du = dh act(g),  h = act(g) u          (g, u: act8.cuh)
//   dA_s,a = x_a^T (s_a d_s B_s,a^T),  dB_s,a = (s_a x A_s,a)_a^T d_s
//                                       (s = 0: gate, d = dg; s = 1: up, d = du)
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "act8.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "sgmv_common.cuh"

namespace lora {
namespace {

// ------------------------------------------------------------------ element-wise part
//
// Bound by HBM: per element 2 bytes of dh and 2 1/16 of checkpoints in, 4 bytes out (6 with
// h). dg and du are rounded to bf16, as the product's operands have to be. A warp takes 256
// columns of a row at a time, 8 per lane, two such tasks in flight.

constexpr int kEThreads = 256;
constexpr int kEWarps = kEThreads / 32;
constexpr int kETaskCols = 256;
constexpr int kEInFlight = 2;

struct PointParams {
    const uint16_t* dh;
    const uint8_t *g_codes, *g_scales, *u_codes, *u_scales;
    uint16_t *dg, *du, *h;
    const int32_t* order;  // dg's and du's rows are these tokens (NULL: the tokens as they come)
    int* count;  // count_words words to zero
    int count_words, F;
    uint32_t tasks, segs;
};

// act(g) and act'(g); the sigmoid of exp(-|g|), whose denominator stays within 2 (see gate in gated.cu).
template <int ACT>
__device__ __forceinline__ void act_and_slope(float g, float& a, float& d)
{
    if (ACT == LORA_ACT_SILU) {
        const float t = __expf(-fabsf(g)), big = __fdividef(1.f, 1.f + t), small = t * big;
        const float s = g < 0.f ? small : big, rest = g < 0.f ? big : small;  // 1 - s
        a = g * s;
        d = s * fmaf(g, rest, 1.f);
    } else {
        const float cdf = 0.5f * erfcf(g * -0.70710678118654752f);
        a = g * cdf;
        d = fmaf(g * 0.3989422804014327f, __expf(-0.5f * g * g), cdf);
    }
}

template <int ACT, bool H, bool ORDER>
__global__ void __launch_bounds__(kEThreads)
gated_point_kernel(const PointParams p)
{
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    if (blockIdx.x == 0 && (int)threadIdx.x < p.count_words) p.count[threadIdx.x] = 0;
    const int lane = threadIdx.x & 31;
    const uint32_t stride = gridDim.x * kEWarps, nb = (uint32_t)((p.F + act8::kBlock - 1) / act8::kBlock);
    for (uint64_t t0 = blockIdx.x * kEWarps + (threadIdx.x >> 5); t0 < p.tasks; t0 += (uint64_t)stride * kEInFlight) {
        uint4 dh[kEInFlight];
        uint2 gc[kEInFlight], uc[kEInFlight];
        uint32_t gE[kEInFlight], uE[kEInFlight];
        size_t at[kEInFlight], to[kEInFlight];
        bool live[kEInFlight];
#pragma unroll
        for (int i = 0; i < kEInFlight; ++i) {
            const uint64_t t = t0 + (uint64_t)i * stride;
            live[i] = false;
            if (t < p.tasks) {
                const uint32_t row = (uint32_t)t / p.segs;
                const int col = (int)((uint32_t)t - row * p.segs) * kETaskCols + lane * 8;
                if (col < p.F) {
                    live[i] = true;
                    const uint32_t tok = ORDER ? (uint32_t)p.order[row] : row;
                    to[i] = (size_t)row * p.F + col;
                    at[i] = (size_t)tok * p.F + col;
                    const size_t sc = (size_t)tok * nb + (col >> 5);
                    dh[i] = __ldcs(reinterpret_cast<const uint4*>(p.dh + at[i]));
                    gc[i] = __ldcs(reinterpret_cast<const uint2*>(p.g_codes + at[i]));
                    uc[i] = __ldcs(reinterpret_cast<const uint2*>(p.u_codes + at[i]));
                    gE[i] = p.g_scales[sc];
                    uE[i] = p.u_scales[sc];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kEInFlight; ++i) {
            if (!live[i]) continue;
            const float gX = act8::scale_value(gE[i]), uX = act8::scale_value(uE[i]);
            const uint32_t w[4] = {dh[i].x, dh[i].y, dh[i].z, dh[i].w};
            uint32_t og[4], ou[4], oh[4];
            float gv[8], uv[8];
            act8::decode4(gc[i].x, gv);
            act8::decode4(gc[i].y, gv + 4);
            act8::decode4(uc[i].x, uv);
            act8::decode4(uc[i].y, uv + 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float a[2], d[2], u[2];
                const float dy[2] = {bf16_lo(w[e]), bf16_hi(w[e])};
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    act_and_slope<ACT>(gv[2 * e + k] * gX, a[k], d[k]);
                    u[k] = uv[2 * e + k] * uX;
                }
                og[e] = pack_bf16x2(dy[0] * u[0] * d[0], dy[1] * u[1] * d[1]);
                ou[e] = pack_bf16x2(dy[0] * a[0], dy[1] * a[1]);
                oh[e] = pack_bf16x2(a[0] * u[0], a[1] * u[1]);
            }
            *reinterpret_cast<uint4*>(p.dg + to[i]) = make_uint4(og[0], og[1], og[2], og[3]);
            *reinterpret_cast<uint4*>(p.du + to[i]) = make_uint4(ou[0], ou[1], ou[2], ou[3]);
            if (H) *reinterpret_cast<uint4*>(p.h + at[i]) = make_uint4(oh[0], oh[1], oh[2], oh[3]);
        }
    }
}

// ------------------------------------------------------------------ adapters' gradients
//
// A segmented sum of outer products over an adapter's tokens: G[l][j] = sum_t lng[t][l] op[t][j],
// lng = x (dA, l along K) or d_s (dB, l along F), op = the bf16 halves hi + lo of s_a u or
// s_a v that operand_kernel wrote (16 bits). On mma.sync m16n8k16: the tensor work is
// 2 r times the long elements, small beside reading them, so HBM bounds it. A CTA owns 64
// values of l of one adapter and slice and walks the adapter's tokens 64 at a time, gathered
// by cp.async into three stages; both operands come out of [token][value] rows by transposing
// ldmatrix. Sums run in token order: the result does not depend on the grid. Adapters without
// tokens get zeros.

constexpr int kOThreads = 128;
constexpr int kOTok = 64;    // tokens per step (shrink: of a CTA)
constexpr int kOL = 64;
constexpr int kOStages = 3;

struct OuterSide {
    const uint16_t* lng;
    long long lng_slice;
    const uint16_t* ops;  // [2][M][hi r16 | lo r16]
    uint16_t* out;        // dA [2][n][L][r_max] or dB [2][n][r_max][L]
    int L;
};
struct OuterParams {
    OuterSide a, b;  // dA, dB
    int a_blocks;    // CTAs of dA along the grid's x, then those of dB
    int run;         // blocks of 64 l that a CTA does one after the other
    const int32_t* perm;
    const int32_t* indptr;
    const int32_t* ranks;
    int M, n_adapters, r_max;
};

// Byte offset of 16-byte chunk c of row t, rows of CH chunks, laid out so that eight
// consecutive rows' chunks c fall on different banks.
template <int CH>
__device__ __forceinline__ uint32_t o_chunk(int t, int c)
{
    if (CH == 2) return (uint32_t)(t * 32 + ((c ^ ((t >> 2) & 1)) << 4));
    if (CH == 4) return (uint32_t)(t * 64 + ((c ^ ((t >> 1) & 3)) << 4));
    return (uint32_t)(t * CH * 16 + ((c ^ (t & 7)) << 4));
}

// T tokens per step. LONG: dA's side. BY_ADAPTER: the operands' rows and d's are in the segments' order.
// (Where the rows lie is fixed at compile time: 2704 tokens of 8 adapters of rank 64 take 104 us so, 169
// with every row looked up, 214 with rows that depend on the side at run time.)
template <int R16, int T, bool LONG, bool BY_ADAPTER>
__device__ __forceinline__ void outer_sums(const OuterParams& p)
{
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr int kOpCh = R16 / 4;               // 16-byte chunks of an operand row (hi and lo)
    constexpr int kLngBytes = T * kOL * 2, kOpBytes = T * kOpCh * 16, kStage = kLngBytes + kOpBytes;
    constexpr int NT = R16 / 8;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const OuterSide& d = LONG ? p.a : p.b;
    const int lb0 = ((int)blockIdx.x - (LONG ? 0 : p.a_blocks)) * p.run, a = (int)blockIdx.y, s = (int)blockIdx.z;
    const int blocks = min(p.run, (d.L + kOL - 1) / kOL - lb0);
    const int t0 = p.indptr[a], n_tok = p.indptr[a + 1] - t0;
    const int r = max(1, min(p.ranks ? p.ranks[a] : p.r_max, p.r_max));
    const uint16_t* lng = d.lng + (size_t)s * d.lng_slice;
    const uint16_t* ops = d.ops + (size_t)s * p.M * (2 * R16);
    // rows of the segments' positions
    const int32_t* perm = p.perm + t0;
    auto l_row = [&](int t) { return (size_t)(LONG || !BY_ADAPTER ? perm[t] : t0 + t); };
    auto op_row = [&](int t) { return (size_t)(BY_ADAPTER ? t0 + t : perm[t]); };
    const uint32_t base = ptx::smem_u32(smem);
    const int steps = (n_tok + T - 1) / T;
    const int i8 = lane >> 3, rr = lane & 7;

    float acc[NT][4];
    auto clear = [&]() {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
    };
    // The block's 64 x r_max values, rounded once to the adapters' type (past the rank zero), through
    // shared memory to whole 16-byte pieces of the gradient.
    auto finish = [&](int l0) {
        uint16_t* o = reinterpret_cast<uint16_t*>(smem + kOStages * kStage);
        const int g = lane >> 2, q = lane & 3;
        constexpr int kPitchA = R16 + 8, kPitchB = kOL + 8;
        __syncthreads();  // the previous block's values are out
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int j = n * 8 + q * 2;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int l = warp * 16 + g + h * 8;
                const uint32_t v = pack_bf16x2(j < r ? acc[n][2 * h] : 0.f, j + 1 < r ? acc[n][2 * h + 1] : 0.f);
                if (LONG) {
                    *reinterpret_cast<uint32_t*>(o + l * kPitchA + j) = v;
                } else {
                    o[j * kPitchB + l] = (uint16_t)(v & 0xffffu);
                    o[(j + 1) * kPitchB + l] = (uint16_t)(v >> 16);
                }
            }
        }
        __syncthreads();
        if (LONG) {  // [64][r_max], one run of memory
            const int pieces = p.r_max >> 3, lg = __ffs(pieces) - 1;
            uint16_t* out = d.out + (((size_t)s * p.n_adapters + a) * d.L + l0) * p.r_max;
            for (int idx = tid; idx < kOL * pieces; idx += kOThreads) {
                const int l = idx >> lg, c = idx & (pieces - 1);
                if (l0 + l < d.L) *reinterpret_cast<uint4*>(out + idx * 8) = *reinterpret_cast<const uint4*>(o + l * kPitchA + c * 8);
            }
        } else {
            for (int idx = tid; idx < p.r_max * (kOL / 8); idx += kOThreads) {
                const int j = idx >> 3, c = idx & 7, l = l0 + c * 8;
                if (l < d.L)
                    *reinterpret_cast<uint4*>(d.out + (((size_t)s * p.n_adapters + a) * p.r_max + j) * d.L + l) =
                        *reinterpret_cast<const uint4*>(o + j * kPitchB + c * 8);
            }
        }
    };

    if (steps <= 1) {
        // All tokens in one step: the operands stay in registers, the blocks' rows stream by.
        const uint16_t* rows[T * 8 / kOThreads];
#pragma unroll
        for (int i = 0; i < T * 8 / kOThreads; ++i) {
            const int t = (tid >> 3) + i * (kOThreads / 8);
            rows[i] = t < n_tok ? lng + l_row(t) * d.L + (tid & 7) * 8 : nullptr;
        }
        auto fetch = [&](int b) {
            if (b < blocks) {
                const uint32_t st = base + (uint32_t)((b % kOStages) * kStage);
                const int l0 = (lb0 + b) * kOL;
#pragma unroll
                for (int i = 0; i < T * 8 / kOThreads; ++i) {
                    const bool in = rows[i] && l0 + (tid & 7) * 8 < d.L;
                    ptx::cp_async16(st + o_chunk<8>((tid >> 3) + i * (kOThreads / 8), tid & 7), in ? rows[i] + l0 : lng, in ? 16 : 0);
                }
            }
            ptx::cp_async_commit();
        };
#pragma unroll
        for (int i = 0; i < T * kOpCh / kOThreads; ++i) {
            const int idx = tid + i * kOThreads, t = idx / kOpCh, c = idx % kOpCh;
            const bool in = t < n_tok;
            const uint16_t* src = in ? ops + op_row(t) * (2 * R16) + c * 8 : ops;
            ptx::cp_async16(base + kLngBytes + o_chunk<kOpCh>(t, c), src, in ? 16 : 0);
        }
        for (int k = 0; k < kOStages - 1; ++k) fetch(k);
        uint32_t bf[T / 16][2][NT][2];
        for (int b = 0; b < blocks; ++b) {
            ptx::cp_async_wait<kOStages - 2>();
            __syncthreads();  // the block's rows are here, and the previous one's are consumed
            fetch(b + kOStages - 1);
            if (b == 0)
#pragma unroll
                for (int ks = 0; ks < T / 16; ++ks)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int n = 0; n < NT; n += 2)
                            ptx::ldsm_x4_t(base + kLngBytes + o_chunk<kOpCh>(ks * 16 + (i8 & 1) * 8 + rr, h * NT + n + (i8 >> 1)),
                                           bf[ks][h][n][0], bf[ks][h][n][1], bf[ks][h][n + 1][0], bf[ks][h][n + 1][1]);
            clear();
            const uint32_t st = base + (uint32_t)((b % kOStages) * kStage);
#pragma unroll
            for (int ks = 0; ks < T / 16; ++ks) {
                if (ks * 16 >= n_tok) break;
                uint32_t A[4];
                ptx::ldsm_x4_t(st + o_chunk<8>(ks * 16 + (i8 >> 1) * 8 + rr, warp * 2 + (i8 & 1)), A[0], A[1], A[2], A[3]);
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int n = 0; n < NT; ++n) ptx::mma_bf16_16816(acc[n], A, bf[ks][h][n][0], bf[ks][h][n][1]);
            }
            finish((lb0 + b) * kOL);
        }
        ptx::cp_async_wait<0>();
        return;
    }

    for (int b = 0; b < blocks; ++b) {
        const int l0 = (lb0 + b) * kOL;
        auto fetch = [&](int step) {
            if (step < steps) {
                const uint32_t st = base + (uint32_t)((step % kOStages) * kStage);
#pragma unroll
                for (int i = 0; i < T * (kOL / 8) / kOThreads; ++i) {
                    const int idx = tid + i * kOThreads, t = idx >> 3, c = idx & 7, pos = step * T + t;
                    const bool in = pos < n_tok && l0 + c * 8 < d.L;
                    const uint16_t* src = in ? lng + l_row(pos) * d.L + l0 + c * 8 : lng;
                    ptx::cp_async16(st + o_chunk<8>(t, c), src, in ? 16 : 0);
                }
#pragma unroll
                for (int i = 0; i < T * kOpCh / kOThreads; ++i) {
                    const int idx = tid + i * kOThreads, t = idx / kOpCh, c = idx % kOpCh, pos = step * T + t;
                    const bool in = pos < n_tok;
                    const uint16_t* src = in ? ops + op_row(pos) * (2 * R16) + c * 8 : ops;
                    ptx::cp_async16(st + kLngBytes + o_chunk<kOpCh>(t, c), src, in ? 16 : 0);
                }
            }
            ptx::cp_async_commit();
        };
        __syncthreads();  // the previous block's rows are consumed
        clear();
        for (int k = 0; k < kOStages - 1; ++k) fetch(k);
        for (int step = 0; step < steps; ++step) {
            ptx::cp_async_wait<kOStages - 2>();
            __syncthreads();  // the step's rows are here, and the previous step's are consumed
            fetch(step + kOStages - 1);
            const uint32_t st = base + (uint32_t)((step % kOStages) * kStage), so = st + kLngBytes;
#pragma unroll
            for (int ks = 0; ks < T / 16; ++ks) {
                uint32_t A[4];
                ptx::ldsm_x4_t(st + o_chunk<8>(ks * 16 + (i8 >> 1) * 8 + rr, warp * 2 + (i8 & 1)), A[0], A[1], A[2], A[3]);
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int n = 0; n < NT; n += 2) {
                        uint32_t f[4];
                        ptx::ldsm_x4_t(so + o_chunk<kOpCh>(ks * 16 + (i8 & 1) * 8 + rr, h * NT + n + (i8 >> 1)), f[0], f[1], f[2],
                                       f[3]);
                        ptx::mma_bf16_16816(acc[n], A, f[0], f[1]);
                        ptx::mma_bf16_16816(acc[n + 1], A, f[2], f[3]);
                    }
            }
        }
        finish(l0);
        ptx::cp_async_wait<0>();
    }
}

template <int R16, int T, bool BY_ADAPTER>
__global__ void __launch_bounds__(kOThreads)
gated_outer_kernel(const OuterParams p)
{
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    if ((int)blockIdx.x < p.a_blocks) outer_sums<R16, T, true, BY_ADAPTER>(p);
    else outer_sums<R16, T, false, BY_ADAPTER>(p);
}

// ------------------------------------------------------------------ shrink
//
// v[t][j] = sum_l lng[t][l] w[l][j] for both slices: x.A_a (w's rows are l, as A is stored) and
// d_s.B_a^T (rows are j, as B is stored: no transposed copy of the pool). A CTA takes a tile row of the
// segments (up to 64 tokens of one adapter), a slice and one of `planes` parts of L; the
// parts' sums go to planes of v that operand_kernel adds in order, so no atomics. mma.sync
// m16n8k16: the products are 2 r16 per element of lng, few beside reading it, so HBM bounds it.
// A warp owns 16 tokens; 64 values of l at a time come by cp.async into three stages.

// One side of the sum: x against A (down) or d against B.
struct ShrinkSide {
    const uint16_t* lng;
    long long lng_slice;
    const uint16_t* w;  // A [2][n][L][r_max] or B [2][n][r_max][L]
    float* v;           // [planes][2][M][r_max]
    int L, planes, steps;  // steps of 64 per plane
    bool down;
    bool by_adapter;  // lng's rows are in the segments' order
};
constexpr int kScanPer = 4;  // scanning CTAs per plane
static_assert(8 * kScanPer <= kGatedScanMax, "marks of a scan's parts");
struct ShrinkParams {
    ShrinkSide side[2];
    int sides;
    const int32_t* perm;
    const int32_t* indptr;
    const int4* tiles;
    const int32_t* ranks;
    int M, n_adapters, r_max;
    // the pool's matrices that the GEMM multiplies with (forward B, backward A)
    const uint16_t* scan;
    bool scan_rows;   // their rows are ranks (B)
    int scan_L, scan_parts;
    uint8_t* bad;     // [2][n_adapters][kGatedScanMax]
};

// Whether adapter a's matrix of slice s holds a non-finite value in part `part` of its live elements.
// The GEMM multiplies every row of a token tile with it, most by zero, and zero times infinity would
// carry one tenant's broken adapter into another's tokens; a marked one is kept out of them
// (operand_kernel). The pass also brings the matrices into L2 for the GEMM.
__device__ __forceinline__ void scan_adapter(const ShrinkParams& p, int a, int s, int part)
{
    const int r = max(1, min(p.ranks ? p.ranks[a] : p.r_max, p.r_max));
    const uint4* m = reinterpret_cast<const uint4*>(p.scan + ((size_t)s * p.n_adapters + a) * p.r_max * p.scan_L);
    const int per_row = p.r_max >> 3;  // 16-byte pieces of a row of A
    const long long all = p.scan_rows ? (long long)r * (p.scan_L >> 3) : (long long)p.scan_L * per_row;
    const long long i0 = all * part / p.scan_parts, i1 = all * (part + 1) / p.scan_parts;
    bool odd = false;
    constexpr int kAhead = 8;
    for (long long i = i0 + threadIdx.x; i < i1; i += kAhead * kOThreads) {
        uint4 v[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) v[k] = i + k * kOThreads < i1 ? m[i + k * kOThreads] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
            // elements of this piece that count: rows of A end at the rank
            const int live = p.scan_rows ? 8 : r - (int)((i + k * kOThreads) & (per_row - 1)) * 8;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                odd = odd || (2 * e < live && (w[e] & 0x7f80u) == 0x7f80u) || (2 * e + 1 < live && (w[e] & 0x7f800000u) == 0x7f800000u);
        }
    }
    odd = __syncthreads_or(odd);
    if (threadIdx.x == 0) p.bad[((size_t)s * p.n_adapters + a) * kGatedScanMax + part] = odd;
}

// R16 ranks; DOWN: the rows of w are l.
template <bool DOWN, int R16>
__device__ __forceinline__ void shrink_tile(const ShrinkParams& p, const ShrinkSide& d, uint8_t* smem)
{
    constexpr int kLngBytes = kOTok * 128, kWBytes = R16 * 128, kStage = kLngBytes + kWBytes;
    constexpr int kWCh = DOWN ? R16 / 8 : 8;  // 16-byte pieces of a w row
    constexpr int kWRows = DOWN ? 64 : R16;
    constexpr int kWPer = kWRows * kWCh / kOThreads;  // pieces per thread
    constexpr int NT = R16 / 8;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int plane = (int)blockIdx.y, s = (int)blockIdx.z & 1;
    const int4 tl = p.tiles[blockIdx.x];
    const int a = tl.x, n_tok = min(tl.z, kOTok);
    if (a < 0 || a >= p.n_adapters || n_tok <= 0) return;
    const uint16_t* lng = d.lng + (size_t)s * d.lng_slice;
    const uint16_t* w = d.w + ((size_t)s * p.n_adapters + a) * p.r_max * d.L;
    const uint32_t base = ptx::smem_u32(smem);
    const int k0 = plane * d.steps, k1 = min(k0 + d.steps, (d.L + 63) / 64);
    // this thread's token rows
    const uint16_t* rows[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = (tid >> 3) + 16 * i;
        rows[i] = t < n_tok ? lng + (size_t)(d.by_adapter ? tl.y + t : p.perm[tl.y + t]) * d.L : nullptr;
    }
    auto fetch = [&](int k) {
        if (k < k1) {
            const uint32_t st = base + (uint32_t)((k - k0) % kOStages * kStage);
            const int l0 = k * 64;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = (tid >> 3) + 16 * i, c = tid & 7;
                const bool in = rows[i] && l0 + c * 8 < d.L;
                ptx::cp_async16(st + o_chunk<8>(t, c), in ? rows[i] + l0 + c * 8 : lng, in ? 16 : 0);
            }
#pragma unroll
            for (int i = 0; i < kWPer; ++i) {
                const int idx = tid + i * kOThreads, t = idx / kWCh, c = idx % kWCh;
                const bool in = DOWN ? l0 + t < d.L && c * 8 < p.r_max : t < p.r_max && l0 + c * 8 < d.L;
                const uint16_t* src = DOWN ? w + (size_t)(l0 + t) * p.r_max + c * 8 : w + (size_t)t * d.L + l0 + c * 8;
                ptx::cp_async16(st + kLngBytes + o_chunk<kWCh>(t, c), in ? src : w, in ? 16 : 0);
            }
        }
        ptx::cp_async_commit();
    };
    float acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
    for (int k = 0; k < kOStages - 1; ++k) fetch(k0 + k);
    for (int k = k0; k < k1; ++k) {
        ptx::cp_async_wait<kOStages - 2>();
        __syncthreads();  // the step's rows are here, and the previous step's are consumed
        fetch(k + kOStages - 1);
        if (warp * 16 >= n_tok) continue;
        const uint32_t st = base + (uint32_t)((k - k0) % kOStages * kStage), sw = st + kLngBytes;
        const int i = lane >> 3, rr = lane & 7;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            uint32_t A[4];
            ptx::ldsm_x4(st + o_chunk<8>(warp * 16 + (i & 1) * 8 + rr, ks * 2 + (i >> 1)), A[0], A[1], A[2], A[3]);
#pragma unroll
            for (int n = 0; n < NT; n += 2) {
                uint32_t b[4];
                if (DOWN)
                    ptx::ldsm_x4_t(sw + o_chunk<kWCh>(ks * 16 + (i & 1) * 8 + rr, n + (i >> 1)), b[0], b[1], b[2], b[3]);
                else
                    ptx::ldsm_x4(sw + o_chunk<kWCh>((n + (i >> 1)) * 8 + rr, ks * 2 + (i & 1)), b[0], b[1], b[2], b[3]);
                ptx::mma_bf16_16816(acc[n], A, b[0], b[1]);
                ptx::mma_bf16_16816(acc[n + 1], A, b[2], b[3]);
            }
        }
    }
    ptx::cp_async_wait<0>();
    const int g = lane >> 2, q = lane & 3;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int t = warp * 16 + g + h * 8;
        if (t >= n_tok) continue;
        float* o = d.v + (((size_t)plane * 2 + s) * p.M + p.perm[tl.y + t]) * p.r_max;
#pragma unroll
        for (int n = 0; n < NT; ++n)
            if (n * 8 < p.r_max)
                *reinterpret_cast<float2*>(o + n * 8 + q * 2) = make_float2(acc[n][2 * h], acc[n][2 * h + 1]);
    }
}

// Grid: tile rows x planes x (side or scan, slice).
template <int R16>
__global__ void __launch_bounds__(kOThreads)
gated_shrink_kernel(const ShrinkParams p)
{
    extern __shared__ __align__(128) uint8_t smem[];
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    const int scan = (int)(blockIdx.z >> 1) - p.sides;
    if (scan >= 0) {  // an adapter's first tile scans its matrix
        const int4 tl = p.tiles[blockIdx.x];
        const int planes = p.side[0].planes;
        if (tl.x >= 0 && tl.x < p.n_adapters && tl.z > 0 && p.indptr[tl.x] == tl.y && (int)blockIdx.y < planes)
            scan_adapter(p, tl.x, (int)blockIdx.z & 1, scan * planes + (int)blockIdx.y);
        return;
    }
    const ShrinkSide& d = p.side[blockIdx.z >> 1];
    if ((int)blockIdx.y >= d.planes) return;
    if (d.down) shrink_tile<true, R16>(p, d, smem);
    else shrink_tile<false, R16>(p, d, smem);
}

// The down shrink of a decode-like batch: a CTA takes a token, a slice and a plane's part of
// L; a thread sums eight ranks over every (128 / pieces)-th l, the rows of A_a as they come. Small
// enough (no shared memory to speak of) to run beside the CTAs of the GEMM, whose weights
// stream meanwhile.
__global__ void __launch_bounds__(kOThreads)
gated_shrink_token_kernel(const ShrinkParams p, const int32_t* __restrict__ tok_adapter)
{
    __shared__ float s_sum[kOThreads / 32][LORA_MAX_RANK];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    const int t = (int)blockIdx.x, plane = (int)blockIdx.y, s = (int)blockIdx.z & 1;
    const ShrinkSide& d = p.side[0];
    const int a = tok_adapter[t];
    if (a < 0 || a >= p.n_adapters) return;
    if (blockIdx.z >= 2) {  // an adapter's first token scans its matrix
        if (p.perm[p.indptr[a]] == t) scan_adapter(p, a, s, ((int)(blockIdx.z >> 1) - 1) * (int)gridDim.y + plane);
        return;
    }
    const uint16_t* x = d.lng + (size_t)s * d.lng_slice + (size_t)t * d.L;
    const uint16_t* w = d.w + ((size_t)s * p.n_adapters + a) * p.r_max * d.L;
    const int pieces = p.r_max >> 3, c = tid & (pieces - 1), step = kOThreads / pieces;
    const int l1 = min((plane + 1) * d.steps * 64, d.L);
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    constexpr int kAhead = 8;
    for (int l = plane * d.steps * 64 + tid / pieces; l < l1; l += kAhead * step) {
        uint4 wv[kAhead];
        float xv[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int at = l + i * step;
            wv[i] = make_uint4(0u, 0u, 0u, 0u);
            xv[i] = 0.f;
            if (at < l1) {
                wv[i] = *reinterpret_cast<const uint4*>(w + (size_t)at * p.r_max + c * 8);
                xv[i] = __uint_as_float((uint32_t)x[at] << 16);
            }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const uint32_t u[4] = {wv[i].x, wv[i].y, wv[i].z, wv[i].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                acc[2 * e] = fmaf(xv[i], bf16_lo(u[e]), acc[2 * e]);
                acc[2 * e + 1] = fmaf(xv[i], bf16_hi(u[e]), acc[2 * e + 1]);
            }
        }
    }
    for (int o = 16; o >= pieces; o >>= 1)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += __shfl_xor_sync(0xffffffffu, acc[e], o);
    if (lane < pieces)
#pragma unroll
        for (int e = 0; e < 8; ++e) s_sum[warp][c * 8 + e] = acc[e];
    __syncthreads();
    if (tid < p.r_max) {
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < kOThreads / 32; ++i) v += s_sum[i][tid];
        d.v[(((size_t)plane * 2 + s) * p.M + t) * p.r_max + tid] = v;
    }
}

template <int R16>
cudaError_t launch_shrink(const ShrinkParams& p, int sides, int rows, cudaStream_t stream)
{
    const size_t smem = (size_t)kOStages * (kOTok * 128 + R16 * 128);
    auto kern = gated_shrink_kernel<R16>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const int planes = sides == 2 && p.side[1].planes > p.side[0].planes ? p.side[1].planes : p.side[0].planes;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)rows, (unsigned)planes, (unsigned)(2 * sides + 2 * kScanPer));
    cfg.blockDim = dim3(kOThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int R16, int T, bool BY_ADAPTER>
cudaError_t launch_outer(const OuterParams& p, cudaStream_t stream)
{
    const size_t smem = (size_t)kOStages * (T * kOL * 2 + T * R16 * 4) + (size_t)(R16 + 8) * (kOL + 8) * 2;
    auto kern = gated_outer_kernel<R16, T, BY_ADAPTER>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.a_blocks + ((p.b.L + kOL - 1) / kOL + p.run - 1) / p.run), (unsigned)p.n_adapters, 2);
    cfg.blockDim = dim3(kOThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

// Few tokens per adapter: short steps, whose buffers let more CTAs run on an SM, and several blocks per
// CTA, so that the next block's rows arrive while one is finished.
template <int R16, bool BY_ADAPTER>
cudaError_t launch_outer(OuterParams& p, cudaStream_t stream)
{
    const bool few = p.M <= 32LL * p.n_adapters;
    p.run = few ? 4 : 1;
    p.a_blocks = ((p.a.L + kOL - 1) / kOL + p.run - 1) / p.run;
    return few ? launch_outer<R16, 32, BY_ADAPTER>(p, stream) : launch_outer<R16, 64, BY_ADAPTER>(p, stream);
}
template <int R16>
cudaError_t launch_outer(OuterParams& p, bool by_adapter, cudaStream_t stream)
{
    return by_adapter ? launch_outer<R16, true>(p, stream) : launch_outer<R16, false>(p, stream);
}

template <int ACT, bool H>
cudaError_t launch_point(const cudaLaunchConfig_t& cfg, const PointParams& p)
{
    return p.order ? cudaLaunchKernelEx(&cfg, gated_point_kernel<ACT, H, true>, p) : cudaLaunchKernelEx(&cfg, gated_point_kernel<ACT, H, false>, p);
}

}  // namespace

cudaError_t launch_gated_point(const void* dh, int M, int F, int act, const lora_act8_t& g8, const lora_act8_t& u8,
                               const int32_t* order, void* dg, void* du, void* h, int* count, cudaStream_t stream)
{
    PointParams p = {};
    p.order = order;
    p.count = count;
    p.count_words = (int)(gated_count_bytes() / 4);  // at most a CTA's threads
    p.dh = static_cast<const uint16_t*>(dh);
    p.g_codes = g8.codes;
    p.g_scales = g8.scales;
    p.u_codes = u8.codes;
    p.u_scales = u8.scales;
    p.dg = static_cast<uint16_t*>(dg);
    p.du = static_cast<uint16_t*>(du);
    p.h = static_cast<uint16_t*>(h);
    p.F = F;
    p.segs = (uint32_t)((F + kETaskCols - 1) / kETaskCols);
    p.tasks = (uint32_t)M * p.segs;
    const uint32_t one = (p.tasks + kEWarps - 1) / kEWarps, all = (one + kEInFlight - 1) / kEInFlight;
    const uint32_t fill = (uint32_t)device_sm_count() * 4;  // as in act8.cu
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(one < fill ? one : (all < fill ? fill : all), 1, 1);
    cfg.blockDim = dim3(kEThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (act == LORA_ACT_SILU) return h ? launch_point<LORA_ACT_SILU, true>(cfg, p) : launch_point<LORA_ACT_SILU, false>(cfg, p);
    return h ? launch_point<LORA_ACT_GELU, true>(cfg, p) : launch_point<LORA_ACT_GELU, false>(cfg, p);
}

// Parts of L: about four CTAs per SM, at most eight planes, at least four steps of 64 each.
int gated_shrink_planes(int M, int L, int n_adapters)
{
    const long long ctas = 2LL * max_tiles_for(M, n_adapters), want = 4LL * device_sm_count();
    const long long n = (want + ctas - 1) / ctas, most = (L + 255) / 256;
    const long long planes = n < most ? n : most;
    return (int)(planes < 1 ? 1 : (planes > 8 ? 8 : planes));
}

int gated_scan_parts(bool down, int M, const lora_pool_t& pool)
{
    return kScanPer * gated_shrink_planes(M, down ? pool.h_in : pool.h_out, pool.n_adapters);
}
size_t gated_bad_bytes(const lora_pool_t& pool) { return (size_t)2 * pool.n_adapters * kGatedScanMax; }

cudaError_t launch_gated_shrink(const GatedSide* sides, int n, int M, const lora_pool_t& pool, const lora_segments_t& seg,
                                uint8_t* bad, cudaStream_t stream)
{
    ShrinkParams p = {};
    p.sides = n;
    p.scan_rows = sides[0].down;
    p.scan = static_cast<const uint16_t*>(p.scan_rows ? pool.B : pool.A);
    p.scan_L = p.scan_rows ? pool.h_out : pool.h_in;
    p.scan_parts = gated_scan_parts(sides[0].down, M, pool);
    p.bad = bad;
    p.indptr = seg.indptr;
    p.ranks = pool.ranks;
    for (int i = 0; i < n; ++i) {
        ShrinkSide& d = p.side[i];
        d.down = sides[i].down;
        d.by_adapter = sides[i].by_adapter;
        d.lng = static_cast<const uint16_t*>(sides[i].lng);
        d.lng_slice = sides[i].lng_slice;
        d.w = static_cast<const uint16_t*>(d.down ? pool.A : pool.B);
        d.v = sides[i].v;
        d.L = d.down ? pool.h_in : pool.h_out;
        d.planes = gated_shrink_planes(M, d.L, pool.n_adapters);
        d.steps = ((d.L + 63) / 64 + d.planes - 1) / d.planes;
    }
    p.perm = seg.perm;
    p.tiles = reinterpret_cast<const int4*>(seg.tiles);
    p.M = M;
    p.n_adapters = pool.n_adapters;
    p.r_max = pool.r_max;
    if (n == 1 && sides[0].down && tile_tokens_for(M, pool.n_adapters) <= LORA_DECODE_TILE_TOKENS) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)M, (unsigned)p.side[0].planes, 2 + 2 * kScanPer);
        cfg.blockDim = dim3(kOThreads, 1, 1);
        cfg.stream = stream;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, gated_shrink_token_kernel, p, (const int32_t*)seg.tok_adapter);
    }
    const int rows = max_tiles_for(M, pool.n_adapters);
    if (pool.r_max <= 16) return launch_shrink<16>(p, n, rows, stream);
    if (pool.r_max == 32) return launch_shrink<32>(p, n, rows, stream);
    return launch_shrink<64>(p, n, rows, stream);
}

cudaError_t launch_gated_outer(const void* x, const void* ops_u, void* dA, const void* d, const void* ops_v, void* dB, int M,
                               const lora_pool_t& pool, const lora_segments_t& seg, bool by_adapter, cudaStream_t stream)
{
    OuterParams p = {};
    p.perm = seg.perm;
    p.a.lng = static_cast<const uint16_t*>(x);
    p.a.ops = static_cast<const uint16_t*>(ops_u);
    p.a.out = static_cast<uint16_t*>(dA);
    p.a.L = pool.h_in;
    p.b.lng = static_cast<const uint16_t*>(d);
    p.b.lng_slice = (long long)M * pool.h_out;
    p.b.ops = static_cast<const uint16_t*>(ops_v);
    p.b.out = static_cast<uint16_t*>(dB);
    p.b.L = pool.h_out;
    p.indptr = seg.indptr;
    p.ranks = pool.ranks;
    p.M = M;
    p.n_adapters = pool.n_adapters;
    p.r_max = pool.r_max;
    if (pool.r_max <= 16) return launch_outer<16>(p, by_adapter, stream);
    if (pool.r_max == 32) return launch_outer<32>(p, by_adapter, stream);
    return launch_outer<64>(p, by_adapter, stream);
}

}  // namespace lora
