// gated.cu -- the gated feed-forward block's matrix products on the tcgen05 tensor cores
// (TMA in, accumulators in TMEM), with the multi-tenant LoRA term of both projections:
//
//   forward   g = x.Wg^T + s_a (x.A0_a).B0_a,  u = x.Wu^T + s_a (x.A1_a).B1_a,
//             h = bf16(act(g) u), and on request g, u as 8-bit checkpoints (act8.cuh);
//   backward  dX = dg.Wg + du.Wu + s_a (dg.B0_a^T).A0_a^T + s_a (du.B1_a^T).A1_a^T.
//
// One kernel, two modes. A tile is 128 tokens (the MMA's M) by up to 256 accumulator
// columns. Forward: the columns are bnh of gate and the same bnh of up, so one MMA per 16 of
// K computes both and the thread that drains a row finds g and u of the same element in the
// same TMEM lane: the activation and the product need no exchange, and a block of 32 columns
// (one checkpoint scale) lies in one thread. Backward: the sum runs over dg then du (2F long),
// and Wg, Wu [F][K] are read as they are, as the MMA's MN-major operand (no transposed copy).
//
// The LoRA term extends the sum of a tile. The kernels before this one list, for every token tile, the
// rank blocks (16 ranks of an adapter) that any of its rows uses; a step adds `ups` blocks of one
// slice: s_a v of the tile's rows (zero in the blocks of other adapters) against the blocks of
// B_a (forward, MN-major as it is stored) or A_a (backward, K-major as it is stored). v is split
// into bf16 halves hi + lo that add up in the accumulator (16 bits of v).
// Forward: a step is a stage of the ring like the others. expand_kernel writes its operand out, zeros
// included, so that it is one or two boxes; B comes by TMA from the pool. The steps lie between the main
// stages, in a unit's first tile in the last eighth, so that the shrink runs under the others.
// (Steps of their own buffers, put together by eight warps with cp.async, had cost 1.5 us each where
// they were many: 512 tokens sorted over 48 adapters of rank 32, 4096 x 11008, 388 us, 171 in the ring.)
// Backward: a step has shared memory beside the ring, where builders put it together with cp.async, one
// ahead of the one that they hand over where two buffers fit; its sums are long beside its steps.
// The tokens of more than one token tile come in the segments' order, by adapter, where that saves
// steps (gated_order): a tile then needs few adapters' blocks however the batch is mixed. gather_kernel
// copies x's rows into that order, except where 128 of them follow one another already, as in a
// batch that comes sorted; h and the checkpoints are written to the tokens' own rows. (4096 x 11008, 2048
// tokens mixed over 48 adapters of rank 16: 940 us in their own order, 301 in this; over 16 of rank 64 1480,
// 329; 20 calls in a row, called for seconds the latter are 343 and 371, by the power cap. TMA's gather of
// four rows at a time took 1.2 us a stage instead of .4.) The backward writes dg and du in that order to
// begin with.
//
// More than 128 tokens usually run on pairs of CTAs (cta_group::2, clusters of two): 256 tokens by
// the same columns, each CTA with its 128 rows of A and half of B (forward: the even CTA the
// gate's rows, the odd one up's), so a stage is 32 KB instead of 48 and six of them cover the
// latency of the loads, which had bounded the products (2048 x 8192 x 11008 without adapters:
// three stages 590 us, four 544, five 506). The even CTA issues the MMAs; loads, LoRA
// steps and drains run in both.
//
// The backward has few tiles where the tokens are few, with long sums: 16 tokens have 32 tiles for
// 148 SMs. The tiles of its last round are then shared: their sums are cut into S pieces of
// equal length, spread over all units; a piece writes its fp32 accumulator to the workspace, and
// whichever piece of a tile is done last adds all of them in order and finishes the tile
// (nobody waits for another, and the sum does not depend on who is last). Units that run side by
// side take the same piece of neighbouring tiles, so they read the same weights at the same
// time. (4096 x 11008: 16 tokens 119 -> 47 us, 512 tokens 156 -> 110 us; cutting the stages of all
// shared tiles into one equal run per unit made 1024 tokens 212 us instead of 164, by reading the
// weights at different times; in the forward, bound by power, sharing gained nothing.)
//
// Roles: warps 0..7 drain accumulators (warp w: TMEM lanes 32 (w % 4), column chunks by w / 4); warp 8
// fills the ring by TMA; warp 9 issues the MMAs; behind them the forward has four warps that fetch the
// steps' B (448 threads), the backward eight that build its LoRA steps (576). Two accumulators
// (512 TMEM columns), so a tile drains under the next one's
// products. Every wait is bounded; on expiry the CTA records a status word, lets what it
// issued land and leaves.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstring>

#include "act8.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "sgmv_common.cuh"

namespace lora {
namespace {

constexpr int kGDrainWarps = 8;
constexpr int kGProducer = kGDrainWarps, kGMma = kGProducer + 1, kGBuilder0 = kGMma + 1;
constexpr int kGBuilders = 256;
constexpr int kGMaxA = 4, kGMaxB = 4;        // 16-byte pieces of a LoRA step per builder
constexpr int kGThreads = (kGBuilder0 + kGBuilders / 32) * 32;
constexpr int kGLoaders = 4;                   // the forward's warps behind the issuer: B of a step, a block each
constexpr int kGFwdThreads = (kGBuilder0 + kGLoaders) * 32;
constexpr int kGTileM = 128;
constexpr int kGMaxStages = 12;
constexpr int kGKBlock = 64;                  // K per stage: 128 bytes of bf16, one swizzle row
constexpr int kGSmem = 226 * 1024;            // dynamic shared memory of the one CTA per SM (1 KB is static)
constexpr int kGSmemShort = 208 * 1024;       // the same with at most 64 tokens
constexpr int kGBarBytes = 512;
constexpr int kGMaxLora = 2;                  // LoRA step buffers
constexpr int kRankBoxes = 5;                // maps of B's rows, boxes of 1, 2, 4, 8 and 16
constexpr int kGAccCols = 256;                // TMEM columns of an accumulator
constexpr int kGCounts = 256;                 // counts of shared tiles (fewer than units, two CTAs each)
constexpr int kListMax = kGTileM * (LORA_MAX_RANK / 16);  // rank blocks of 128 tokens
enum { kGFwd = 0, kGBwd = 1 };
// status bits of the bounded waits
enum { kGStRing = 0x1, kGStMma = 0x2, kGStBuild = 0x4, kGStDrain = 0x8, kGStStall = 0x10 };

struct GatedParams {
    int M, NC;        // tokens; output columns (F forward, K backward)
    int mt, tiles;    // token tiles (of 128, or 256 for a pair), all tiles
    int bn, cols;     // accumulator columns of a tile; output columns of a tile (bn / 2 forward)
    int b_bytes;      // a CTA's part of B in a stage
    int kb, kb_half;  // ring stages of a tile's main sum; backward: those of dg
    int stages, stage_bytes, a_bytes;
    int smem;         // dynamic shared memory
    int units, rounds;    // CTAs or pairs; whole tiles of each: tile = unit + round * units
    int whole, shared;    // tiles before the shared ones; shared tiles
    int split;            // pieces of a shared tile
    float* part;          // [shared][split][CTAs][bn / 4][128][4] accumulators of pieces
    int* count;           // [shared][CTAs] pieces done, zero on entry (the element-wise kernel)
    int act;
    uint16_t* out;    // h [M][F] or dX [M][K]
    uint8_t *g_codes, *g_scales, *u_codes, *u_scales;  // forward checkpoints or NULL
    uint32_t* status;
    unsigned long long timeout_ns;
    int inject_stall;
    // LoRA
    const uint16_t* ops;      // backward: [2][M][hi r16 | lo r16]: s_a v as bf16 halves
    const uint16_t* B;        // backward: A [2][n_adapters][NC][r_max]
    const int32_t* lists;     // [mt][kListMax per 128 tokens] rank blocks of a token tile (see block_code)
    const int32_t* list_len;  // [mt]
    const int32_t* list_base; // forward: the tile's first step in the expanded operand, per slice
    const int32_t* tok_adapter;
    const int32_t* order;     // the token of each row of the tiles (NULL: the rows are the tokens)
    int n_adapters, r_max, r16;
    int ups;                  // rank blocks per step (forward: those of both slices counted)
    int lbufs, lora_bytes;    // backward: step buffers behind the ring
};
template <bool RING>
struct GatedMaps {
    CUtensorMap a[2], b[2];                // x and its rows by adapter, or dg, du; Wg, Wu
    CUtensorMap e;                         // RING: the expanded operand (expand_kernel)
    CUtensorMap l[RING ? kRankBoxes : 1];  // RING: the pool's B [2 n_adapters][r_max][NC]
};

// K-major operand, 128-byte rows, 128-byte swizzle: 8-row groups 1024 bytes apart.
__device__ __forceinline__ uint64_t g_desc_k(uint32_t a)
{
    return (uint64_t)((a >> 4) & 0x3FFFu) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) |
           ((uint64_t)2 << 61);
}
// MN-major operand in 64-column boxes of 128-byte rows (one per k), 128-byte swizzle, boxes
// `atom` bytes apart.
__device__ __forceinline__ uint64_t g_desc_mn(uint32_t a, uint32_t atom)
{
    return (uint64_t)((a >> 4) & 0x3FFFu) | ((uint64_t)((atom >> 4) & 0x3FFFu) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// kind::f16, bf16 operands, fp32 accumulator, M = m, N = n; B MN-major or K-major.
__device__ __forceinline__ uint32_t g_idesc(int m, int n, bool b_mn)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// Bounded wait by one thread that sleeps between its probes.
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int32_t* status, int code,
                                       unsigned long long limit, bool honor_abort)
{
    const unsigned long long t0 = ptx::globaltimer();
    while (!ptx::mbar_try_wait_ns(bar, parity, 20000)) {
        if (honor_abort && *abort_flag) return false;
        if (ptx::globaltimer() - t0 > limit) {
            *abort_flag = 1;
            atomicOr(status, code);
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int32_t* status, int code,
                                         unsigned long long limit, bool honor_abort = true)
{
    return ptx::mbar_try_wait(bar, parity) || wait_slow(bar, parity, abort_flag, status, code, limit, honor_abort);
}
// The same for a converged warp; every lane gets the same answer.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int32_t* status, int code,
                                          unsigned long long limit, bool honor_abort = true)
{
    if (__all_sync(0xffffffffu, ptx::mbar_try_wait(bar, parity))) return true;
    return __all_sync(0xffffffffu, wait_slow(bar, parity, abort_flag, status, code, limit, honor_abort));
}
// The same for the warps of a role (n threads, named barrier id): one thread probes, the
// others sleep at the barrier; all get the same answer.
__device__ __forceinline__ bool wait_role(int id, int n, bool prober, uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                          int32_t* status, int code, unsigned long long limit)
{
    const bool bad = prober && !wait_bar(bar, parity, abort_flag, status, code, limit);
    if (ptx::named_sync_or(id, n, bad)) return false;
    if (!prober) ptx::mbar_try_wait(bar, parity);  // complete: every thread observes the phase itself
    return true;
}

// act(g): x sigmoid(x), or x Phi(x) through the complementary error function (no
// cancellation in the lower tail). The sigmoid of exp(-|g|): with exp(-g) the denominator passes 2^126 below
// g = -87, where the fast division gives zero.
__device__ __forceinline__ float gate(int act, float g)
{
    if (act == LORA_ACT_SILU) {
        const float t = __expf(-fabsf(g));
        return __fdividef(g < 0.f ? g * t : g, 1.f + t);
    }
    return 0.5f * g * erfcf(g * -0.70710678118654752f);
}

__device__ __forceinline__ void store_bf16x8(uint16_t* dst, const float* v)
{
    *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                                pack_bf16x2(v[6], v[7]));
}

// One thread's block of 32 accumulator columns as a checkpoint block; columns past the row's
// end hold zeros and are not stored (n: 32 or 16 live columns).
__device__ __forceinline__ void save_block(const float* v, int n, uint8_t* codes, uint8_t* scale)
{
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) top = fmaxf(top, act8::finite(v[i]) ? fabsf(v[i]) : 0.f);
    const uint32_t E = act8::scale_code(top);
    const float inv = act8::inv_scale(E);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float* w = v + h * 16 + i * 4;
            o[i] = (uint32_t)ptx::cvt_e4m3x2(act8::scaled(w[0], inv), act8::scaled(w[1], inv)) |
                   ((uint32_t)ptx::cvt_e4m3x2(act8::scaled(w[2], inv), act8::scaled(w[3], inv)) << 16);
        }
        if (h * 16 < n) *reinterpret_cast<uint4*>(codes + h * 16) = make_uint4(o[0], o[1], o[2], o[3]);
    }
    *scale = (uint8_t)E;
}

// A unit's work, as every role walks it: stages [k0, k1) of a tile at a time.
struct Walk {
    int unit, round, tile, piece, k0, k1, seen;
    __device__ explicit Walk(int u) : unit(u), round(0), seen(0) {}
    __device__ __forceinline__ bool next(const GatedParams& p)
    {
        ++seen;
        piece = -1;
        k0 = 0;
        k1 = p.kb;
        if (round < p.rounds) {
            tile = unit + round++ * p.units;
            if (tile < p.tiles) return true;
        }
        const int q = unit + (round - p.rounds) * p.units;
        if (q >= p.shared * p.split) return false;
        ++round;
        piece = q / p.shared;
        tile = p.whole + q - piece * p.shared;
        k0 = (int)((long long)p.kb * piece / p.split);
        k1 = (int)((long long)p.kb * (piece + 1) / p.split);
        return true;
    }
    // The stage after which the tile's LoRA steps begin to be spread: a unit's first piece leaves the
    // shrink time. (The forward's steps are stages like others, so they may all come in the last
    // eighth; the backward's take their time each.)
    __device__ __forceinline__ int lora_first(bool fwd) const { return seen == 1 ? k0 + (k1 - k0) * (fwd ? 7 : 2) / 8 : k0; }
};
// A rank block as the lists hold it: adapter, which 16 of its ranks, how many of them it has, the
// slices whose matrix is marked as non-finite (bits).
__device__ __forceinline__ int block_code(int adapter, int block, int live, int bad) { return adapter << 9 | block << 7 | bad << 5 | live; }
__device__ __forceinline__ int block_adapter(int u) { return u >> 9; }
__device__ __forceinline__ int block_rank0(int u) { return (u >> 7 & 3) * 16; }
__device__ __forceinline__ int block_live(int u) { return u & 31; }
__device__ __forceinline__ int block_bad(int u) { return u >> 5 & 3; }
constexpr int kNoBlock = -3 * 512;  // an adapter that no row has, nothing live
// The rank in column j of block b of an adapter of rank R in the forward's operand, -1: zero. A box of B's
// rows must not reach past the rank, where the pool holds anything, so the last block of several is the
// last 16 ranks, and a single one below 16 is its first p and its last p ranks, p the largest power of
// two, zeros behind them. What comes twice is used once. (Boxes of the powers of two that make up the
// rank, and zeros to 16, five or six copies: side by side, 4096 x 11008, 512 tokens of 48 adapters of ranks drawn up
// to 32 139 us, so 135; 36 of 32 53.6, 52.)
__device__ __forceinline__ int block_rank(int R, int b, int j)
{
    if (R >= 16) {
        const int r = min(16 * b, R - 16) + j;
        return r >= 16 * b ? r : -1;
    }
    const int p = 1 << (31 - __clz(R));
    if (j < p) return j;
    const int r = R - 2 * p + j;
    return j < 2 * p && r >= p ? r : -1;
}
// LoRA steps of a token tile with this many rank blocks: forward ups / 2 blocks with both slices each (one
// block, a sorted batch's usual tile, is one stage then and not two), backward ups of one
// slice. A piece of a shared tile has its share of them.
template <int MODE>
__device__ __forceinline__ int lora_steps(const GatedParams& p, int blocks)
{
    return MODE == kGFwd ? (blocks + p.ups / 2 - 1) / (p.ups / 2) : 2 * ((blocks + p.ups - 1) / p.ups);
}
__device__ __forceinline__ int steps_begin(const GatedParams& p, int steps, int piece) { return piece < 0 ? 0 : steps * piece / p.split; }
__device__ __forceinline__ int steps_end(const GatedParams& p, int steps, int piece) { return piece < 0 ? steps : steps * (piece + 1) / p.split; }
// A step's operand: tiles of 64 columns (four groups of 16: ups of hi, ups of lo), the B part behind
// them.
__host__ __device__ __forceinline__ uint32_t lora_b_offset(const GatedParams& p) { return (uint32_t)(p.ups / 2 * p.a_bytes); }
// A tile in the order in which every role takes it: main stages [k0, k1), and between them from
// lora_first on, evenly, the LoRA steps [e, e + due) that `begin` names. False: given up.
template <typename Main, typename Begin, typename Step>
__device__ __forceinline__ bool walk_tile(const Walk& w, bool fwd, Main main_stages, Begin begin, Step step)
{
    const int first = w.lora_first(fwd), spread = w.k1 - first;
    int kb = first + 1, e = 0, due = 0;
    if (!main_stages(w.k0, kb)) return false;
    begin(e, due);
    const int ext = due;
    for (;;) {
        for (; due >= spread; due -= spread, ++e)
            if (!step(e)) return false;
        if (kb >= w.k1) return true;
        const int n = ext ? min((spread - due + ext - 1) / ext, w.k1 - kb) : w.k1 - kb;
        if (!main_stages(kb, kb + n)) return false;
        kb += n;
        due += n * ext;
    }
}
// K-major operand of 64-byte rows (32 columns), 64-byte swizzle.
__device__ __forceinline__ uint64_t g_desc_k64(uint32_t a)
{
    return (uint64_t)((a >> 4) & 0x3FFFu) | ((uint64_t)1 << 16) | ((uint64_t)(512 >> 4) << 32) | ((uint64_t)1 << 46) |
           ((uint64_t)4 << 61);
}

// A warp's look at the 128 rows of a tile from row0 on, in the segments' order: are their tokens a run?
// Then the rows are read where they are, else from the copy that gather_kernel made.
struct RowRun {
    int tok[4];
    __device__ __forceinline__ void load(const int32_t* order, int M, int row0, int lane)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) tok[i] = order[min(row0 + lane * 4 + i, M - 1)];
    }
    // the first token, or -1: no run
    __device__ __forceinline__ int first(int M, int row0, int lane) const
    {
        const int t0 = __shfl_sync(0xffffffffu, tok[0], 0);
        bool run = true;
#pragma unroll
        for (int i = 0; i < 4; ++i) run = run && (row0 + lane * 4 + i >= M || tok[i] == t0 + lane * 4 + i);
        return __all_sync(0xffffffffu, run) ? t0 : -1;
    }
};

template <int MODE, bool LORA, bool PAIR>
__global__ void __launch_bounds__(MODE == kGFwd ? kGFwdThreads : kGThreads, 1)
gated_gemm_kernel(const __grid_constant__ GatedMaps<MODE == kGFwd && LORA> maps, const GatedParams p)
{
    constexpr bool kRing = MODE == kGFwd && LORA;  // LoRA steps come through the ring
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ int s_abort;
    __shared__ uint32_t s_tmem;
    __shared__ int s_last;       // this CTA's part of a shared tile was the last
    __shared__ uint32_t s_fills[kGMaxStages];  // PAIR: stages this CTA's producer filled, for the leader,
    __shared__ uint32_t s_tx[kGMaxStages];     // and the bytes of each one's last fill
    __shared__ int4 s_job[2];                  // a step for the loaders: stage (-1: the end), tile, first block
    constexpr int kCtas = PAIR ? 2 : 1, kTokens = kCtas * kGTileM;
    const int rank = PAIR ? (int)(blockIdx.x & 1) : 0;
    const int unit = (int)blockIdx.x / kCtas;
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // warp: uniform
    const uint32_t raw_u = ptx::smem_u32(smem_raw);
    const uint32_t base_u = (raw_u + 1023u) & ~1023u;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem_raw + p.smem - kGBarBytes);
    uint64_t* empty = full + kGMaxStages;
    uint64_t* lfull = empty + kGMaxStages;  // LoRA step buffers
    uint64_t* lempty = lfull + kGMaxLora;
    uint64_t* tfull = lempty + kGMaxLora;
    uint64_t* tempty = tfull + 2;
    uint64_t* mdone = tempty + 2;
    uint64_t* stall = mdone + 1;  // test hook: never completed
    volatile int* abort_flag = &s_abort;
    int32_t* status = reinterpret_cast<int32_t*>(p.status);

    if (threadIdx.x == 0) {
        s_abort = 0;
        for (int s = 0; s < kGMaxStages; ++s) {
            ptx::mbar_init(&full[s], 1);
            ptx::mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < kGMaxLora; ++b) {
            ptx::mbar_init(&lfull[b], kCtas);
            ptx::mbar_init(&lempty[b], 1);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(&tfull[b], 1);
            ptx::mbar_init(&tempty[b], kCtas * kGDrainWarps);
        }
        ptx::mbar_init(mdone, 1);
        ptx::mbar_init(stall, 1);
        ptx::fence_mbar_init();
    }
    __syncwarp();
    if (PAIR) ptx::cluster_sync();  // the other CTA runs, its barriers are set up
    if (warp == kGMma) {
        if (PAIR) {
            ptx::tmem_alloc2(&s_tmem, 2 * kGAccCols);
            ptx::tmem_relinquish2();
        } else {
            ptx::tmem_alloc(&s_tmem, 2 * kGAccCols);
            ptx::tmem_relinquish();
        }
    }
    // Without adapters the operands may come from the kernel before this one. With them that
    // kernel is operand_kernel, and the one before it the shrink, which let operand_kernel (and so
    // this one) start only after all that ran before the shrink was complete: x, dg, du and the
    // weights may be read at once, operand_kernel's outputs after the wait.
    if (!LORA) ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = s_tmem;
    // the leader's barriers that both CTAs signal (shared::cluster addresses)
    auto leaders = [&](uint64_t* bar) { return PAIR ? ptx::mapa(ptx::smem_u32(bar), 0) : ptx::smem_u32(bar); };

    if (warp == kGProducer) {
        // ================================================================ producer
        const bool leader = ptx::elect_one();
        int st = 0;
        uint32_t use = 0;  // uses of stage st before this one (of the stages below st: one more)
        bool ok = true;
        if (p.inject_stall && blockIdx.x == 0)  // test hook: a wait that runs out
            ok = wait_warp(stall, 0, abort_flag, status, kGStStall, p.timeout_ns);
        auto load = [&](uint32_t dst, const CUtensorMap* map, int c0, int c1) {
            if (PAIR) ptx::tma_load_2d_pair(dst, map, leaders(&full[st]), c0, c1);
            else ptx::tma_load_2d(dst, map, &full[st], c0, c1);
        };
        auto stage_free = [&]() {
            return ok = use == 0 || wait_warp(&empty[st], (use - 1) & 1, abort_flag, status, kGStRing, p.timeout_ns);
        };
        auto expect = [&](uint32_t bytes) {  // per CTA
            if (!leader) return;
            if (rank == 0) ptx::mbar_arrive_expect_tx(&full[st], kCtas * bytes);
            if (PAIR) s_tx[st] = bytes;
        };
        auto next_stage = [&]() {
            __syncwarp();
            if (++st == p.stages) {
                st = 0;
                ++use;
            }
        };
        // where a tile's rows of x are (see RowRun), of the next tile's a tile ahead
        RowRun run, next_run;
        if (kRing && p.order && unit < p.tiles) next_run.load(p.order, p.M, (unit % p.mt) * kTokens + rank * kGTileM, lane);
        // the tile's rank blocks and where its steps' operands are; the next tile's a tile ahead
        int blocks = 0, base = 0, next_blocks = 0, next_base = 0;
        auto fetch_list = [&](int tile) {
            if (tile >= p.tiles) return;
            next_blocks = p.list_len[tile % p.mt];
            next_base = p.list_base[tile % p.mt];
        };
        const uint64_t once = ptx::l2_policy_evict_first();
        // A job for the loaders; they are done with the one before when they come to the barrier.
        int jobs = 0;
        auto hand_out = [&](int4 job) {
            if (lane == 0) s_job[jobs & 1] = job;
            ++jobs;
            __syncwarp();
            ptx::named_sync(1, (1 + kGLoaders) * 32);
        };
        bool waited = false;
        for (Walk w(unit); ok && w.next(p);) {
            int row0 = (w.tile % p.mt) * kTokens + rank * kGTileM;
            const int n0 = (w.tile / p.mt) * p.cols;
            bool copied = false;
            if (kRing && p.order) {
                run = next_run;
                const int t0 = run.first(p.M, row0, lane);
                copied = t0 < 0;
                if (!copied) row0 = t0;
                const int after = w.tile + p.units;
                if (after < p.tiles) next_run.load(p.order, p.M, (after % p.mt) * kTokens + rank * kGTileM, lane);
            }
            auto main_stages = [&](int kb, int stop) {
                for (; kb < stop; ++kb) {
                    if (!stage_free()) return false;
                    const uint32_t sa = base_u + (uint32_t)(st * p.stage_bytes), sb = sa + (uint32_t)p.a_bytes;
                    expect((uint32_t)(p.a_bytes + p.b_bytes));
                    if (leader) {
                        if (MODE == kGFwd) {
                            load(sa, kRing && copied ? &maps.a[1] : &maps.a[0], kb * kGKBlock, row0);
                            if (PAIR) {
                                load(sb, &maps.b[rank], kb * kGKBlock, n0);
                            } else {
                                // one token tile reads the weights once: they leave L2 to the adapters
                                // (16 tokens, 8192 x 28672, 16 adapters: 158 us, without 163)
                                for (int i = 0; i < 2; ++i)
                                    if (kRing && p.mt == 1)
                                        ptx::tma_load_2d_hint(sb + (uint32_t)(i * p.cols * 128), &maps.b[i], &full[st], kb * kGKBlock, n0, once);
                                    else
                                        load(sb + (uint32_t)(i * p.cols * 128), &maps.b[i], kb * kGKBlock, n0);
                            }
                        } else {
                            const bool up = kb >= p.kb_half;
                            const int f0 = (up ? kb - p.kb_half : kb) * kGKBlock, c0 = n0 + rank * (p.bn / 2);
                            load(sa, &maps.a[up], f0, row0);
                            for (int b = 0; b < p.b_bytes / 8192; ++b)
                                load(sb + (uint32_t)(b * 8192), &maps.b[up], c0 + b * 64, f0);
                        }
                    }
                    next_stage();
                }
                return true;
            };
            if (!kRing) {
                main_stages(w.k0, w.k1);
                continue;
            }
            auto begin = [&](int& e, int& due) {
                if (!waited) {
                    ptx::pdl_wait();
                    waited = true;
                    fetch_list(w.tile);
                }
                blocks = __shfl_sync(0xffffffffu, next_blocks, 0);
                base = __shfl_sync(0xffffffffu, next_base, 0);
                fetch_list(w.tile + p.units);
                e = 0;
                due = lora_steps<MODE>(p, blocks);
            };
            const int atoms = (p.cols / kCtas + 63) >> 6, rows = PAIR ? kTokens : p.a_bytes >> 7;
            auto step = [&](int e) {  // the operand; the loaders fetch B into the same stage
                if (!stage_free()) return false;
                const int first = e * (p.ups / 2);
                hand_out(make_int4(st, w.tile, first, 0));
                const uint32_t sa = base_u + (uint32_t)(st * p.stage_bytes);
                expect(lora_b_offset(p) + (uint32_t)(min(p.ups, 2 * (blocks - first)) * atoms * 2048));
                if (leader)
                    for (int c = 0; c < p.ups / 2; ++c)
                        load(sa + (uint32_t)(c * p.a_bytes), &maps.e, 0, ((base + e) * (p.ups / 2) + c) * rows + rank * kGTileM);
                next_stage();
                return true;
            };
            walk_tile(w, MODE == kGFwd, main_stages, begin, step);
        }
        if (kRing) hand_out(make_int4(-1, 0, 0, 0));
        if (PAIR) {  // landed below, once both producers have stopped
            if (lane < p.stages) s_fills[lane] = use + (lane < st ? 1 : 0);
        } else {
            // every copy this CTA issued lands before it leaves: the last fill of each stage
            for (int s = 0; s < p.stages; ++s) {
                const uint32_t fills = use + (s < st ? 1 : 0);
                if (fills) wait_warp(&full[s], (fills - 1) & 1, abort_flag, status, kGStRing, p.timeout_ns, false);
            }
        }
    } else if (warp == kGMma) {
        // ================================================================ MMA issuer
        // The whole warp walks the ring and one lane issues: what the descriptors are made of stays
        // in uniform registers. (With the walk inside a lane-0 branch, an issue of four MMAs took
        // longer than their 512 cycles of products: 2048 x 8192 x 11008 with adapters 645 us.)
        const bool leader = ptx::elect_one();
        int st = 0, acc = 0;
        uint32_t use = 0, lb = 0, turn = 0;  // turns of the ring; buffer of the next LoRA step, its turns
        bool ok = true, waited = false;
        const uint32_t id_main = g_idesc(kTokens, p.bn, MODE == kGBwd), id_lora = g_idesc(kTokens, p.cols, MODE == kGFwd);
        auto mma = [](uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t more) {
            if (PAIR) ptx::tc_mma2_f16(d, a, b, id, more);
            else ptx::tc_mma_f16_all(d, a, b, id, more);
        };
        auto commit = [](uint64_t* bar) {
            if (PAIR) ptx::tc_commit2(bar);
            else ptx::tc_commit(bar);
        };
        // descriptors of stage 0 and of LoRA buffer 0; the address field counts 16-byte units
        const uint32_t lora_u = base_u + (kRing ? 0u : (uint32_t)(p.stages * p.stage_bytes)), lora_bu = lora_u + lora_b_offset(p);
        const uint64_t da0 = g_desc_k(base_u);
        const uint64_t db0 = MODE == kGFwd ? g_desc_k(base_u + (uint32_t)p.a_bytes) : g_desc_mn(base_u + (uint32_t)p.a_bytes, 8192);
        const uint64_t la0 = g_desc_k(lora_u);
        const uint64_t lb0 = MODE == kGFwd ? g_desc_mn(lora_bu, (uint32_t)(p.ups * 2048)) : g_desc_k64(lora_bu);
        const uint32_t stage16 = (uint32_t)p.stage_bytes >> 4;
        for (Walk w(unit); rank == 0 && ok && w.next(p); ++acc) {
            const int m = w.tile % p.mt, buf = acc & 1;
            int blocks = LORA && waited ? p.list_len[m] : 0;
            if (acc >= 2 && !(ok = wait_warp(&tempty[buf], (uint32_t)(((acc >> 1) - 1) & 1), abort_flag, status, kGStMma,
                                             p.timeout_ns)))
                break;
            const uint32_t d = tmem + (uint32_t)(buf * kGAccCols);
            auto next_stage = [&]() {
                __syncwarp();
                if (++st == p.stages) {
                    st = 0;
                    ++use;
                }
            };
            // main stages [kb, stop) of the tile
            auto main_stages = [&](int kb, int stop) {
                for (; kb < stop; ++kb) {
                    if (!(ok = wait_warp(&full[st], use & 1, abort_flag, status, kGStMma, p.timeout_ns))) return false;
                    ptx::tc_fence_after();
                    if (leader) {
                        const uint64_t da = da0 + (uint32_t)st * stage16, db = db0 + (uint32_t)st * stage16;
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            mma(d, da + ks * 2, db + ks * (MODE == kGFwd ? 2 : 128), id_main, kb > w.k0 || ks ? 1u : 0u);
                        commit(&empty[st]);
                    }
                    next_stage();
                }
                return true;
            };
            auto begin = [&](int& e, int& due) {
                if (!waited) {
                    ptx::pdl_wait();
                    waited = true;
                    blocks = p.list_len[m];
                }
                blocks = __shfl_sync(0xffffffffu, blocks, 0);  // uniform, and so the walk
                const int all = lora_steps<MODE>(p, blocks);
                e = steps_begin(p, all, w.piece);
                due = steps_end(p, all, w.piece) - e;
            };
            auto step = [&](int e) {
                if (!(ok = kRing ? wait_warp(&full[st], use & 1, abort_flag, status, kGStMma, p.timeout_ns)
                                 : wait_warp(&lfull[lb], turn & 1, abort_flag, status, kGStMma, p.timeout_ns)))
                    return false;
                ptx::tc_fence_after();
                if (leader) {
                    const uint32_t at = kRing ? (uint32_t)st * stage16 : lb * ((uint32_t)p.lora_bytes >> 4);
                    // forward: block k / 2, slice k & 1
                    const int n = MODE == kGFwd ? min(p.ups, 2 * (blocks - e * (p.ups / 2))) : min(p.ups, blocks - (e >> 1) * p.ups);
                    for (int h = 0; h < 2; ++h)
                        for (int k = 0; k < n; ++k) {
                            const int c = h * p.ups + k;  // 16-column group of the operand: 4 per swizzle row
                            const uint32_t ds = MODE == kGFwd ? d + (uint32_t)((k & 1) * p.cols) : d;
                            mma(ds, la0 + at + (uint32_t)((c >> 2) * (p.a_bytes >> 4) + (c & 3) * 2),
                                lb0 + at + (uint32_t)(k * (MODE == kGFwd ? 128 : 2)), id_lora, 1u);
                        }
                    commit(kRing ? &empty[st] : &lempty[lb]);
                }
                if (kRing) {
                    next_stage();
                } else {
                    __syncwarp();
                    if (++lb == (uint32_t)p.lbufs) {
                        lb = 0;
                        ++turn;
                    }
                }
                return true;
            };
            if (LORA) walk_tile(w, MODE == kGFwd, main_stages, begin, step);
            else main_stages(w.k0, w.k1);
            if (ok && leader) commit(&tfull[buf]);
            __syncwarp();
        }
        // every MMA issued is complete before the CTA (of a pair: either, by the barrier below) leaves
        if (rank == 0) {
            if (leader) commit(mdone);
            __syncwarp();
            wait_warp(mdone, 0, abort_flag, status, kGStMma, p.timeout_ns, false);
        }
    } else if (kRing && warp >= kGBuilder0) {
        // ================================================================ B of the LoRA steps
        // A warp per block of a step, since issuing copies of changing shapes is what takes time (by the
        // producer's lanes alone a step took 1 us, which was all that 64 tokens of 64 adapters of rank
        // 64 waited for: 169 us, 148 with the loaders).
        const int k = warp - kGBuilder0, s = k & 1, atoms = (p.cols / kCtas + 63) >> 6;
        int m = -1, q = 0, u = 0, ahead = 0;  // this warp's block of the last step, of the one after it
        for (int jobs = 0;; ++jobs) {
            ptx::named_sync(1, (1 + kGLoaders) * 32);
            const int4 job = s_job[jobs & 1];
            if (job.x < 0) break;
            if (jobs == 0) ptx::pdl_wait();
            if (k >= p.ups) continue;
            const int jm = job.y % p.mt, per = p.ups / 2;
            const int32_t* list = p.lists + (size_t)jm * kListMax * kCtas + job.z + (k >> 1);
            const int left = p.list_len[jm] - job.z - (k >> 1);  // blocks from this one on
            u = left <= 0 ? kNoBlock : jm == m && job.z == q + per ? ahead : list[0];
            ahead = left > per ? list[per] : kNoBlock;
            m = jm;
            q = job.z;
            if (u != kNoBlock && lane < atoms) {
                // see block_rank; what is past the last matrix comes as zeros (a marked one too, see Eight)
                const int x = (job.y / p.mt) * p.cols + rank * (p.cols / kCtas) + lane * 64, nothing = 2 * p.n_adapters;
                const uint32_t dst = base_u + (uint32_t)(job.x * p.stage_bytes) + lora_b_offset(p) + (uint32_t)((lane * p.ups + k) * 2048);
                const int z = block_bad(u) >> s & 1 ? nothing : s * p.n_adapters + block_adapter(u), live = block_live(u);
                auto box = [&](int row, int b, int y, int matrix) {
                    if (PAIR) ptx::tma_load_3d_pair(dst + (uint32_t)(row * 128), &maps.l[b], leaders(&full[job.x]), x, y, matrix);
                    else ptx::tma_load_3d(dst + (uint32_t)(row * 128), &maps.l[b], &full[job.x], x, y, matrix);
                };
                if (live == 16 || block_rank0(u)) {
                    box(0, 4, block_rank0(u) + live - 16, z);
                } else {
                    const int b = 31 - __clz(live);
                    box(0, b, 0, z);
                    box(1 << b, b, live - (1 << b), z);
                    for (int k2 = b + 1; k2 < 4; ++k2) box(1 << k2, k2, 0, nothing);
                }
            }
            __syncwarp();
        }
    } else if (warp >= kGBuilder0) {
        // ================================================================ LoRA steps
        if (LORA && MODE == kGBwd) {
            ptx::pdl_wait();
            const int bt = threadIdx.x - kGBuilder0 * 32;
            // A builder's pieces lie in one column of 16-byte pieces, a fixed number of rows apart
            // (a multiple of eight, so their swizzle is the same): piece i of the operand in row
            // a_row + i a_step, column a_c; of A_a in row b_row + i b_step (an output column), column b_c.
            const int a_c = bt & 7, a_row = bt >> 3, a_step = kGBuilders >> 3;  // (two blocks per step)
            const int a_rows = p.a_bytes >> 7;
            const int a_half = a_c >> 2, a_k = a_c & 3;  // hi or lo; piece of the blocks
            const int b_c = bt & 3, b_row = bt >> 2, b_step = kGBuilders >> 2;
            const int b_cols = p.cols / kCtas, b_n0 = rank * b_cols;  // this CTA's columns of the tile
            const uint32_t a_off = (uint32_t)(a_row * 128 + ((a_c ^ (a_row & 7)) << 4));
            const uint32_t b_off = lora_b_offset(p) + (uint32_t)(b_row * 64 + ((b_c ^ ((b_row >> 1) & 3)) << 4));
            // the walk over the steps: step e of `ext` of the tile
            Walk w(unit);
            int e = -1, ext = 0, m = 0, n0 = 0, row0 = 0, blocks = 0;  // the tile's next step, where they end
            int ids[kGMaxA];  // adapters of this builder's operand rows
            auto advance = [&]() -> bool {
                while (++e >= ext) {
                    if (!w.next(p)) return false;
                    m = w.tile % p.mt;
                    n0 = (w.tile / p.mt) * p.cols + b_n0;
                    row0 = m * kTokens + rank * kGTileM;
                    blocks = p.list_len[m];
                    const int all = lora_steps<MODE>(p, blocks);
                    ext = steps_end(p, all, w.piece);
                    e = steps_begin(p, all, w.piece) - 1;
#pragma unroll
                    for (int i = 0; i < kGMaxA; ++i) {
                        const int row = a_row + i * a_step, tok = row0 + row;
                        ids[i] = row < a_rows && tok < p.M ? p.tok_adapter[p.order ? p.order[tok] : tok] : -2;
                    }
                }
                return true;
            };
            // the blocks that the next step's pieces come from: of the operand, of A_a
            int ua, ub;
            auto blocks_of_step = [&]() {
                const int b0 = (e >> 1) * p.ups;
                const int32_t* list = p.lists + (size_t)m * kListMax * kCtas;
                const int ka = b0 + (a_k >> 1), kb = b0 + (b_c >> 1);
                ua = ka < blocks ? list[ka] : kNoBlock;
                ub = kb < blocks ? list[kb] : kNoBlock;
            };
            auto copy = [&](uint32_t buf) {  // the step's pieces into its buffer; zero where nothing belongs
                const int s = e & 1;
                const uint16_t* src = p.ops + (size_t)s * p.M * (2 * p.r16) + a_half * p.r16 + block_rank0(ua) + (a_k & 1) * 8;
#pragma unroll
                for (int i = 0; i < kGMaxA; ++i) {
                    const bool in = ids[i] == block_adapter(ua);
                    if (a_row + i * a_step < a_rows)
                        ptx::cp_async16(buf + a_off + (uint32_t)(i * a_step * 128),
                                        in ? src + (size_t)(row0 + a_row + i * a_step) * (2 * p.r16) : p.ops, in ? 16 : 0);
                }
#pragma unroll
                for (int i = 0; i < kGMaxB; ++i) {
                    const int row = b_row + i * b_step;
                    if (row >= b_cols) continue;
                    const uint16_t* pool = p.B + ((size_t)s * p.n_adapters + block_adapter(ub)) * p.r_max * p.NC;
                    // a row of A_a, eight ranks; what lies past the rank is not a number
                    const int j = (b_c & 1) * 8, live = n0 + row < p.NC ? min(8, max(0, block_live(ub) - j)) : 0;
                    ptx::cp_async16(buf + b_off + (uint32_t)(i * b_step * 64),
                                    live ? pool + (size_t)(n0 + row) * p.r_max + block_rank0(ub) + j : p.B, 2 * live);
                }
                ptx::cp_async_commit();
            };
            const uint32_t bufs = base_u + (uint32_t)(p.stages * p.stage_bytes);
            const int ahead = p.lbufs - 1;  // steps copied beyond the one handed over
            uint32_t lb = 0, turn = 0, hb = 0;  // the next step's buffer and its turns; the next to hand over
            int held = 0;                       // steps copied and not handed over
            uint32_t odd = 0, odd_next = 0;     // of the step to hand over and the one behind: pieces of marked adapters
            auto hand_over = [&]() {
                if (odd) {  // their non-finite elements become zero (see operand_kernel)
                    uint8_t* at = smem_raw + (bufs - raw_u) + hb * (uint32_t)p.lora_bytes + b_off;
#pragma unroll
                    for (int i = 0; i < kGMaxB; ++i)
                        if (odd >> i & 1) {
                            uint4* v = reinterpret_cast<uint4*>(at + i * b_step * 64);
                            uint4 w = *v;
                            uint32_t* e = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
                            for (int h = 0; h < 4; ++h) {
                                if ((e[h] & 0x7f80u) == 0x7f80u) e[h] &= 0xffff0000u;
                                if ((e[h] & 0x7f800000u) == 0x7f800000u) e[h] &= 0xffffu;
                            }
                            *v = w;
                        }
                }
                odd = odd_next;
                odd_next = 0;
                ptx::fence_proxy_async_smem();
                ptx::named_sync(2, kGBuilders);
                if (bt == 0) {
                    if (PAIR) ptx::mbar_arrive_remote(leaders(&lfull[hb]));
                    else ptx::mbar_arrive(&lfull[hb]);
                }
                if (++hb == (uint32_t)p.lbufs) hb = 0;
                --held;
            };
            bool more = advance();
            if (more) blocks_of_step();
            while (more) {
                if (turn > 0 && !wait_role(1, kGBuilders, bt == 0, &lempty[lb], (turn - 1) & 1, abort_flag, status, kGStBuild,
                                           p.timeout_ns))
                    break;
                copy(bufs + lb * (uint32_t)p.lora_bytes);
                uint32_t marks = 0;
#pragma unroll
                for (int i = 0; i < kGMaxB; ++i)
                    if (b_row + i * b_step < b_cols && block_bad(ub)) marks |= 1u << i;
                if (held == 0) odd = marks;
                else odd_next = marks;
                if (++lb == (uint32_t)p.lbufs) {
                    lb = 0;
                    ++turn;
                }
                more = advance();
                if (more) blocks_of_step();
                if (++held > ahead) {
                    if (ahead == 0) ptx::cp_async_wait<0>();
                    else ptx::cp_async_wait<1>();
                    hand_over();
                }
            }
            ptx::cp_async_wait<0>();
            while (held > 0) hand_over();  // (after an abort nobody reads them)
        }
    } else {
        // ================================================================ drain
        const int q = warp & 3, half = warp >> 2;
        int acc = 0;
        if (MODE == kGBwd && LORA && p.shared) ptx::pdl_wait();  // the counts were zeroed
        for (Walk w(unit); w.next(p); ++acc) {
            const int row0 = (w.tile % p.mt) * kTokens + rank * kGTileM + q * 32, n0 = (w.tile / p.mt) * p.cols, buf = acc & 1;
            const int row = row0 + lane;
            // the row's place in the outputs
            const int out_row = LORA && p.order && row < p.M ? p.order[row] : row;
            if (!wait_role(3, kGDrainWarps * 32, threadIdx.x == 0, &tfull[buf], (uint32_t)((acc >> 1) & 1), abort_flag, status,
                           kGStDrain, p.timeout_ns))
                break;
            ptx::tc_fence_after();
            const uint32_t ta = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * kGAccCols);
            bool mine = true;  // this CTA finishes the tile
            if (MODE == kGBwd && w.piece >= 0) {
                // a piece of a shared tile, to the workspace; the last one done takes the sum of all
                // back into TMEM (sixteen loads in flight per thread) and finishes the tile
                const int s = w.tile - p.whole;
                const size_t piece4 = (size_t)kCtas * (p.bn / 4) * kGTileM;
                float4* part = reinterpret_cast<float4*>(p.part) + (size_t)s * p.split * piece4 +
                               (size_t)rank * (p.bn / 4) * kGTileM + q * 32 + lane;
                if (row0 < p.M) {
                    float4* dst = part + w.piece * piece4;
                    for (int c = half * 32; c < p.bn; c += 64) {
                        float v[32];
                        ptx::tmem_ld32(ta + (uint32_t)c, v);
                        if (row < p.M)
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                __stcg(dst + (size_t)(c / 4 + i) * kGTileM, make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
                    }
                }
                __threadfence();
                ptx::named_sync(4, kGDrainWarps * 32);
                if (threadIdx.x == 0) s_last = atomicAdd(p.count + s * kCtas + rank, 1) == p.split - 1;
                ptx::named_sync(4, kGDrainWarps * 32);
                mine = s_last;
                if (mine) {
                    __threadfence();
                    if (row0 < p.M)
                        for (int c = half * 16; c < p.bn; c += 32) {
                            float v[16] = {};
                            for (int k0 = 0; k0 < p.split; k0 += 4) {
                                float4 x[4][4];
#pragma unroll
                                for (int k = 0; k < 4; ++k)
#pragma unroll
                                    for (int i = 0; i < 4; ++i)
                                        x[k][i] = k0 + k < p.split
                                                      ? __ldcg(part + (size_t)(k0 + k) * piece4 + (size_t)(c / 4 + i) * kGTileM)
                                                      : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                                for (int k = 0; k < 4; ++k)
#pragma unroll
                                    for (int i = 0; i < 4; ++i) {
                                        v[4 * i] += x[k][i].x;
                                        v[4 * i + 1] += x[k][i].y;
                                        v[4 * i + 2] += x[k][i].z;
                                        v[4 * i + 3] += x[k][i].w;
                                    }
                            }
                            ptx::tmem_st16(ta + (uint32_t)c, v);
                        }
                    ptx::tc_fence_before();
                    ptx::named_sync(4, kGDrainWarps * 32);  // the halves' columns of a row differ below
                    ptx::tc_fence_after();
                }
            }
            // the tile's outputs of this thread's row
            if (mine && row0 < p.M) {  // the warp has live rows
                if (MODE == kGFwd && p.g_codes) {
                    const int nb = (p.NC + act8::kBlock - 1) / act8::kBlock;
                    for (int c = half * 32; c < p.cols; c += 64) {
                        const int col = n0 + c;
                        if (col >= p.NC) break;
                        float g[32], u[32];
                        ptx::tmem_ld32(ta + (uint32_t)c, g);
                        ptx::tmem_ld32(ta + (uint32_t)(p.cols + c), u);
                        if (row < p.M) {
                            const int live = min(32, p.NC - col);
                            const size_t at = (size_t)out_row * p.NC + col, sc = (size_t)out_row * nb + (col >> 5);
                            save_block(g, live, p.g_codes + at, p.g_scales + sc);
                            save_block(u, live, p.u_codes + at, p.u_scales + sc);
#pragma unroll
                            for (int i = 0; i < 32; ++i) g[i] = gate(p.act, g[i]) * u[i];
#pragma unroll
                            for (int i = 0; i < 32; i += 8)
                                if (i < live) store_bf16x8(p.out + at + i, g + i);
                        }
                    }
                } else {
                    constexpr int kN = MODE == kGFwd ? 16 : 32;
                    for (int c = half * kN; c < p.cols; c += 2 * kN) {
                        const int col = n0 + c;
                        if (col >= p.NC) break;
                        float g[kN], u[MODE == kGFwd ? kN : 1];
                        if constexpr (MODE == kGFwd) {
                            ptx::tmem_ld16(ta + (uint32_t)c, g);
                            ptx::tmem_ld16(ta + (uint32_t)(p.cols + c), u);
#pragma unroll
                            for (int i = 0; i < kN; ++i) g[i] = gate(p.act, g[i]) * u[i];
                        } else {
                            ptx::tmem_ld32(ta + (uint32_t)c, g);
                        }
                        if (row < p.M) {
                            uint16_t* o = p.out + (size_t)out_row * p.NC + col;
#pragma unroll
                            for (int i = 0; i < kN; i += 8)
                                if (col + i < p.NC) store_bf16x8(o + i, g + i);
                        }
                    }
                }
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (PAIR) ptx::mbar_arrive_remote(leaders(&tempty[buf]));
                else ptx::mbar_arrive(&tempty[buf]);
            }
        }
    }

    ptx::tc_fence_before();
    if (PAIR) {
        // Both CTAs' roles are done and no more copies are issued. Every copy counts on the leader's
        // barriers: it sees each stage's last fill through before either CTA leaves. After an
        // abort the two producers may differ by one fill; the missing side's bytes are counted
        // here then.
        __syncwarp();
        ptx::cluster_sync();
        if (rank == 0 && threadIdx.x < p.stages) {
            const int s = (int)threadIdx.x;
            const uint32_t mine = s_fills[s], other = ptx::ld_dsmem_u32(ptx::mapa(ptx::smem_u32(&s_fills[s]), 1));
            const uint32_t fills = mine > other ? mine : other;
            if (mine > other) ptx::mbar_complete_tx(&full[s], s_tx[s]);
            if (mine < other) ptx::mbar_arrive_expect_tx(&full[s], ptx::ld_dsmem_u32(ptx::mapa(ptx::smem_u32(&s_tx[s]), 1)));
            if (fills) wait_bar(&full[s], (fills - 1) & 1, abort_flag, status, kGStRing, p.timeout_ns, false);
        }
        __syncwarp();
        ptx::cluster_sync();
    } else {
        __syncthreads();
    }
    if (warp == kGMma) {
        ptx::tc_fence_after();
        if (PAIR) ptx::tmem_dealloc2(tmem, 2 * kGAccCols);
        else ptx::tmem_dealloc(tmem, 2 * kGAccCols);
    }
}

// ------------------------------------------------------------------ tokens by adapter
//
// Rows of x in the segments' order, for the tiles that RowRun calls copied (the GEMM decides the same
// way). A CTA copies kGatherRows rows of 2048 columns, all of them in flight.

constexpr int kGatherThreads = 256, kGatherRows = 16, kGatherCols = kGatherThreads * 8;

__global__ void __launch_bounds__(kGatherThreads)
gather_kernel(const uint16_t* __restrict__ x, const int32_t* __restrict__ order, int M, int K, uint16_t* __restrict__ out)
{
    ptx::pdl_launch_dependents();  // the shrink waits for this kernel to be complete
    ptx::pdl_wait();
    const int row0 = (int)blockIdx.x * kGatherRows, lane = threadIdx.x & 31;
    RowRun run;
    run.load(order, M, row0 / kGTileM * kGTileM, lane);
    if (run.first(M, row0 / kGTileM * kGTileM, lane) >= 0) return;
    const int col = (int)blockIdx.y * kGatherCols + (int)threadIdx.x * 8;
    if (col >= K) return;
    uint4 v[kGatherRows];
#pragma unroll
    for (int i = 0; i < kGatherRows; ++i)
        if (row0 + i < M) v[i] = *reinterpret_cast<const uint4*>(x + (size_t)order[row0 + i] * K + col);
#pragma unroll
    for (int i = 0; i < kGatherRows; ++i)
        if (row0 + i < M) *reinterpret_cast<uint4*>(out + (size_t)(row0 + i) * K + col) = v[i];
}

// ------------------------------------------------------------------ LoRA operands

struct OperandParams {
    struct {
        const float* v;  // `planes` planes of [2][M][r_max], summed in plane order
        int planes;
        uint16_t* ops;
    } side[2];           // backward: blockIdx.y; the lists are made with the first
    long long plane;
    const int32_t* tok_adapter;
    const int32_t* order;  // as the GEMM's
    const int32_t* indptr;
    const int32_t* ranks;
    const float* scales;
    int M, n_adapters, r_max, r16;
    const uint8_t* bad;  // [2][n_adapters][kGatedScanMax], bad_parts of them written (a multiple of 4)
    int bad_parts;
    int tile;  // tokens a list covers: 128 or 256
    int32_t *lists, *list_len, *list_base;
    // forward: the GEMM's steps, see FwdSteps
    int ups, rows, per_tile;
};

constexpr int kOpThreads = 256;
constexpr int kOpRows = 16;   // tokens per CTA: a thread has eight ranks of one of them
static_assert(2 * kOpRows * (LORA_MAX_RANK / 8) <= kOpThreads, "one piece per thread");
constexpr int kPlanesMax = 8;

// Whether the matrix of adapter a and slice s was marked as non-finite.
__device__ __forceinline__ bool marked(const OperandParams& p, int a, int s)
{
    const uint4* at = reinterpret_cast<const uint4*>(p.bad + ((size_t)s * p.n_adapters + a) * kGatedScanMax);
    const uint4 v[2] = {at[0], at[1]};
    const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
    bool bad = false;
#pragma unroll
    for (int k = 0; k < 8; ++k) bad = bad || (4 * k < p.bad_parts && w[k]);
    return bad;
}

__device__ __forceinline__ int rank_of(const OperandParams& p, int a) { return max(1, min(p.ranks ? p.ranks[a] : p.r_max, p.r_max)); }

// The rank blocks that a token tile's rows use, adapters in order of first appearance.
struct TileBlocks {
    alignas(16) int id[kOpThreads];  // per row: its adapter (-1: none),
    int first[kOpThreads];           // the adapter's first block in the list,
    int count[kOpThreads];           // and its blocks (0 without an adapter)
    int warp[kOpThreads / 32];
    int total;
};
// Nothing in it waits for the shrink: the kernels do it before their wait.
__device__ __forceinline__ bool tile_blocks(const OperandParams& p, int m, TileBlocks& t)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, row = m * p.tile + tid;
    int id = tid < p.tile && row < p.M ? p.tok_adapter[p.order ? p.order[row] : row] : -1;
    if (id >= p.n_adapters) id = -1;
    t.id[tid] = id;
    __syncthreads();
    int f = tid;  // the first row of the same adapter
#pragma unroll 8
    for (int j = (tid & ~3) - 4; j >= 0; j -= 4) {
        const int4 o = *reinterpret_cast<const int4*>(t.id + j);
        f = o.x == id ? j : o.y == id ? j + 1 : o.z == id ? j + 2 : o.w == id ? j + 3 : f;
    }
    for (int j = tid - 1; j >= (tid & ~3); --j)
        if (t.id[j] == id && j < f) f = j;
    const int n = id >= 0 ? (rank_of(p, id) + 15) / 16 : 0;
    const int mine = f == tid ? n : 0;
    int at = mine;  // blocks up to this thread's, by a scan over the tile
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, at, o);
        if (lane >= o) at += v;
    }
    if (lane == 31) t.warp[warp] = at;
    __syncthreads();
    int total = 0;
    at -= mine;
    for (int w = 0; w < kOpThreads / 32; ++w) {
        if (w < warp) at += t.warp[w];
        total += t.warp[w];
    }
    t.first[tid] = at;
    t.count[tid] = n;
    if (tid == 0) t.total = total;
    __syncthreads();
    at = t.first[f];
    __syncthreads();
    t.first[tid] = at;
    __syncthreads();
    return mine > 0;
}
// The list, by the threads whose row is its adapter's first.
__device__ __forceinline__ void write_list(const OperandParams& p, int m, const TileBlocks& t, bool first)
{
    if (first) {
        const int id = t.id[threadIdx.x], at = t.first[threadIdx.x], n = t.count[threadIdx.x];
        const int rank = rank_of(p, id);
        int32_t* list = p.lists + (size_t)m * kListMax * (p.tile / kGTileM);
        const int bad = (marked(p, id, 0) ? 1 : 0) | (marked(p, id, 1) ? 2 : 0);
        for (int b = 0; b < n; ++b) list[at + b] = block_code(id, b, min(16, rank - 16 * b), bad);
    }
    if (threadIdx.x == 0) p.list_len[m] = t.total;
}

// Eight ranks of s_a v (columns past the rank zero; NaN for an adapter whose matrix is not finite, so
// that its own tokens show it: the GEMM takes that matrix, or its non-finite elements, as zeros, and
// the other tokens' zeros stay zeros), and their bf16 half hi (h == 0) or lo.
struct Eight {
    float f[8];
    // planes of v; the rank and scale of the token's adapter
    __device__ __forceinline__ void load(const OperandParams& p, const float* planes, int n_planes, int s, int tok, int r, float scale,
                                         int c, bool bad)
    {
        float4 v[kPlanesMax][2];
        const float* src = planes + ((size_t)s * p.M + tok) * p.r_max + 8 * c;
#pragma unroll
        for (int k = 0; k < kPlanesMax; ++k)
            if (k < n_planes && 8 * c < p.r_max) {
                v[k][0] = *reinterpret_cast<const float4*>(src + k * p.plane);
                v[k][1] = *reinterpret_cast<const float4*>(src + k * p.plane + 4);
            }
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = 0.f;
#pragma unroll
        for (int k = 0; k < kPlanesMax; ++k)
            if (k < n_planes && 8 * c < r) {
                f[0] += v[k][0].x; f[1] += v[k][0].y; f[2] += v[k][0].z; f[3] += v[k][0].w;
                f[4] += v[k][1].x; f[5] += v[k][1].y; f[6] += v[k][1].z; f[7] += v[k][1].w;
            }
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = bad ? __uint_as_float(0x7fc00000u) : 8 * c + e < r ? scale * f[e] : 0.f;
    }
    // the values' bf16 half; what it leaves stays
    __device__ __forceinline__ uint4 half()
    {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            w[e] = pack_bf16x2(f[2 * e], f[2 * e + 1]);
            f[2 * e] = rest(f[2 * e], w[e], 0);
            f[2 * e + 1] = rest(f[2 * e + 1], w[e], 16);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    // v less its half, the bf16 at `at` of w: nothing of an infinity or NaN, which the half holds (infinity less
    // infinity would make NaN of it); a finite v that rounds to an infinity takes the largest bf16 as its half.
    static __device__ __forceinline__ float rest(float v, uint32_t& w, int at)
    {
        if ((w >> at & 0x7f80u) == 0x7f80u) {
            if (!act8::finite(v)) return 0.f;
            w -= 1u << at;
        }
        return v - __uint_as_float(w >> at << 16);
    }
};

// Backward: s_a v of both slices as bf16 halves [2][M][hi r16 | lo r16], and the token tiles' lists. Lets
// the GEMM start at once (see the wait there).
__global__ void __launch_bounds__(kOpThreads)
operand_kernel(const OperandParams p)
{
    __shared__ TileBlocks t;
    ptx::pdl_launch_dependents();
    const int tid = threadIdx.x, per = p.tile / kOpRows, m = (int)blockIdx.x / per;
    const bool lists = !blockIdx.y && (int)blockIdx.x % per == 0;  // one CTA of the tile makes its list
    // this thread's eight ranks of a row and slice
    const auto& d = p.side[blockIdx.y];
    const int chunks = p.r16 >> 3, c = tid % chunks, rs = tid / chunks, s = rs & 1, row = (int)blockIdx.x * kOpRows + (rs >> 1);
    int a = -1, tok = 0, r = 0;
    float scale = 1.f;
    if (rs < 2 * kOpRows && row < p.M) {
        tok = p.order ? p.order[row] : row;
        a = p.tok_adapter[tok];
        if (a >= p.n_adapters) a = -1;
        if (a >= 0) {  // (nobody reads the other rows)
            r = rank_of(p, a);
            if (p.scales) scale = p.scales[a];
        }
    }
    const bool first = lists && tile_blocks(p, m, t);
    ptx::pdl_wait();  // from here on what the shrink wrote
    if (a >= 0) {
        Eight v;
        v.load(p, d.v, d.planes, s, tok, r, scale, c, blockIdx.y == 0 && marked(p, a, s));
        uint4* o = reinterpret_cast<uint4*>(d.ops + ((size_t)s * p.M + row) * (2 * p.r16));
        o[c] = v.half();
        o[chunks + c] = v.half();
    }
    if (lists) write_list(p, m, t, first);
}

// Forward: the operand as the GEMM's steps have it, zeros in the blocks of other adapters written out,
// so that a step is a few boxes of the GEMM's ring: step e of a tile is ups / 2 arrays [rows][64] of
// bf16, four groups of 16 columns each (ups of hi, ups of lo; of ups the group of block k / 2 and
// slice k & 1), from array (base + e) ups / 2 on. The bases grow by what the tiles before can need at
// most: tokens that come by adapter have (adapters before the tile's first + tiles before it) R blocks
// at most, R = ceil(r_max / 16); in the caller's order every tile may need per_tile steps.
__global__ void __launch_bounds__(kOpThreads)
expand_kernel(const OperandParams p)
{
    ptx::pdl_launch_dependents();
    __shared__ TileBlocks t;
    __shared__ int s_base;
    const int tid = threadIdx.x, per = p.tile / kOpRows, m = (int)blockIdx.x / per, row0 = (int)blockIdx.x % per * kOpRows;
    if (m * p.tile + row0 >= p.M) return;
    const bool first = tile_blocks(p, m, t);
    const int per_step = p.ups / 2;  // blocks, of both slices
    if (p.per_tile < 0) {
        int before = 0;  // adapters with tokens before the tile's first
        for (int a0 = 0; a0 < t.id[0]; a0 += kOpThreads) {
            const int a = a0 + tid;
            before += __syncthreads_count(a < t.id[0] && p.indptr[a + 1] > p.indptr[a]);
        }
        if (tid == 0) s_base = ((before + m) * (p.r16 >> 4) + (per_step - 1) * m) / per_step;
    } else if (tid == 0) {
        s_base = m * p.per_tile;
    }
    __syncthreads();
    const auto& d = p.side[0];
    const int base = s_base, steps = (t.total + per_step - 1) / per_step, lg = p.ups == 4 ? 4 : 3;
    // where a 16-byte piece of a step's row is: groups of 16 columns, four to an array
    auto piece_at = [&](int e, int piece, int row) {
        return reinterpret_cast<uint4*>(d.ops) + (((size_t)(base + e) * per_step + (piece >> 3)) * p.rows + row) * 8 + (piece & 7);
    };
    for (int i = tid; i < steps * kOpRows << lg; i += kOpThreads) {
        const int piece = i & ((1 << lg) - 1), row = row0 + ((i >> lg) & (kOpRows - 1)), e = (i >> lg) / kOpRows;
        const int b = e * per_step + (((piece >> 1) & (p.ups - 1)) >> 1) - t.first[row];
        if (m * p.tile + row < p.M && (b < 0 || b >= t.count[row])) *piece_at(e, piece, row) = make_uint4(0u, 0u, 0u, 0u);
    }
    // this thread's eight ranks of a row and slice
    const int chunks = p.r16 >> 3, c = tid % chunks, mine = tid / chunks, s = mine & 1, row = row0 + (mine >> 1), pos = m * p.tile + row;
    const bool live = mine < 2 * kOpRows && pos < p.M && (c >> 1) < t.count[row];
    int a = 0, tok = 0, r = 0;
    float scale = 1.f;
    if (live) {
        a = t.id[row];
        tok = p.order ? p.order[pos] : pos;
        r = rank_of(p, a);
        if (p.scales) scale = p.scales[a];
    }
    ptx::pdl_wait();  // from here on what the shrink wrote
    __shared__ float s_v[2 * kOpRows][LORA_MAX_RANK + 4];
    Eight v;
    if (live) {
        v.load(p, d.v, d.planes, s, tok, r, scale, c, marked(p, a, s));
        if (r < p.r16) {  // ranks to their columns
#pragma unroll
            for (int e = 0; e < 8; ++e) s_v[mine][8 * c + e] = v.f[e];
        }
    }
    __syncthreads();
    if (live) {
        if (r < p.r16)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int k = block_rank(r, c >> 1, (c & 1) * 8 + e);
                v.f[e] = k < 0 ? 0.f : s_v[mine][k];
            }
        const int b = t.first[row] + (c >> 1), e = b / per_step, piece = ((b - e * per_step) * 2 + s) * 2 + (c & 1);
        *piece_at(e, piece, row) = v.half();
        *piece_at(e, 2 * p.ups + piece, row) = v.half();
    }
    if (row0 == 0) {
        write_list(p, m, t, first);
        if (tid == 0) p.list_base[m] = base;
    }
}

// The backward's LoRA step buffers beside a ring of enough stages.
int lora_buffers(const GatedParams& p, int room, bool pair)
{
    int n = 1;
    while (n < kGMaxLora && room - (n + 1) * p.lora_bytes >= (pair ? 5 : 4) * p.stage_bytes) ++n;
    return n;
}

template <int MODE, bool LORA, bool PAIR>
cudaError_t launch_mode(const GatedMaps<true>& all, const GatedParams& p, int grid, cudaStream_t stream)
{
    auto kern = gated_gemm_kernel<MODE, LORA, PAIR>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kGSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3(MODE == kGFwd ? kGFwdThreads : kGThreads, 1, 1);
    cfg.dynamicSmemBytes = (size_t)p.smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = PAIR ? 2 : 1;
    GatedMaps<MODE == kGFwd && LORA> maps;
    memcpy(&maps, &all, sizeof(maps));
    return cudaLaunchKernelEx(&cfg, kern, maps, p);
}

// Pairs of CTAs that the current device runs at once (an SM without a partner stays idle).
int pair_count()
{
    static std::atomic<int> cached[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    int n = cached[dev].load(std::memory_order_relaxed);
    if (n) return n > 0 ? n : 0;
    auto kern = gated_gemm_kernel<kGFwd, true, true>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(device_sm_count() / 2 * 2), 1, 1);
    cfg.blockDim = dim3(kGFwdThreads, 1, 1);
    cfg.dynamicSmemBytes = kGSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kGSmem) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1)
        n = -1;
    cached[dev].store(n, std::memory_order_relaxed);
    return n > 0 ? n : 0;
}

// Whether the GEMM takes its tokens by adapter: where it saves a unit some rank blocks, if the batch is
// mixed. Forward: six (the launch costs a sorted batch 1 us and the copy a mixed one 4: 300 tokens
// of 5 adapters, three blocks saved, 30 us without, 34 with; 1024 tokens, seven saved, 66 and 58).
// Backward: twelve (reading rows by the order costs the element-wise kernel 6 us of 32 at 2048 tokens:
// 2 adapters have one block to save; 512 tokens of 48 of rank 32 save 46: 248 us without, 201 with; 2704 of 8
// of rank 64 633 and 551, 611 and 549 if they come sorted).
bool gated_order(const GatedPlan& plan, bool bwd, int M, int n_adapters, int r_max)
{
    if (plan.mt < 2) return false;
    const int R = (r_max + 15) / 16, all = (n_adapters < M ? n_adapters : M) * R;
    return (double)(all - (double)all / plan.mt - R) * plan.tiles / plan.units >= (bwd ? 12 : 6);
}

// A choice of tile: output columns, and the microseconds a CTA or pair takes per stage (64 of K)
// with all of them at work, measured on 2048 tokens, 4096 x 11008. Pairs gain by their deeper ring;
// narrow tiles read their operands from shared memory more often per product, and below 64
// columns a stage takes the same time whatever its width.
struct TileChoice {
    bool pair;
    int cols;
    double us;
};
constexpr TileChoice kFwdTiles[] = {{true, 128, .373}, {true, 96, .309}, {true, 64, .267}, {false, 128, .411},
                                    {false, 96, .329}, {false, 64, .292}, {false, 32, .30}, {false, 112, .364},
                                    {false, 80, .304}, {false, 48, .30}, {false, 16, .30}};
constexpr int kFwdSaveTiles = 7;  // with checkpoints: whole blocks of 32 columns
constexpr TileChoice kBwdTiles[] = {{true, 256, .42}, {true, 128, .357}, {false, 256, .45}, {false, 128, .38}, {false, 64, .336}};
// What a single CTA's tile costs above that next to a pair's. A row pitch off 128 bytes makes each
// row of a load straddle two lines, and a pair loads half as much of B per CTA (2048 x 7624 x 5056
// forward: pairs 275 us, single CTAs 332; backward 512 x 1024 x 5216: 39 and 52). On aligned rows
// the pair is ahead where the table calls it even (937 x 6144 x 9952: 165 us, 174).
constexpr double kSingleCost = 1.03, kSingleSplitRows = 1.3;
// What pieces have to gain: accumulators go out and in, the tail is longer. Found on 4096 x 11008,
// it does not scale with the tile or the pieces, so a product that takes less than this is never shared
// (333 tokens, 1040 x 2768: 18 pairs of 74 at work for 29 us).
constexpr double kShareUs = 40;
constexpr double kPieceUs = 1.2;  // and each more of a tile
constexpr int kMaxSplit = 16, kPieces = 3;  // pieces of a tile; of all tiles per unit, at most

}  // namespace

// The cheapest choice: rounds of the units over the tiles, whole or with the last one shared. A
// single token tile is bound by the weights' stream instead: there time per stage goes by bytes
// (8192 x 28672, 16 tokens: 112 columns in two rounds 6.4 TB/s, 16 columns in thirteen 2 TB/s). A
// pair's one tile is 256 tokens and half as many pairs share the stream (200 x 7424 x 8640: pairs,
// which read the weights once, 53 us, single CTAs 61).
GatedPlan gated_plan(bool bwd, int M, int K, int F, bool save, const lora_pool_t* pool)
{
    const int NC = bwd ? K : F, red = bwd ? 2 * ((F + 63) / 64) : (K + 63) / 64;
    const TileChoice* tiles = bwd ? kBwdTiles : kFwdTiles;
    const int n = bwd ? (int)(sizeof(kBwdTiles) / sizeof(TileChoice)) : (save ? kFwdSaveTiles : (int)(sizeof(kFwdTiles) / sizeof(TileChoice)));
    const int pairs = M > kGTileM ? pair_count() : 0, sms = device_sm_count();
    const double single = K % 64 || (bwd && F % 64) ? kSingleSplitRows : kSingleCost;
    const double weights = 4. * K * F / 6.5e6;  // their stream at 6.5 TB/s: no sharing beats it
    GatedPlan best = {};
    double least = 0;
    for (int i = 0; i < n; ++i) {
        const TileChoice& c = tiles[i];
        const int units = c.pair ? pairs : sms;
        if (units < 1) continue;
        const int mt = (M + (c.pair ? 255 : 127)) / (c.pair ? 256 : 128);
        const long long all = (long long)mt * ((NC + c.cols - 1) / c.cols);
        const double stream = (bwd ? .0028 : .0055) * c.cols / (c.pair ? 2 : 1), work = c.pair || !pairs ? c.us : c.us * single;
        const double us = red * (mt == 1 && stream > work ? stream : work);
        const long long rem = all % units;
        for (int split = 1; split <= kMaxSplit; ++split) {
            if (split > 1 && (!bwd || rem == 0 || rem * split > (long long)kPieces * units || red < 8 * split))
                break;
            const double last = (double)((rem * split + units - 1) / units) / split;
            double t = ((double)(all / units) + last) * us;
            if (split > 1) t = (t < weights ? weights : t) + kShareUs + split * kPieceUs;
            if (best.cols && t >= least) continue;
            least = t;
            best.pair = c.pair;
            best.split = split;
            best.cols = c.cols;
            best.mt = mt;
            best.tiles = (int)all;
            best.units = (int)(split == 1 && all < units ? all : units);
        }
    }
    best.by_adapter = pool && gated_order(best, bwd, M, pool->n_adapters, pool->r_max);
    return best;
}

// Room for the pieces of the backward's shared tiles, and for their counts.
size_t gated_part_bytes() { return (size_t)device_sm_count() * kPieces * kGTileM * kGAccCols * 4; }
size_t gated_count_bytes() { return kGCounts * 4; }
size_t gated_operand_bytes(int M, int r_max)
{
    const size_t r16 = (size_t)(r_max + 15) / 16 * 16;
    return (size_t)2 * M * 2 * r16 * 2;
}
size_t gated_list_bytes(int M)
{
    return (size_t)(M + 2 * kGTileM - 1) / (2 * kGTileM) * 2 * (kListMax + 2) * 4;
}

namespace {

// Steps that expand_kernel's bases may reach, for tiles of `tile` tokens.
size_t gated_steps(int M, int tile, int ups, bool order, int n_adapters, int r_max)
{
    const size_t mt = (size_t)(M + tile - 1) / tile, R = (size_t)(r_max + 15) / 16;
    const size_t all = n_adapters < M ? n_adapters : M, in_tile = all < (size_t)tile ? all : (size_t)tile;
    const size_t per_step = ups / 2;  // blocks
    if (!order) return mt * ((in_tile * R + per_step - 1) / per_step);
    return ((all + mt) * R + (per_step - 1) * mt) / per_step + 1;
}
// Rows of a step's arrays, and their bytes in the ring.
int gated_a_rows(int M) { return M >= kGTileM ? kGTileM : (M + 7) / 8 * 8; }
// The forward's rank blocks per step (both slices counted) and its ring's stage, where a step has to fit: four with few tokens
// (whose operand is short) or where that much is free in a stage, else two.
struct FwdSteps {
    int ups, stage;
};
FwdSteps gated_fwd_steps(const GatedPlan& plan, int M)
{
    const int ctas = plan.pair ? 2 : 1, a = gated_a_rows(M) * 128, stage = a + 2 * plan.cols * 128 / ctas;
    const int four = 2 * a + (plan.cols / ctas + 63) / 64 * 4 * 2048;
    if (four <= stage) return {4, stage};
    if (a <= kGTileM / 2 * 128) return {4, four};
    return {2, stage};
}

}  // namespace

// The largest of what the plans for M tokens need. A batch of several tiles keeps the caller's order only where
// its pool has few rank blocks (gated_order: fewer than 2 (6 + R)).
size_t gated_expand_bytes(int M, int n_adapters, int r_max)
{
    const size_t R = (size_t)(r_max + 15) / 16;
    size_t most = 0;
    for (int tile = kGTileM; tile <= 2 * kGTileM; tile += kGTileM) {
        const size_t rows = M > kGTileM ? tile : gated_a_rows(M);
        const int few = (int)((2 * (6 + R)) / R + 1), kept = M > tile && n_adapters > few ? few : n_adapters;
        for (int ups = 2; ups <= 4; ups += 2) {
            const size_t a = gated_steps(M, tile, ups, false, kept, r_max), b = gated_steps(M, tile, ups, true, n_adapters, r_max);
            const size_t bytes = (a > b ? a : b) * (ups / 2) * rows * 128;
            if (bytes > most) most = bytes;
        }
    }
    return most;
}

size_t gated_gather_bytes(int M, int K) { return M > kGTileM ? (size_t)M * K * 2 : 0; }

cudaError_t launch_gated_gather(const GatedPlan& plan, const void* x, int M, int K, const lora_segments_t& seg, void* out,
                                cudaStream_t stream)
{
    if (!plan.by_adapter) return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((M + kGatherRows - 1) / kGatherRows), (unsigned)((K + kGatherCols - 1) / kGatherCols), 1);
    cfg.blockDim = dim3(kGatherThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, gather_kernel, static_cast<const uint16_t*>(x), (const int32_t*)seg.perm, M, K, static_cast<uint16_t*>(out));
}

cudaError_t launch_gated_operands(const GatedPlan& plan, const GatedSide* sides, int n, int M, const lora_pool_t& pool,
                                  const lora_segments_t& seg, const uint8_t* bad, bool backward, void* lists, cudaStream_t stream)
{
    OperandParams p = {};
    p.tile = plan.pair ? 2 * kGTileM : kGTileM;
    for (int i = 0; i < n; ++i) {
        p.side[i].v = sides[i].v;
        p.side[i].planes = gated_shrink_planes(M, sides[i].down ? pool.h_in : pool.h_out, pool.n_adapters);
        p.side[i].ops = static_cast<uint16_t*>(sides[i].ops);
    }
    p.plane = (long long)pool.n_slices * M * pool.r_max;
    p.bad = bad;
    p.bad_parts = gated_scan_parts(sides[0].down, M, pool);
    p.tok_adapter = seg.tok_adapter;
    if (plan.by_adapter) p.order = seg.perm;
    p.indptr = seg.indptr;
    p.ranks = pool.ranks;
    p.scales = pool.scales;
    p.M = M;
    p.n_adapters = pool.n_adapters;
    p.r_max = pool.r_max;
    p.r16 = (pool.r_max + 15) / 16 * 16;
    p.lists = static_cast<int32_t*>(lists);
    p.list_len = p.lists + (size_t)plan.mt * kListMax * (p.tile / kGTileM);
    p.list_base = p.list_len + plan.mt;
    if (!backward) {
        p.ups = gated_fwd_steps(plan, M).ups;
        p.rows = plan.pair ? 2 * kGTileM : gated_a_rows(M);
        p.per_tile = plan.by_adapter ? -1 : (int)(gated_steps(M, p.tile, p.ups, false, pool.n_adapters, pool.r_max) / plan.mt);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(plan.mt * (p.tile / kOpRows)), (unsigned)n, 1);
    cfg.blockDim = dim3(kOpThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return backward ? cudaLaunchKernelEx(&cfg, operand_kernel, p) : cudaLaunchKernelEx(&cfg, expand_kernel, p);
}

cudaError_t launch_gated_gemm(const GatedPlan& plan, const GatedGemmArgs& a, cudaStream_t stream)
{
    const bool bwd = a.backward;
    GatedParams p = {};
    p.M = a.M;
    p.NC = bwd ? a.K : a.F;
    const bool save = a.g8 != nullptr;
    p.mt = plan.mt;
    p.cols = plan.cols;
    p.bn = bwd ? p.cols : 2 * p.cols;
    p.tiles = plan.tiles;
    p.units = plan.units;
    p.split = plan.split;
    p.rounds = plan.split > 1 ? plan.tiles / plan.units : (plan.tiles + plan.units - 1) / plan.units;
    p.whole = plan.whole();
    p.shared = plan.tiles - p.whole;
    p.part = a.part;
    p.count = a.count;
    const int red = bwd ? a.F : a.K;
    p.kb_half = (red + kGKBlock - 1) / kGKBlock;
    p.kb = bwd ? 2 * p.kb_half : p.kb_half;
    // few tokens: only their rows (in eights) are loaded; the MMA's other rows read whatever
    // the shared memory holds and land in accumulator rows that nobody drains
    const int a_rows = gated_a_rows(a.M);
    p.a_bytes = a_rows * 128;
    p.b_bytes = p.bn * 128 / (plan.pair ? 2 : 1);
    p.stage_bytes = p.a_bytes + p.b_bytes;
    // Many tokens take all shared memory. Few leave some of it, so that the small kernels before this
    // one keep running beside its CTAs (which then start at once, the weights streaming under the
    // shrink). At the end: what the MMA may read past a short operand tile.
    p.smem = a_rows > kGTileM / 2 ? kGSmem : kGSmemShort;
    int room = p.smem - (kGTileM - a_rows) * 128 - kGBarBytes - 1024;
    if (a.lora && !bwd) {
        const FwdSteps f = gated_fwd_steps(plan, a.M);
        p.ups = f.ups;
        p.stage_bytes = f.stage;
    } else if (a.lora) {
        p.r16 = (a.r_max + 15) / 16 * 16;
        p.ups = 2;  // what four pieces per builder and the space beside four stages hold
        p.lora_bytes = (int)lora_b_offset(p) + p.cols / (plan.pair ? 2 : 1) * 64;
        p.lora_bytes = (p.lora_bytes + 1023) / 1024 * 1024;
        p.lbufs = lora_buffers(p, room, plan.pair);
        room -= p.lbufs * p.lora_bytes;
    }
    p.stages = room / p.stage_bytes;
    if (p.stages > kGMaxStages) p.stages = kGMaxStages;
    p.act = a.act;
    p.out = static_cast<uint16_t*>(a.out);
    if (save) {
        p.g_codes = a.g8->codes;
        p.g_scales = a.g8->scales;
        p.u_codes = a.u8->codes;
        p.u_scales = a.u8->scales;
    }
    p.status = a.status;
    p.timeout_ns = debug_wait_limit_ns();
    p.inject_stall = debug_inject_stall();
    if (a.lora) {
        p.ops = static_cast<const uint16_t*>(a.ops);
        p.B = static_cast<const uint16_t*>(a.B);
        p.lists = static_cast<const int32_t*>(a.lists);
        p.list_len = p.lists + (size_t)p.mt * kListMax * (plan.pair ? 2 : 1);
        p.list_base = p.list_len + p.mt;
        p.tok_adapter = a.tok_adapter;
        if (plan.by_adapter) p.order = a.order;
        p.n_adapters = a.n_adapters;
        p.r_max = a.r_max;
    }
    GatedMaps<true> maps;
    const CUtensorMapDataType dt = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
    bool ok = true;
    for (int i = 0; i < 2; ++i) {
        ok = ok && encode_tmap_2d(&maps.a[i], dt, bwd || p.order ? a.a[i] : a.a[0], (uint64_t)red, (uint64_t)a.M, (uint64_t)red * 2,
                                  kGKBlock, (uint32_t)a_rows, sw);
        ok = ok && encode_tmap_2d(&maps.b[i], dt, a.W[i], (uint64_t)a.K, (uint64_t)a.F, (uint64_t)a.K * 2, kGKBlock,
                                  bwd ? kGKBlock : (uint32_t)p.cols, sw);
    }
    if (a.lora && !bwd) {
        const size_t rows = plan.pair ? 2 * kGTileM : a_rows;
        const size_t steps = gated_steps(a.M, plan.pair ? 2 * kGTileM : kGTileM, p.ups, p.order != nullptr, a.n_adapters, a.r_max);
        ok = ok && encode_tmap_2d(&maps.e, dt, a.ops, 64, steps * (p.ups / 2) * rows, 128, 64, (uint32_t)a_rows, sw);
        const uint64_t dims[3] = {(uint64_t)a.F, (uint64_t)a.r_max, (uint64_t)(2 * a.n_adapters)};
        const uint64_t strides[2] = {(uint64_t)a.F * 2, (uint64_t)a.F * a.r_max * 2};
        for (int b = 0; b < kRankBoxes; ++b) {
            const uint32_t box[3] = {64, 1u << b, 1};
            ok = ok && encode_tmap_3d(&maps.l[b], dt, a.B, dims, strides, box, sw);
        }
    }
    if (!ok) return cudaErrorInvalidValue;
    const int grid = p.units * (plan.pair ? 2 : 1);
    if (plan.pair) {
        if (bwd) return a.lora ? launch_mode<kGBwd, true, true>(maps, p, grid, stream) : launch_mode<kGBwd, false, true>(maps, p, grid, stream);
        return a.lora ? launch_mode<kGFwd, true, true>(maps, p, grid, stream) : launch_mode<kGFwd, false, true>(maps, p, grid, stream);
    }
    if (bwd) return a.lora ? launch_mode<kGBwd, true, false>(maps, p, grid, stream) : launch_mode<kGBwd, false, false>(maps, p, grid, stream);
    return a.lora ? launch_mode<kGFwd, true, false>(maps, p, grid, stream) : launch_mode<kGFwd, false, false>(maps, p, grid, stream);
}

}  // namespace lora
