// act8.cu -- 8-bit activation checkpoints (format: act8.cuh): compressing bf16 rows
// and expanding them again.
//
// Both are bound by HBM: 3 1/32 bytes per element either way. A warp takes a task of
// 512 columns of one row, 16 columns (32 bytes of bf16, 16 of codes) per lane, so that
// every load and store of a warp is one contiguous run; two lanes share a block's scale, and
// its amax takes one shuffle. A warp has two tasks' loads in flight before it works on the
// first. Packed arithmetic (two bf16 per instruction up to the conversion) keeps the
// instructions per element low: with 8 columns per lane in fp32 they, not HBM, had set the
// pace.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "act8.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace lora {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kLaneCols = 16;
constexpr int kTaskCols = 32 * kLaneCols;
constexpr int kInFlight = 2;

__device__ __forceinline__ uint32_t abs2(uint32_t w) { return w & 0x7fff7fffu; }

// 32 bytes at a 16-byte aligned address, as one access where the rows are 32-byte aligned.
template <bool A32>
__device__ __forceinline__ void load32(const void* src, uint32_t* w)
{
    if (A32) {
        asm volatile("ld.global.cs.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                     : "l"(src));
    } else {
        const uint4 a = __ldcs(static_cast<const uint4*>(src)), b = __ldcs(static_cast<const uint4*>(src) + 1);
        w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
        w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
    }
}
template <bool A32>
__device__ __forceinline__ void store32(void* dst, const uint32_t* w)
{
    if (A32) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                     "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        static_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        static_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b)
{
    const __nv_bfloat162 r = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}

// Sixteen bf16 (one lane's piece) -> sixteen codes; writes the block's scale code to E. Every
// lane of the warp calls it (a shuffle between neighbours); lanes past the row hold zeros.
__device__ __forceinline__ uint4 compress_piece(uint32_t* w, uint32_t& E)
{
    // magnitudes compare as 16-bit integers; infinities and NaN are 0x7f80 and above
    uint32_t m = abs2(w[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) m = __vmaxu2(m, abs2(w[i]));
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
    uint32_t top = max(m & 0xffffu, m >> 16);
    if (__any_sync(0xffffffffu, top >= 0x7f80u)) {
        // some block holds a non-finite element: the largest finite magnitude, and NaN for what is not
        uint32_t t = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t lo = w[i] & 0x7fffu, hi = (w[i] >> 16) & 0x7fffu;
            t = max(t, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
            w[i] |= (lo >= 0x7f80u ? 0x7fffu : 0u) | (hi >= 0x7f80u ? 0x7fff0000u : 0u);
        }
        top = max(t, __shfl_xor_sync(0xffffffffu, t, 1));
    }
    E = act8::scale_code(__uint_as_float(top << 16));
    const uint32_t inv = __float_as_uint(act8::inv_scale(E)), inv2 = inv | inv >> 16;  // a power of two: its bf16 twice
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t a = mul2(w[2 * i], inv2), b = mul2(w[2 * i + 1], inv2);  // exact: powers of two
        o[i] = (uint32_t)ptx::cvt_e4m3x2(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u)) |
               ((uint32_t)ptx::cvt_e4m3x2(__uint_as_float(b << 16), __uint_as_float(b & 0xffff0000u)) << 16);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// Sixteen codes of a block of scale code E -> sixteen bf16, rounded once (exact unless subnormal).
__device__ __forceinline__ void expand_piece(const uint4 c, uint32_t E, uint32_t* o)
{
    const float X = act8::scale_value(E);
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float v[4];
        act8::decode4(w[i], v);
        const __nv_bfloat162 a = __floats2bfloat162_rn(v[0] * X, v[1] * X), b = __floats2bfloat162_rn(v[2] * X, v[3] * X);
        o[2 * i] = *reinterpret_cast<const uint32_t*>(&a);
        o[2 * i + 1] = *reinterpret_cast<const uint32_t*>(&b);
    }
}

// Tasks t = row * segs + seg; segs = ceil(N / 512).
template <bool A32>
__global__ void __launch_bounds__(kThreads)
act8_compress_kernel(const uint16_t* __restrict__ x, int N, uint32_t tasks, uint32_t segs, uint8_t* __restrict__ codes,
                     uint8_t* __restrict__ scales)
{
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const uint32_t stride = gridDim.x * kWarps, nb = (uint32_t)((N + act8::kBlock - 1) / act8::kBlock);
    for (uint64_t t0 = blockIdx.x * kWarps + (threadIdx.x >> 5); t0 < tasks; t0 += (uint64_t)stride * kInFlight) {
        uint32_t w[kInFlight][8];
        uint32_t row[kInFlight];
        int col[kInFlight];  // -1: nothing here
#pragma unroll
        for (int i = 0; i < kInFlight; ++i) {
            const uint64_t t = t0 + (uint64_t)i * stride;
#pragma unroll
            for (int e = 0; e < 8; ++e) w[i][e] = 0u;
            col[i] = -1;
            if (t < tasks) {
                row[i] = (uint32_t)t / segs;
                const int at = (int)((uint32_t)t - row[i] * segs) * kTaskCols + lane * kLaneCols;
                if (at < N) {
                    col[i] = at;
                    load32<A32>(x + (size_t)row[i] * N + at, w[i]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kInFlight; ++i) {
            uint32_t E;
            const uint4 o = compress_piece(w[i], E);
            if (col[i] >= 0) {
                *reinterpret_cast<uint4*>(codes + (size_t)row[i] * N + col[i]) = o;
                if ((lane & 1) == 0) scales[(size_t)row[i] * nb + (col[i] >> 5)] = (uint8_t)E;
            }
        }
    }
}

template <bool A32>
__global__ void __launch_bounds__(kThreads)
act8_expand_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int N, uint32_t tasks,
                   uint32_t segs, uint16_t* __restrict__ x)
{
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const uint32_t stride = gridDim.x * kWarps, nb = (uint32_t)((N + act8::kBlock - 1) / act8::kBlock);
    for (uint64_t t0 = blockIdx.x * kWarps + (threadIdx.x >> 5); t0 < tasks; t0 += (uint64_t)stride * kInFlight) {
        uint4 c[kInFlight];
        uint32_t E[kInFlight];
        size_t out[kInFlight];
        bool live[kInFlight];
#pragma unroll
        for (int i = 0; i < kInFlight; ++i) {
            const uint64_t t = t0 + (uint64_t)i * stride;
            live[i] = false;
            if (t < tasks) {
                const uint32_t row = (uint32_t)t / segs;
                const int at = (int)((uint32_t)t - row * segs) * kTaskCols + lane * kLaneCols;
                if (at < N) {
                    live[i] = true;
                    out[i] = (size_t)row * N + at;
                    c[i] = __ldcs(reinterpret_cast<const uint4*>(codes + out[i]));
                    E[i] = scales[(size_t)row * nb + (at >> 5)];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kInFlight; ++i)
            if (live[i]) {
                uint32_t o[8];
                expand_piece(c[i], E[i], o);
                store32<A32>(x + out[i], o);
            }
    }
}

template <typename... P, typename... A>
cudaError_t launch_tasks(void (*kern)(P...), uint32_t tasks, cudaStream_t stream, A... args)
{
    // a warp per task while that fills the SMs once, then kInFlight tasks per warp: many small CTAs
    // end more evenly than a grid of resident ones walking the rest (30.7 -> 28 us for the pair at
    // 2704 x 11008)
    const uint32_t one = (tasks + kWarps - 1) / kWarps, all = (one + kInFlight - 1) / kInFlight;
    const uint32_t fill = (uint32_t)device_sm_count() * 4;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(one < fill ? one : (all < fill ? fill : all), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace

// M * segs < 2^31 for every array that fits the device (checked by api.cu)
cudaError_t launch_act8_compress(const void* x, int M, int N, const lora_act8_t& out, cudaStream_t stream)
{
    const uint32_t segs = (uint32_t)((N + kTaskCols - 1) / kTaskCols), tasks = (uint32_t)M * segs;
    const bool a32 = (reinterpret_cast<uintptr_t>(x) & 31) == 0;  // N % 16 == 0: then every row is
    return launch_tasks(a32 ? act8_compress_kernel<true> : act8_compress_kernel<false>, tasks, stream,
                        static_cast<const uint16_t*>(x), N, tasks, segs, out.codes, out.scales);
}

cudaError_t launch_act8_expand(const lora_act8_t& in, int M, int N, void* x, cudaStream_t stream)
{
    const uint32_t segs = (uint32_t)((N + kTaskCols - 1) / kTaskCols), tasks = (uint32_t)M * segs;
    const bool a32 = (reinterpret_cast<uintptr_t>(x) & 31) == 0;
    return launch_tasks(a32 ? act8_expand_kernel<true> : act8_expand_kernel<false>, tasks, stream,
                        static_cast<const uint8_t*>(in.codes), static_cast<const uint8_t*>(in.scales), N, tasks, segs,
                        static_cast<uint16_t*>(x));
}

}  // namespace lora
