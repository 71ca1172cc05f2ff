// act8.cu -- 8-bit activation checkpoints (format: act8.cuh): compressing bf16 rows
// and expanding them again.
//
// Both are bound by HBM: 3 1/32 bytes per element either way. A warp takes a task of
// 256 columns of one row, 8 columns (16 bytes of bf16, 8 of codes) per lane, so that
// every load and store of a warp is one contiguous run; four lanes share a block's
// scale, and its amax takes two shuffles. A warp has four tasks' loads in flight
// before it works on the first.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "act8.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace lora {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTaskCols = 256;
constexpr int kInFlight = 4;
constexpr int kCtasPerSm = 8;

__device__ __forceinline__ uint32_t abs2(uint32_t w) { return w & 0x7fff7fffu; }

// Eight bf16 (one lane's chunk) -> eight codes; writes the block's scale code to E. Every
// lane of the warp calls it (shuffles within groups of four); lanes past the row hold zeros.
__device__ __forceinline__ uint2 compress_chunk(const uint4 c, uint32_t& E)
{
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    // magnitudes compare as 16-bit integers; infinities and NaN are 0x7f80 and above
    uint32_t m = __vmaxu2(__vmaxu2(abs2(w[0]), abs2(w[1])), __vmaxu2(abs2(w[2]), abs2(w[3])));
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
    uint32_t top = max(m & 0xffffu, m >> 16);
    const bool odd = top >= 0x7f80u;  // the block holds a non-finite element
    if (__any_sync(0xffffffffu, odd)) {
        uint32_t t = 0;  // the largest finite magnitude
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = w[i] & 0x7fffu, hi = (w[i] >> 16) & 0x7fffu;
            t = max(t, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
        }
        t = max(t, __shfl_xor_sync(0xffffffffu, t, 1));
        t = max(t, __shfl_xor_sync(0xffffffffu, t, 2));
        top = t;
    }
    E = act8::scale_code(__uint_as_float(top << 16));
    const float inv = act8::inv_scale(E);
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = odd ? act8::scaled(v[i], inv) : v[i] * inv;
    uint2 o;
    o.x = (uint32_t)ptx::cvt_e4m3x2(v[0], v[1]) | ((uint32_t)ptx::cvt_e4m3x2(v[2], v[3]) << 16);
    o.y = (uint32_t)ptx::cvt_e4m3x2(v[4], v[5]) | ((uint32_t)ptx::cvt_e4m3x2(v[6], v[7]) << 16);
    return o;
}

// Eight codes of a block of scale code E -> eight bf16, rounded once (exact unless subnormal).
__device__ __forceinline__ uint4 expand_chunk(const uint2 c, uint32_t E)
{
    const float X = act8::scale_value(E);
    float v[8];
    act8::decode4(c.x, v);
    act8::decode4(c.y, v + 4);
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i] * X, v[2 * i + 1] * X);
        o[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// Tasks t = row * segs + seg; segs = ceil(N / 256).
__global__ void __launch_bounds__(kThreads)
act8_compress_kernel(const uint16_t* __restrict__ x, int N, uint32_t tasks, uint32_t segs, uint8_t* __restrict__ codes,
                     uint8_t* __restrict__ scales)
{
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const uint32_t stride = gridDim.x * kWarps, nb = (uint32_t)((N + act8::kBlock - 1) / act8::kBlock);
    for (uint64_t t0 = blockIdx.x * kWarps + (threadIdx.x >> 5); t0 < tasks; t0 += (uint64_t)stride * kInFlight) {
        uint4 c[kInFlight];
        uint32_t row[kInFlight];
        int col[kInFlight];  // -1: nothing here
#pragma unroll
        for (int i = 0; i < kInFlight; ++i) {
            const uint64_t t = t0 + (uint64_t)i * stride;
            c[i] = make_uint4(0u, 0u, 0u, 0u);
            col[i] = -1;
            if (t < tasks) {
                row[i] = (uint32_t)t / segs;
                const int at = (int)((uint32_t)t - row[i] * segs) * kTaskCols + lane * 8;
                if (at < N) {
                    col[i] = at;
                    c[i] = __ldcs(reinterpret_cast<const uint4*>(x + (size_t)row[i] * N + at));
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kInFlight; ++i) {
            uint32_t E;
            const uint2 o = compress_chunk(c[i], E);
            if (col[i] >= 0) {
                *reinterpret_cast<uint2*>(codes + (size_t)row[i] * N + col[i]) = o;
                if ((lane & 3) == 0) scales[(size_t)row[i] * nb + (col[i] >> 5)] = (uint8_t)E;
            }
        }
    }
}

__global__ void __launch_bounds__(kThreads)
act8_expand_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int N, uint32_t tasks,
                   uint32_t segs, uint16_t* __restrict__ x)
{
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const uint32_t stride = gridDim.x * kWarps, nb = (uint32_t)((N + act8::kBlock - 1) / act8::kBlock);
    for (uint64_t t0 = blockIdx.x * kWarps + (threadIdx.x >> 5); t0 < tasks; t0 += (uint64_t)stride * kInFlight) {
        uint2 c[kInFlight];
        uint32_t E[kInFlight];
        size_t out[kInFlight];
        bool live[kInFlight];
#pragma unroll
        for (int i = 0; i < kInFlight; ++i) {
            const uint64_t t = t0 + (uint64_t)i * stride;
            live[i] = false;
            if (t < tasks) {
                const uint32_t row = (uint32_t)t / segs;
                const int at = (int)((uint32_t)t - row * segs) * kTaskCols + lane * 8;
                if (at < N) {
                    live[i] = true;
                    out[i] = (size_t)row * N + at;
                    c[i] = __ldcs(reinterpret_cast<const uint2*>(codes + out[i]));
                    E[i] = scales[(size_t)row * nb + (at >> 5)];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kInFlight; ++i)
            if (live[i]) *reinterpret_cast<uint4*>(x + out[i]) = expand_chunk(c[i], E[i]);
    }
}

template <typename... P, typename... A>
cudaError_t launch_tasks(void (*kern)(P...), uint32_t tasks, cudaStream_t stream, A... args)
{
    const uint32_t most = (uint32_t)device_sm_count() * kCtasPerSm;
    const uint32_t need = (tasks + kWarps - 1) / kWarps;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(need < most ? need : most, 1, 1);
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

// tasks of 256 columns; M * segs < 2^31 for every array that fits the device (checked by api.cu)
cudaError_t launch_act8_compress(const void* x, int M, int N, const lora_act8_t& out, cudaStream_t stream)
{
    const uint32_t segs = (uint32_t)((N + kTaskCols - 1) / kTaskCols), tasks = (uint32_t)M * segs;
    return launch_tasks(act8_compress_kernel, tasks, stream, static_cast<const uint16_t*>(x), N, tasks, segs, out.codes,
                        out.scales);
}

cudaError_t launch_act8_expand(const lora_act8_t& in, int M, int N, void* x, cudaStream_t stream)
{
    const uint32_t segs = (uint32_t)((N + kTaskCols - 1) / kTaskCols), tasks = (uint32_t)M * segs;
    return launch_tasks(act8_expand_kernel, tasks, stream, static_cast<const uint8_t*>(in.codes),
                        static_cast<const uint8_t*>(in.scales), N, tasks, segs, static_cast<uint16_t*>(x));
}

}  // namespace lora
