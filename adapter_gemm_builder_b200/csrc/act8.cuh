// act8.cuh -- the 8-bit activation checkpoint format, shared by the kernels that
// write it (act8.cu, the gated GEMM's epilogue) and read it (act8.cu, gated_grad.cu).
//
// A row is cut into blocks of 32 columns (the last may be shorter). The block's scale
// is the smallest power of two X = 2^p with amax <= 448 X, amax over its finite
// elements, stored as an E8M0 byte E = p + 127 clamped to 0..254 (0 when amax is 0);
// an element's code is E4M3(v / X), round to nearest even: nothing saturates, v / X is
// exact (a power of two), and code times X has four significant bits, so bf16 holds it
// exactly unless it is subnormal there. A non-finite element is stored as NaN (E4M3 has
// no infinity) and does not touch its block's scale.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "ptx.cuh"

namespace lora {
namespace act8 {

constexpr int kBlock = 32;

// E of a block whose largest finite magnitude is amax >= 0 (fp32 bits): 448 = 1.75 2^8,
// so p = exponent - 8, one more when the significand is past 1.75.
__device__ __forceinline__ uint32_t scale_code(float amax)
{
    const uint32_t b = __float_as_uint(amax);
    const int e = (int)(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
    return (uint32_t)max(e, 0);
}
// 2^(127 - E), what an element is multiplied by before the rounding (E <= 247 here).
__device__ __forceinline__ float inv_scale(uint32_t E) { return __uint_as_float((254u - E) << 23); }
// X = 2^(E - 127) (E = 0: subnormal; 255: NaN, as E8M0 has it).
__device__ __forceinline__ float scale_value(uint32_t E)
{
    return __uint_as_float(E == 0 ? 0x00400000u : (E == 255 ? 0x7fc00000u : E << 23));
}
__device__ __forceinline__ bool finite(float v) { return (__float_as_uint(v) & 0x7f800000u) != 0x7f800000u; }
// v times the scale's inverse, NaN for an infinite v (whose conversion would saturate).
__device__ __forceinline__ float scaled(float v, float inv)
{
    return finite(v) ? v * inv : __uint_as_float(0x7fc00000u);
}
// Four E4M3 codes (byte i the i-th) -> fp32 values.
__device__ __forceinline__ void decode4(uint32_t w, float* v)
{
    uint32_t h0, h1;
    asm("{\n.reg .b16 lo, hi;\nmov.b32 {lo, hi}, %2;\ncvt.rn.f16x2.e4m3x2 %0, lo;\ncvt.rn.f16x2.e4m3x2 %1, hi;\n}"
        : "=r"(h0), "=r"(h1) : "r"(w));
    asm("{\n.reg .f16 l, h;\nmov.b32 {l, h}, %2;\ncvt.f32.f16 %0, l;\ncvt.f32.f16 %1, h;\n}" : "=f"(v[0]), "=f"(v[1]) : "r"(h0));
    asm("{\n.reg .f16 l, h;\nmov.b32 {l, h}, %2;\ncvt.f32.f16 %0, l;\ncvt.f32.f16 %1, h;\n}" : "=f"(v[2]), "=f"(v[3]) : "r"(h1));
}

}  // namespace act8
}  // namespace lora
