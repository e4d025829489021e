// kda_fp8.cuh -- 8-bit activations: e4m3 codes with one fp32 scale for each
// token and block of 128 channels.
//
//   s = max(max |y|, 2^-96) / 448,  code = e4m3(y / s)   over a block's channels
//
// 448 is the largest e4m3 value, so a block's largest channel keeps full
// range. The floor 2^-96 keeps a block of zeros (codes 0) at a normal scale
// whose reciprocal is finite. A NaN stays in its own channel: the maximum
// ignores it and its code is NaN. An infinity makes the block's scale infinite.
#pragma once

#include <cuda_fp8.h>

#include "kda_common.cuh"

namespace kda {

constexpr int QBLOCK = 128;       // channels per scale
constexpr float QMAX = 448.f;     // largest e4m3 value
constexpr float QAMAX_MIN = 0x1p-96f;

// 1 / sqrt(den) with 0 for a row whose mean square plus eps is exactly zero;
// a NaN in the row makes it NaN. The hardware reciprocal root is off by less
// than 2^-22 and takes one instruction; the exact root and division took a
// tenth of the gated norm's.
__device__ __forceinline__ float rms_inv(float den) { return den == 0.f ? 0.f : rsqrtf(den); }

// A block's scale max / 448 and its reciprocal. The product with 1 / 448 and
// the hardware reciprocal (1 ulp) stand in for two divisions; the factor 2^-8
// keeps the reciprocal of the largest fp32 values normal.
__device__ __forceinline__ float block_scale(float m) { return m * (1.0f / QMAX); }
__device__ __forceinline__ float block_inv(float m) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(m * 0x1p-8f));
    return r * (QMAX * 0x1p-8f);
}

// 8 consecutive channels of one thread, loaded as fp32.
template <typename T> struct Raw8;
template <> struct Raw8<__nv_bfloat16> { uint4 v; };
template <> struct Raw8<float> { float4 a, b; };

__device__ __forceinline__ void load8(const __nv_bfloat16 *p, Raw8<__nv_bfloat16> &r) {
    r.v = __ldcs(reinterpret_cast<const uint4 *>(p));
}
__device__ __forceinline__ void load8(const float *p, Raw8<float> &r) {
    r.a = __ldcs(reinterpret_cast<const float4 *>(p));
    r.b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
}
__device__ __forceinline__ void unpack8(const Raw8<__nv_bfloat16> &r, float (&f)[8]) {
    const uint32_t w[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // a bf16 is the upper half of its fp32
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void unpack8(const Raw8<float> &r, float (&f)[8]) {
    f[0] = r.a.x; f[1] = r.a.y; f[2] = r.a.z; f[3] = r.a.w;
    f[4] = r.b.x; f[5] = r.b.y; f[6] = r.b.z; f[7] = r.b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        memcpy(&w[i], &b, 4);
    }
    __stcs(reinterpret_cast<uint4 *>(p), make_uint4(w[0], w[1], w[2], w[3]));
}
__device__ __forceinline__ void store8(float *p, const float (&f)[8]) {
    __stcs(reinterpret_cast<float4 *>(p), make_float4(f[0], f[1], f[2], f[3]));
    __stcs(reinterpret_cast<float4 *>(p) + 1, make_float4(f[4], f[5], f[6], f[7]));
}

// Largest |y| of a block whose 128 channels lie 8 each in 16 neighbouring
// lanes (a channel past the row's end holds 0). All 32 lanes call.
__device__ __forceinline__ float block_amax(const float (&y)[8]) {
    float m = QAMAX_MIN;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(y[i]));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}

// The 8 codes of y / s, with inv = 1 / s: products in fp32, then one rounding
// to e4m3 (inv's own rounding can only move a value that lies within an ulp
// of a border between two codes).
__device__ __forceinline__ uint2 codes8(const float (&y)[8], float inv) {
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        c[i] = __nv_cvt_float2_to_fp8x2(make_float2(y[2 * i] * inv, y[2 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

}  // namespace kda
