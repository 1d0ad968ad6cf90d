// gdr_kv8.cuh -- the 8-bit paged cache: codes, scales and addressing shared by the kernels
// that write it (gdr_kv8_append.cu) and read it (gdr_kv8_split.cuh, gdr_kv8_tile.cuh).
//
// Keys and values are two arrays of codes [num_pages][Hkv][page][D] (e4m3 or int8) with fp32
// scales [num_pages][Hkv]: value = code * scale.  A (page, head) block of page * D bytes is
// contiguous.  The writer's scales are powers of two: rescaling a code is then an exponent
// shift (exact but for the final rounding), and quantising divides exactly.
#pragma once

#include "gdr_internal.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>

namespace gdr {
namespace {

constexpr int kScaleMinExp = -40, kScaleMaxExp = 40;

// The least power of two s with amax <= Qmax s (Qmax = 448 = 1.75 2^8 for e4m3, 127 =
// 1.984375 2^6 for int8), within [2^-40, 2^40].  amax is finite and >= 0.
template <Kv8 KV>
__device__ __forceinline__ float scale_for(float amax) {
    const uint32_t u = __float_as_uint(amax);
    constexpr uint32_t mant = KV == Kv8::E4M3 ? 0x600000u : 0x7e0000u;   // Qmax's fraction bits
    constexpr int qexp = KV == Kv8::E4M3 ? 8 : 6;
    int e = (int)(u >> 23) - 127 - qexp + ((u & 0x7fffffu) > mant ? 1 : 0);
    e = min(max(e, kScaleMinExp), kScaleMaxExp);   // zero and subnormal maxima land at the least
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Code of y = x / scale: round to nearest even, saturate; NaN gives 0.
template <Kv8 KV>
__device__ __forceinline__ uint32_t encode2(float y0, float y1) {   // two codes, low byte first
    y0 = y0 == y0 ? y0 : 0.f;
    y1 = y1 == y1 ? y1 : 0.f;
    if (KV == Kv8::E4M3)
        return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(y0, y1), __NV_SATFINITE, __NV_E4M3);
    const int a = __float2int_rn(fminf(fmaxf(y0, -127.f), 127.f));
    const int b = __float2int_rn(fminf(fmaxf(y1, -127.f), 127.f));
    return ((uint32_t)a & 0xffu) | (((uint32_t)b & 0xffu) << 8);
}

// The two halves of two codes (low byte first), exactly.
template <Kv8 KV>
__device__ __forceinline__ uint32_t decode2_h(uint32_t c) {
    if (KV == Kv8::E4M3) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c & 0xffffu), __NV_E4M3);
        return (uint32_t)h.x | ((uint32_t)h.y << 16);
    }
    // 1024 + (code + 128) as a half is 0x6400 | biased byte; subtracting 1152 leaves the code
    const uint32_t b = __byte_perm(c ^ 0x8080u, 0x64646464u, 0x4140);
    const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&b), __float2half2_rn(1152.f));
    return *reinterpret_cast<const uint32_t *>(&r);
}
// The halves of the four codes of a word.
template <Kv8 KV>
__device__ __forceinline__ void decode4_h(uint32_t w, uint32_t &lo, uint32_t &hi) {
    if (KV == Kv8::E4M3) {
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
            "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
    } else {
        const uint32_t c = w ^ 0x80808080u;
        const uint32_t b0 = __byte_perm(c, 0x64646464u, 0x4140), b1 = __byte_perm(c, 0x64646464u, 0x4342);
        const __half2 off = __float2half2_rn(1152.f);
        const __half2 r0 = __hsub2(*reinterpret_cast<const __half2 *>(&b0), off);
        const __half2 r1 = __hsub2(*reinterpret_cast<const __half2 *>(&b1), off);
        lo = *reinterpret_cast<const uint32_t *>(&r0);
        hi = *reinterpret_cast<const uint32_t *>(&r1);
    }
}
template <Kv8 KV>
__device__ __forceinline__ float2 decode2(uint32_t c) {
    const uint32_t h = decode2_h<KV>(c);
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

}  // namespace
}  // namespace gdr
