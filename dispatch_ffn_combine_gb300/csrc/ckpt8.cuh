// ckpt8.cuh -- the 8-bit activation checkpoint's number format.
//
// A tensor is kept as one e4m3 code per value and one scale byte per block of
// 32 consecutive values.  The block's scale is the smallest power of two 2^q
// (q >= -124) with  amax <= 448 * 2^q,  amax the largest finite magnitude of
// the block and 448 the largest e4m3 value; the scale byte is q + 127.  A
// code is v / 2^q rounded to nearest even, so the largest value of a block is
// never clipped and a value v with |v| >= 2^(q - 6) is off by at most 2^-4 |v|.
// NaN and infinities are kept as e4m3's NaN (it has no infinity), so that what
// went wrong in the forward pass is still seen in the backward pass.  Finite
// values stay finite: magnitudes that would round to 2^128 become 1.875 2^127.
//
// Scales are powers of two so that both divisions are exact and a restored
// value (4 significant bits, a multiple of 2^-133) is exact in bf16: save and
// restore round once.  With the bound on q every 2^q and 2^-q used is a normal
// fp32 number.
#pragma once

#include <cuda_fp8.h>

#include "mk_device.cuh"
#include "mk_internal.h"

namespace mk {
namespace ckpt8 {

constexpr int kBlock = 32;       // values per scale byte
constexpr uint32_t kMinExp = 3;  // q = -124

// Scale byte of a block with largest finite magnitude amax (>= 0).
__device__ __forceinline__ uint32_t scale_byte(float amax) {
    const uint32_t b = __float_as_uint(amax);
    const int e = static_cast<int>(b >> 23);  // amax = 1.m 2^(e - 127); 448 = 1.75 2^8
    const int q = e - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
    return static_cast<uint32_t>(max(q, static_cast<int>(kMinExp)));
}

__device__ __forceinline__ float scale_value(uint32_t byte) { return __uint_as_float(byte << 23); }          // 2^q
__device__ __forceinline__ float scale_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }  // 2^-q

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

// Codes and scale byte of 8 consecutive bf16 values; the four lanes of a
// 4-lane group hold one block of 32 (every lane of the warp calls).
__device__ __forceinline__ uint2 encode8(const uint4& v, uint32_t& byte) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t m = 0;  // bf16 magnitudes order like their bits
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, max(w[i] & 0x7fff0000u, (w[i] << 16) & 0x7fff0000u));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    float f[8];
    unpack8(v, f);
    if (__any_sync(0xffffffffu, m > 0x7f600000u)) {
        // a block with NaN, infinities or magnitudes above 1.75 2^127: the largest finite
        // magnitude, and no finite value that would round up to 2^128
        uint32_t n = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t b = __float_as_uint(f[i]), a = b & 0x7fffffffu;
            if (a < 0x7f800000u) {
                n = max(n, a);
                f[i] = __uint_as_float((b & 0x80000000u) | min(a, 0x7f700000u));
            } else {
                f[i] = __uint_as_float(0x7fffffffu);
            }
        }
        n = max(n, __shfl_xor_sync(0xffffffffu, n, 1));
        n = max(n, __shfl_xor_sync(0xffffffffu, n, 2));
        m = n;
    }
    byte = scale_byte(__uint_as_float(m));
    const float inv = scale_inverse(byte);
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        c[i] = __nv_cvt_float2_to_fp8x2(make_float2(f[2 * i] * inv, f[2 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// The values that 8 codes stand for.
__device__ __forceinline__ void decode8(const uint2& c, float scale, float (&f)[8]) {
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
            static_cast<__nv_fp8x2_storage_t>(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
        const float2 v = __half22float2(__half2(h));
        f[2 * i] = v.x * scale;
        f[2 * i + 1] = v.y * scale;
    }
}

}  // namespace ckpt8
}  // namespace mk
