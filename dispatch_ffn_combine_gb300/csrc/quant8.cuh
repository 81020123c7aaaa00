// quant8.cuh -- e4m3 codes with one fp32 scale per block of 128 values, as the
// 8-bit grouped GEMM takes them.
//
// A block's scale is amax / 448 (2^-126 at least), amax the largest finite
// magnitude of the block and 448 the largest e4m3 value; a code is the quotient
// v / scale, rounded to nearest in fp32 and then to nearest even, so a value is off by at
// most 2^-4 |v|, or half a step of 2^-9 scale where the code is subnormal.  The quotient
// is v times the reciprocal of the scale, corrected by its remainder (Markstein's
// division: with the reciprocal rounded to nearest and an exact remainder the corrected
// quotient is rounded to nearest); the product alone, off by two roundings, gave other
// codes next to the middle between two.  The bound of 2^-126 keeps the reciprocal finite.
// NaN and infinities become e4m3's NaN, so that what went wrong is still seen.
#pragma once

#include <cuda_fp8.h>

#include "f32x2.cuh"
#include "mk_device.cuh"
#include "mk_internal.h"

namespace mk {
namespace quant8 {

__device__ __forceinline__ float scale_of(float amax) {
    return fmaxf(__fdiv_rn(amax, 448.0f), 1.17549435e-38f);
}

// Largest magnitude of N values; NaN if one is NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
template <int N>
__device__ __forceinline__ float magnitude(const float (&f)[N]) {
    float m = fabsf(f[0]);
#pragma unroll
    for (int i = 1; i < N; ++i) m = max_nan(m, fabsf(f[i]));
    return m;
}
// The same of the finite ones; the others become NaN.
template <int N>
__device__ __forceinline__ float finite_magnitude(float (&f)[N]) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (fabsf(f[i]) <= 3.40282347e38f)
            m = fmaxf(m, fabsf(f[i]));
        else
            f[i] = __uint_as_float(0x7fffffffu);
    }
    return m;
}
__device__ __forceinline__ bool not_finite(float m) { return !(m <= 3.40282347e38f); }
template <int LANES>
__device__ __forceinline__ float group_max(float m) {
#pragma unroll
    for (int o = LANES / 2; o >= 1; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}

// The scales of NB blocks that LANES neighbouring lanes hold, N values of each (zeros
// past the row's end); every lane of the warp calls.
template <int NB, int N, int LANES>
__device__ __forceinline__ void block_scales(float (&f)[NB][N], float (&scale)[NB]) {
    float m[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) m[b] = magnitude(f[b]);
#pragma unroll
    for (int o = LANES / 2; o >= 1; o >>= 1)
#pragma unroll
        for (int b = 0; b < NB; ++b) m[b] = max_nan(m[b], __shfl_xor_sync(0xffffffffu, m[b], o));
    if (__any_sync(0xffffffffu, not_finite(magnitude(m)))) {
#pragma unroll
        for (int b = 0; b < NB; ++b) m[b] = group_max<LANES>(finite_magnitude(f[b]));
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) scale[b] = scale_of(m[b]);
}
template <int N, int LANES>
__device__ __forceinline__ float block_scale(float (&f)[N]) {
    float m = group_max<LANES>(magnitude(f));
    if (__any_sync(0xffffffffu, not_finite(m))) m = group_max<LANES>(finite_magnitude(f));
    return scale_of(m);
}

// Codes of N values.  The smallest blocks' values and scale are raised by 2^64, exactly: the remainders of
// what is not rounded to zero are normal numbers.
template <int N, bool kRaised>
__device__ __forceinline__ void encode_block(const float (&f)[N], float scale, uint32_t (&c)[N / 4]) {
    if (kRaised) scale *= 0x1p64f;
    const f2 inv = both(__frcp_rn(scale)), minus = both(-scale);
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        f2 q[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            f2 v(f[4 * i + 2 * h], f[4 * i + 2 * h + 1]);
            if (kRaised) v = mul2(v, both(0x1p64f));
            q[h] = mul2(v, inv);
            q[h] = fma2(fma2(q[h], minus, v), inv, q[h]);
        }
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(q[0].x(), q[0].y()), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(q[1].x(), q[1].y()), __NV_SATFINITE, __NV_E4M3);
        c[i] = lo | (hi << 16);
    }
}
template <int N>
__device__ __forceinline__ void encode(const float (&f)[N], float scale, uint32_t (&c)[N / 4]) {
    if (scale >= 0x1p-64f)
        encode_block<N, false>(f, scale, c);
    else
        encode_block<N, true>(f, scale, c);
}

}  // namespace quant8
}  // namespace mk
