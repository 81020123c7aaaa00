// f32x2.cuh -- two fp32 values in one 64-bit register, and their arithmetic: each of
// the pair rounded to nearest, as by the instruction on one.
#pragma once

#include <cstdint>

namespace mk {

// Two fp32 values in one 64-bit register, the operands of the f32x2 instructions.
struct f2 {
    uint64_t v;
    __device__ __forceinline__ f2() {}
    __device__ __forceinline__ f2(float x, float y) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y)); }
    __device__ __forceinline__ float x() const {
        return __uint_as_float(static_cast<uint32_t>(v));
    }
    __device__ __forceinline__ float y() const {
        return __uint_as_float(static_cast<uint32_t>(v >> 32));
    }
};
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ f2 both(float v) { return f2(v, v); }

}  // namespace mk
