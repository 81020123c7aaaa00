// quant8.cu -- what the 8-bit grouped GEMM's operands are made by: rows of bf16
// values, SwiGLU's output, and weights, as e4m3 codes with a scale per block of
// 128 values (weights: 128 x 128).
//
// All three are bound by HBM: each value is read once and each code written once (262144 x
// 2048: rows 249 us, 0.96 of the copy rate, SwiGLU 402, 0.99; weights at 0.90).
//
// Rows: eight lanes hold a block, 16 values each (two 16-byte loads per tensor, one
// 16-byte store), so a warp has four blocks at a time: of one row, or of two or four
// rows that have so few.  Its largest magnitude takes three shuffles.  SwiGLU is
// rounded once, to the code; its bf16 output is never formed.  Its exponential is within 6.5 units of
// 2^-24 for every gate, the rest rounded to nearest.  (With the fast exponential, off by up to
// 1.2 |g| units of 2^-23 more, and the fast quotient, zero for gates below -87.3, 379 us; with expf and
// a division 510, with expf and the corrected quotient 480.)
//
// Weights: a thread block per 128 x 128 values, held in registers between the pass
// for the largest magnitude and the one for the codes.
#include <algorithm>

#include "quant8.cuh"

namespace mk {
namespace {

constexpr int kRowWarps = 8;    // per thread block
constexpr int kLaneVals = 16;   // values per lane: one 16-byte store of codes
constexpr int kBlockLanes = kScaleBlock / kLaneVals;
constexpr int kGroups = 32 / kBlockLanes;  // blocks per warp and step

struct Raw16 {
    uint4 a, b;
};
__device__ __forceinline__ Raw16 load_raw(const bf16* p) {
    return {__ldg(reinterpret_cast<const uint4*>(p)), __ldg(reinterpret_cast<const uint4*>(p) + 1)};
}
__device__ __forceinline__ void unpack(const Raw16& r, float (&f)[16]) {
    const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void load16(const bf16* p, float (&f)[16]) { unpack(load_raw(p), f); }

// silu(g) u = g / (1 + exp(-g)) u in fp32 for a bf16 g.  exp(-g) = 2^(-g a) exp(-g b) with a the 16 bits nearest to
// log2 e, so that g a is exact, and b = 1 - a ln 2; g b is below 2^-11, so 1 - g b stands for the second factor (2^-23).
// The quotient is the product with the reciprocal, corrected as in quant8::encode.
constexpr float kLog2E16 = 47274.0f / 32768.0f, kLog2ERest = 4.888495e-6f;
constexpr float kLeastGate = -87.0f;  // 1 + exp(87) is below 2^126: the reciprocal is a normal number
__device__ __forceinline__ float ex2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_approx(float d) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
    return r;
}
__device__ __forceinline__ float least(const Raw16& r) {
    const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
    __nv_bfloat162 m = reinterpret_cast<const __nv_bfloat162&>(w[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) m = __hmin2(m, reinterpret_cast<const __nv_bfloat162&>(w[i]));
    return __bfloat162float(__hmin(m.x, m.y));
}
// silu(g) for g < kLeastGate, where 1 is no part of the sum: g exp(g), the exponential raised by 2^64 until the product
// is a normal number.  Zero where exp(-g) is past fp32 (of bf16 gates those from -89 down).
__device__ __forceinline__ float silu_low(float g) {
    const float e = ex2_approx(fmaf(g, kLog2E16, 64.0f));
    return g > -88.75f ? g * fmaf(e, g * kLog2ERest, e) * 0x1p-64f : g * 0.0f;
}
__device__ __forceinline__ void swiglu(const Raw16& gate, const Raw16& up, float (&f)[16]) {
    float u[16];
    unpack(gate, f);
    unpack(up, u);
    const bool low = least(gate) < kLeastGate;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const f2 g(f[2 * i], f[2 * i + 1]);
        const f2 t = mul2(g, both(-kLog2E16)), rest = mul2(g, both(-kLog2ERest));
        f2 e(ex2_approx(t.x()), ex2_approx(t.y()));
        e = fma2(e, rest, e);
        const f2 d = add2(e, both(1.0f)), minus = fma2(e, both(-1.0f), both(-1.0f));
        const f2 y(rcp_approx(d.x()), rcp_approx(d.y()));
        f2 q = mul2(g, y);
        q = fma2(fma2(q, minus, g), y, q);
        if (low) q = f2(g.x() < kLeastGate ? silu_low(g.x()) : q.x(), g.y() < kLeastGate ? silu_low(g.y()) : q.y());
        q = mul2(q, f2(u[2 * i], u[2 * i + 1]));
        f[2 * i] = q.x(), f[2 * i + 1] = q.y();
    }
}

// x (kSwiGLU: gate) and up with row strides ld; a warp takes rows of 1 << row_shift
// per step and blockIdx.y's `steps` steps of blocks.
template <bool kSwiGLU>
__global__ void __launch_bounds__(kRowWarps * 32) quant8_rows_kernel(const bf16* __restrict__ x,
                                                                     const bf16* __restrict__ up, int64_t ld,
                                                                     int64_t rows, int c, int pitch, int row_shift,
                                                                     int steps, uint8_t* __restrict__ codes,
                                                                     float* __restrict__ scales) {
    const int lane = threadIdx.x & 31, group = lane / kBlockLanes, in_block = lane % kBlockLanes;
    const int per_row = kGroups >> row_shift;  // blocks of a row per step
    const int64_t row = ((static_cast<int64_t>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5)) << row_shift) + group / per_row;
    const int blocks = (c + kScaleBlock - 1) / kScaleBlock;
    const bool live = row < rows;
    const bf16* xr = x + (live ? row : 0) * ld;
    const bf16* ur = kSwiGLU ? up + (live ? row : 0) * ld : nullptr;
    int b = blockIdx.y * steps * per_row + group % per_row;
#pragma unroll 1
    for (int s = 0; s < steps; ++s, b += per_row) {
        const int col = b * kScaleBlock + in_block * kLaneVals;
        const bool in = live && col < c;  // c is a multiple of 64: all 16 values or none
        float f[kLaneVals];
        if (in) {
            if constexpr (kSwiGLU)
                swiglu(load_raw(xr + col), load_raw(ur + col), f);
            else
                load16(xr + col, f);
        } else {
#pragma unroll
            for (int i = 0; i < kLaneVals; ++i) f[i] = 0.0f;
        }
        const float scale = quant8::block_scale<kLaneVals, kBlockLanes>(f);
        if (!live) continue;
        if (in_block == 0 && b < pitch) scales[row * pitch + b] = b < blocks ? scale : 0.0f;
        if (in) {
            uint32_t q[4];
            quant8::encode(f, scale, q);
            *reinterpret_cast<uint4*>(codes + row * c + col) = make_uint4(q[0], q[1], q[2], q[3]);
        }
    }
}

constexpr int kWThreads = 256;

__global__ void __launch_bounds__(kWThreads, 3) quant8_weights_kernel(const bf16* __restrict__ w, int n, int d, int k_blocks,
                                                                   int n_blocks, int pitch, uint8_t* __restrict__ codes,
                                                                   float* __restrict__ scales) {
    __shared__ float most[2][kWThreads / 32];
    const int kb = blockIdx.x % k_blocks, nb = blockIdx.x / k_blocks, e = blockIdx.y;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r0 = nb * kScaleBlock + (threadIdx.x >> 3), col = kb * kScaleBlock + (threadIdx.x & 7) * 16;
    const int64_t base = static_cast<int64_t>(e) * n;
    // Rows r0, r0 + 32, ..., kept as bf16: half the registers, three thread blocks per SM instead of two (16 experts of
    // 4096 x 7168: 230 us, 0.90 of the copy rate; with fp32 values held 408, with four blocks, whose 64 registers spill, 240).
    Raw16 raw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        raw[i] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
        if (r0 + 32 * i < n && col < d) raw[i] = load_raw(w + (base + r0 + 32 * i) * d + col);
    }
    float f[16], m = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        unpack(raw[i], f);
        m = quant8::max_nan(m, quant8::magnitude(f));
    }
    m = quant8::group_max<32>(m);
    if (lane == 0) most[0][warp] = m;
    __syncthreads();
    m = 0.0f;
#pragma unroll
    for (int i = 0; i < kWThreads / 32; ++i) m = quant8::max_nan(m, most[0][i]);
    if (quant8::not_finite(m)) {  // the same for the whole thread block
        m = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            unpack(raw[i], f);
            m = fmaxf(m, quant8::finite_magnitude(f));
        }
        m = quant8::group_max<32>(m);
        if (lane == 0) most[1][warp] = m;
        __syncthreads();
        m = 0.0f;
#pragma unroll
        for (int i = 0; i < kWThreads / 32; ++i) m = fmaxf(m, most[1][i]);
    }
    const float scale = quant8::scale_of(m);
    float* row = scales + (static_cast<int64_t>(e) * n_blocks + nb) * pitch;
    if (threadIdx.x == 0) row[kb] = scale;
    if (kb == k_blocks - 1 && threadIdx.x < pitch - k_blocks) row[k_blocks + threadIdx.x] = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (r0 + 32 * i < n && col < d) {
            uint32_t q[4];
            unpack(raw[i], f);
            quant8::finite_magnitude(f);  // what is not finite becomes NaN
            quant8::encode(f, scale, q);
            *reinterpret_cast<uint4*>(codes + (base + r0 + 32 * i) * d + col) = make_uint4(q[0], q[1], q[2], q[3]);
        }
}

template <bool kSwiGLU>
cudaError_t launch_rows(const void* x, const void* up, int64_t ld, int64_t rows, int c, uint8_t* codes, float* scales,
                        cudaStream_t s) {
    const int pitch = scale_pitch(c);
    // Rows of one or two blocks share a warp.
    const int row_shift = pitch > kGroups ? 0 : (c + kScaleBlock - 1) / kScaleBlock > 2 ? 0 : c > kScaleBlock ? 1 : 2;
    const int per_row = kGroups >> row_shift;
    const int64_t warps = (rows + (1 << row_shift) - 1) >> row_shift;
    const unsigned grid_x = static_cast<unsigned>((warps + kRowWarps - 1) / kRowWarps);
    const int all = (pitch + per_row - 1) / per_row;  // steps of a row, its unused scales included
    // Few rows: a row's steps are spread over thread blocks until each SM has two.
    int parts = 1;
    while (parts < all && static_cast<int64_t>(grid_x) * parts < 2 * device_sm_count()) parts *= 2;
    parts = std::min(parts, all);
    const int steps = (all + parts - 1) / parts;
    quant8_rows_kernel<kSwiGLU><<<dim3(grid_x, static_cast<unsigned>((all + steps - 1) / steps)), kRowWarps * 32, 0, s>>>(
        static_cast<const bf16*>(x), static_cast<const bf16*>(up), ld, rows, c, pitch, row_shift, steps, codes, scales);
    return cudaGetLastError();
}

mk_status check_rows(int64_t rows, int c, int64_t ld) {
    if (rows < 0 || c <= 0 || c % 64 != 0 || ld < c || ld % 8 != 0) return MK_ERR_INVALID_ARG;
    // Columns are counted in 32 bits, a warp's last step past the row's end included.
    if (c >= 1 << 30 || rows >= (int64_t(1) << 31) || ld >= (int64_t(1) << 31) || rows * ld >= (int64_t(1) << 40)) return MK_ERR_UNSUPPORTED;
    return MK_OK;
}

}  // namespace
}  // namespace mk

using namespace mk;

extern "C" mk_status mk_moe_quant8_rows(const void* x, int64_t ld, int64_t S, int c, uint8_t* codes, float* scales,
                                        void* stream) {
    const mk_status st = check_rows(S, c, ld);
    if (st != MK_OK) return st;
    if (S == 0) return MK_OK;
    if (!x || !codes || !scales || !aligned16(x) || !aligned16(codes) || !aligned16(scales)) return MK_ERR_INVALID_ARG;
    if (!device_is_sm103()) return MK_ERR_UNSUPPORTED;
    const cudaError_t err = launch_rows<false>(x, nullptr, ld, S, c, codes, scales, static_cast<cudaStream_t>(stream));
    return err == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}

extern "C" mk_status mk_moe_swiglu8(const void* gate, const void* up, int64_t ld, int64_t S, int f, uint8_t* codes,
                                    float* scales, void* stream) {
    const mk_status st = check_rows(S, f, ld);
    if (st != MK_OK) return st;
    if (S == 0) return MK_OK;
    if (!gate || !up || !codes || !scales) return MK_ERR_INVALID_ARG;
    if (!aligned16(gate) || !aligned16(up) || !aligned16(codes) || !aligned16(scales)) return MK_ERR_INVALID_ARG;
    if (!device_is_sm103()) return MK_ERR_UNSUPPORTED;
    const cudaError_t err = launch_rows<true>(gate, up, ld, S, f, codes, scales, static_cast<cudaStream_t>(stream));
    return err == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}

extern "C" mk_status mk_moe_quant8_weights(const void* w, int E, int n, int d, uint8_t* codes, float* scales,
                                           void* stream) {
    const mk_status st = check_sizes(0, d, E, 1, n);
    if (st != MK_OK) return st;
    if (n >= 1 << 30 || d >= 1 << 30) return MK_ERR_UNSUPPORTED;  // rows and columns are counted in 32 bits, a block's past the end included
    if (!w || !codes || !scales || !aligned16(w) || !aligned16(codes) || !aligned16(scales)) return MK_ERR_INVALID_ARG;
    const int k_blocks = (d + kScaleBlock - 1) / kScaleBlock, n_blocks = (n + kScaleBlock - 1) / kScaleBlock;
    if (static_cast<int64_t>(k_blocks) * n_blocks >= (int64_t(1) << 31)) return MK_ERR_UNSUPPORTED;
    if (!device_is_sm103()) return MK_ERR_UNSUPPORTED;
    quant8_weights_kernel<<<dim3(static_cast<unsigned>(k_blocks * n_blocks), static_cast<unsigned>(E)), kWThreads, 0,
                            static_cast<cudaStream_t>(stream)>>>(static_cast<const bf16*>(w), n, d, k_blocks, n_blocks,
                                                                 scale_pitch(d), codes, scales);
    return cudaGetLastError() == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}
