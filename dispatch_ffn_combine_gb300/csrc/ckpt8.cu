// ckpt8.cu -- activations kept in 8 bits for the backward pass (the format is
// in ckpt8.cuh): the layer's tokens, and SwiGLU's two inputs.
//
// Tokens.  The weight gradients of gate and up need the dispatched rows
// x_perm again: T k rows of bf16 that a training step would otherwise hold
// from the forward to the backward pass.  Kept instead: one 8-bit copy of
// every token (d + d / 32 bytes, 1 / (2 k) of the dispatched rows), restored
// straight into the dispatched rows through slot_row.
//
// SwiGLU.  h = silu(g) u is recomputed from 8-bit g and u in the backward
// pass, so neither g, u nor h is held in 16 bits:
//   s = 1 / (1 + exp(-g)),  a = g s,  slope = da/dg = s + a (1 - s)
//   dg = w dh u slope,  du = w dh a,  hw = w a u,  dw = sum_f dh a u
// for the routing weight w of the row, dh the gradient of the unweighted
// expert output's input (dP W2), and hw the weighted activation that the
// gradient of W2 multiplies.  All sums and products are fp32, rounded to bf16
// once where a tensor is stored.
//
// All four kernels move each byte once and are bound by HBM.  Measured, of the
// measured copy rate: save 32768 x 7168 113 us (0.94), dispatch into 8 rows
// 604 us (0.99), SwiGLU 262144 x 2048 forward 640 us (1.01), backward 856 us
// (0.94).
#include <algorithm>

#include "ckpt8.cuh"

namespace mk {
namespace {

using namespace ckpt8;

constexpr int kThreads = 256;

// Eight values per thread and step, so that a block of 32 is four lanes; two
// independent loads in flight per thread.
__global__ void __launch_bounds__(kThreads) ckpt8_save_kernel(const uint4* __restrict__ x, int64_t n8,
                                                              uint2* __restrict__ codes, uint8_t* __restrict__ scales) {
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * (2 * kThreads) + threadIdx.x;
    uint4 v[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t i = i0 + h * kThreads;
        v[h] = i < n8 ? __ldcs(x + i) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t i = i0 + h * kThreads;
        uint32_t byte;
        const uint2 c = encode8(v[h], byte);
        if (i < n8) {
            codes[i] = c;
            if ((i & 3) == 0) scales[i >> 2] = static_cast<uint8_t>(byte);
        }
    }
}

// A block per token: its codes are read once and its k rows written.
__global__ void __launch_bounds__(kThreads) ckpt8_dispatch_kernel(const uint8_t* __restrict__ codes,
                                                                  const uint8_t* __restrict__ scales,
                                                                  const int32_t* __restrict__ slot_row, int64_t S,
                                                                  int d, int k, bf16* __restrict__ x_perm,
                                                                  uint32_t* status) {
    __shared__ int64_t rows[kMaxTopK];
    const int64_t t = blockIdx.x;
    pdl_wait();  // the status comes from the kernel before
    if (threadIdx.x < k) {
        const int64_t r = slot_row[t * k + threadIdx.x];
        const bool ok = r >= 0 && r < S;
        if (!ok) report_error(status, MK_ERR_BOUNDS, kSiteCkptSlot);
        rows[threadIdx.x] = ok ? r : -1;
    }
    __syncthreads();
    const uint2* c8 = reinterpret_cast<const uint2*>(codes + t * d);
    const uint8_t* s8 = scales + t * (d / kBlock);
    for (int c = threadIdx.x; c < d / 8; c += kThreads) {
        float f[8];
        decode8(__ldg(c8 + c), scale_value(__ldg(s8 + (c >> 2))), f);
        const uint4 v = pack8(f);
        for (int j = 0; j < k; ++j)
            if (rows[j] >= 0) reinterpret_cast<uint4*>(x_perm + rows[j] * d)[c] = v;
    }
}

__device__ __forceinline__ float sigmoid(float g) { return __fdividef(1.0f, 1.0f + __expf(-g)); }

// h = silu(gate) up from the bf16 inputs; codes [2, S, f] and scales
// [2, S, f / 32] of gate and up.
__global__ void __launch_bounds__(kThreads) swiglu_ckpt8_kernel(const uint4* __restrict__ gate,
                                                                const uint4* __restrict__ up, int64_t n8,
                                                                uint4* __restrict__ h, uint2* __restrict__ codes,
                                                                uint8_t* __restrict__ scales) {
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * (2 * kThreads) + threadIdx.x;
    uint4 g[2], u[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int64_t i = i0 + q * kThreads;
        const bool ok = i < n8;
        g[q] = ok ? __ldcs(gate + i) : make_uint4(0, 0, 0, 0);
        u[q] = ok ? __ldcs(up + i) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int64_t i = i0 + q * kThreads;
        uint32_t gb, ub;
        const uint2 gc = encode8(g[q], gb);
        const uint2 uc = encode8(u[q], ub);
        float a[8], b[8];
        unpack8(g[q], a);
        unpack8(u[q], b);
#pragma unroll
        for (int e = 0; e < 8; ++e) a[e] = a[e] * sigmoid(a[e]) * b[e];
        if (i < n8) {
            h[i] = pack8(a);
            codes[i] = gc;
            codes[n8 + i] = uc;
            if ((i & 3) == 0) {
                scales[i >> 2] = static_cast<uint8_t>(gb);
                scales[(n8 + i) >> 2] = static_cast<uint8_t>(ub);
            }
        }
    }
}

// WPR warps per row, kThreads / 32 / WPR rows per block; dw is summed inside a
// lane, then over the lanes by the shuffle tree, then over the row's warps in
// order: one fixed order.
template <int WPR>
__global__ void __launch_bounds__(kThreads) swiglu_ckpt8_bwd_kernel(
    const bf16* __restrict__ dh, const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
    const float* __restrict__ row_weight, int64_t S, int f, bf16* __restrict__ dgate, bf16* __restrict__ dup,
    bf16* __restrict__ hw, float* __restrict__ drow_weight) {
    constexpr int kWarps = kThreads / 32;
    constexpr int kRows = kWarps / WPR;
    __shared__ float part[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + warp / WPR;
    const bool row_ok = row < S;
    const int64_t plane = S * f;
    float dw = 0.0f;
    if (row_ok) {
        const int64_t base = row * f;
        const float w = row_weight != nullptr ? __ldg(row_weight + row) : 1.0f;
        // without a sign: c passes f, which may be 2^31 - 64, by up to 2048
#pragma unroll 2
        for (uint32_t c = ((warp % WPR) * 32 + lane) * 8; c < static_cast<uint32_t>(f); c += WPR * 256) {
            const int64_t at = base + c;
            const uint4 dv = __ldcs(reinterpret_cast<const uint4*>(dh + at));
            const uint2 gc = __ldcs(reinterpret_cast<const uint2*>(codes + at));
            const uint2 uc = __ldcs(reinterpret_cast<const uint2*>(codes + plane + at));
            const uint32_t gb = __ldg(scales + at / kBlock), ub = __ldg(scales + (plane + at) / kBlock);
            float d[8], g[8], u[8];
            unpack8(dv, d);
            decode8(gc, scale_value(gb), g);
            decode8(uc, scale_value(ub), u);
            float og[8], ou[8], oh[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float s = sigmoid(g[e]);
                const float a = g[e] * s;
                const float wd = w * d[e];
                const float au = a * u[e];
                og[e] = wd * u[e] * fmaf(a, 1.0f - s, s);
                ou[e] = wd * a;
                oh[e] = w * au;
                dw = fmaf(d[e], au, dw);
            }
            *reinterpret_cast<uint4*>(dgate + at) = pack8(og);
            *reinterpret_cast<uint4*>(dup + at) = pack8(ou);
            if (hw != nullptr) *reinterpret_cast<uint4*>(hw + at) = pack8(oh);
        }
    }
    if (drow_weight == nullptr) return;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) dw += __shfl_xor_sync(0xffffffffu, dw, o);
    if (WPR == 1) {
        if (row_ok && lane == 0) drow_weight[row] = dw;
        return;
    }
    if (lane == 0) part[warp] = dw;
    __syncthreads();
    if (row_ok && lane == 0 && warp % WPR == 0) {
#pragma unroll
        for (int i = 1; i < WPR; ++i) dw += part[warp + i];
        drow_weight[row] = dw;
    }
}

template <int WPR>
cudaError_t launch_swiglu_bwd(const bf16* dh, const uint8_t* codes, const uint8_t* scales, const float* row_weight,
                              int64_t S, int f, bf16* dgate, bf16* dup, bf16* hw, float* drow_weight,
                              cudaStream_t s) {
    constexpr int kRows = kThreads / 32 / WPR;
    swiglu_ckpt8_bwd_kernel<WPR><<<static_cast<unsigned>((S + kRows - 1) / kRows), kThreads, 0, s>>>(
        dh, codes, scales, row_weight, S, f, dgate, dup, hw, drow_weight);
    return cudaGetLastError();
}

// Rows and row length of a checkpointed tensor; `k` rows are restored per row.
mk_status check_rows(int64_t rows, int d, int k) {
    if (rows < 0 || d <= 0 || k <= 0 || d % 64 != 0 || k > kMaxTopK) return MK_ERR_INVALID_ARG;
    if (rows >= (int64_t(1) << 31) / k) return MK_ERR_UNSUPPORTED;
    if (rows * k >= (int64_t(1) << 40) / d) return MK_ERR_UNSUPPORTED;
    return MK_OK;
}

}  // namespace
}  // namespace mk

using namespace mk;

extern "C" mk_status mk_moe_ckpt8_save(const void* x, int64_t T, int d, uint8_t* codes, uint8_t* scales,
                                       void* stream) {
    const mk_status st = check_rows(T, d, 1);
    if (st != MK_OK) return st;
    if (T == 0) return MK_OK;
    if (!x || !codes || !scales || !aligned16(x) || !aligned16(codes)) return MK_ERR_INVALID_ARG;
    if (!device_is_sm103()) return MK_ERR_UNSUPPORTED;
    const int64_t n8 = T * (d / 8);
    ckpt8_save_kernel<<<static_cast<unsigned>((n8 + 2 * kThreads - 1) / (2 * kThreads)), kThreads, 0,
                        static_cast<cudaStream_t>(stream)>>>(static_cast<const uint4*>(x), n8,
                                                             reinterpret_cast<uint2*>(codes), scales);
    return cudaGetLastError() == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}

extern "C" mk_status mk_moe_ckpt8_dispatch(const uint8_t* codes, const uint8_t* scales, const int32_t* slot_row,
                                           int64_t T, int d, int k, void* x_perm, void* ws, size_t ws_bytes,
                                           void* stream) {
    const mk_status st = check_rows(T, d, k);
    if (st != MK_OK) return st;
    if (T == 0) return MK_OK;
    if (!codes || !scales || !slot_row || !x_perm || !aligned16(codes) || !aligned16(x_perm))
        return MK_ERR_INVALID_ARG;
    if (ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0 || ws_bytes < 256) return MK_ERR_WORKSPACE;
    if (!device_is_sm103()) return MK_ERR_UNSUPPORTED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint32_t* status = static_cast<uint32_t*>(ws);
    if (launch_clear_control(status, s) != cudaSuccess) return MK_ERR_CUDA;
    LaunchCfg lc(dim3(static_cast<unsigned>(T)), dim3(kThreads), 0, s, true);
    const cudaError_t err = cudaLaunchKernelEx(&lc.cfg, ckpt8_dispatch_kernel, codes, scales, slot_row, T * k, d, k,
                                               static_cast<bf16*>(x_perm), status);
    return err == cudaSuccess && cudaGetLastError() == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}

extern "C" mk_status mk_moe_swiglu_ckpt8(const void* gate, const void* up, int64_t S, int f, void* h, uint8_t* codes,
                                         uint8_t* scales, void* stream) {
    const mk_status st = check_rows(S, f, 1);
    if (st != MK_OK) return st;
    if (S == 0) return MK_OK;
    if (!gate || !up || !h || !codes || !scales) return MK_ERR_INVALID_ARG;
    if (!aligned16(gate) || !aligned16(up) || !aligned16(h) || !aligned16(codes)) return MK_ERR_INVALID_ARG;
    if (!device_is_sm103()) return MK_ERR_UNSUPPORTED;
    const int64_t n8 = S * (f / 8);
    swiglu_ckpt8_kernel<<<static_cast<unsigned>((n8 + 2 * kThreads - 1) / (2 * kThreads)), kThreads, 0,
                          static_cast<cudaStream_t>(stream)>>>(
        static_cast<const uint4*>(gate), static_cast<const uint4*>(up), n8, static_cast<uint4*>(h),
        reinterpret_cast<uint2*>(codes), scales);
    return cudaGetLastError() == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}

extern "C" mk_status mk_moe_swiglu_ckpt8_bwd(const void* dh, const uint8_t* codes, const uint8_t* scales,
                                             const float* row_weight, int64_t S, int f, void* dgate, void* dup,
                                             void* hw, float* drow_weight, void* stream) {
    const mk_status st = check_rows(S, f, 1);
    if (st != MK_OK) return st;
    if (S == 0) return MK_OK;
    if (!dh || !codes || !scales || !dgate || !dup) return MK_ERR_INVALID_ARG;
    if (!aligned16(dh) || !aligned16(codes) || !aligned16(dgate) || !aligned16(dup) || (hw && !aligned16(hw)))
        return MK_ERR_INVALID_ARG;
    if (!device_is_sm103()) return MK_ERR_UNSUPPORTED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // One warp per row where there are rows enough to fill the GPU (262144 x 2048: 856 us, with 8
    // warps per row 1058), more for fewer rows (16384 x 1408: 2 warps 45 us, 1 warp 49, 4 warps 57);
    // a warp has 256 columns at least.
    int wpr = 1;
    while (wpr < 8 && S * wpr < 32768 && f >= 512 * wpr) wpr *= 2;
    auto run = wpr == 8 ? launch_swiglu_bwd<8> : wpr == 4 ? launch_swiglu_bwd<4> : wpr == 2 ? launch_swiglu_bwd<2>
                                                                                        : launch_swiglu_bwd<1>;
    const cudaError_t err = run(static_cast<const bf16*>(dh), codes, scales, row_weight, S, f,
                                static_cast<bf16*>(dgate), static_cast<bf16*>(dup), static_cast<bf16*>(hw),
                                drow_weight, s);
    return err == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}
