// layernorm.cu -- the layer norm ahead of the MoE layer, forward and backward.
//
//   mean = sum x / d,  var = sum (x - mean)^2 / d,  rstd = 1 / sqrt(var + eps)
//   xh = (x - mean) rstd,  y = xh gamma + beta
//   t = dy gamma
//   dx = rstd (t - sum t / d - xh sum(t xh) / d)  (+ dres)
//   dgamma = sum_rows dy xh,  dbeta = sum_rows dy
//
// x (and dx, dres) bf16 or fp32 (a residual stream), y and dy bf16, the
// weights, statistics and their gradients fp32.  A row is held in registers by
// a group of warps, so that the variance is the sum of squared differences
// from the mean (no cancellation) with x read once; everything is fp32 and
// rounded where it is stored.
//
// Both kernels are bound by HBM.  The backward pass reads x and dy once: each
// block walks over many rows and keeps its columns' dgamma and dbeta in
// registers, writes one partial row per block, and a second kernel adds the
// partial rows in block order.  The number of blocks depends on the sizes and
// the GPU alone, so the sums have one order and repeat bit for bit.
#include <algorithm>

#include "mk_device.cuh"
#include "mk_internal.h"

namespace mk {
namespace {

constexpr int kMaxD = 16384;
constexpr int kMaxWarps = 16;    // per block
constexpr int kBwdBlocks = 304;  // two per SM

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f<float>(float v) {
    return v;
}
template <>
__device__ __forceinline__ float to_f<bf16>(bf16 v) {
    return __bfloat162float(v);
}

// VEC consecutive elements, loaded with one instruction where VEC > 1 (16
// bytes of fp32, 16 or 8 of bf16).
template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T* p, float (&f)[VEC]) {
    if constexpr (VEC == 1) {
        f[0] = to_f<T>(__ldcs(p));
    } else if constexpr (sizeof(T) == 4) {
        static_assert(VEC == 4);
        const float4 v = __ldcs(reinterpret_cast<const float4*>(p));
        f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
    } else {
        uint32_t w[VEC / 2];
        if constexpr (VEC == 8) {
            const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p));
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        } else {
            static_assert(VEC == 4);
            const uint2 v = __ldcs(reinterpret_cast<const uint2*>(p));
            w[0] = v.x, w[1] = v.y;
        }
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}

template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T* p, const float (&f)[VEC]) {
    if constexpr (VEC == 1) {
        if constexpr (sizeof(T) == 4)
            *p = f[0];
        else
            *p = __float2bfloat16_rn(f[0]);
    } else if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    } else if constexpr (VEC == 8) {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                                  pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
    } else {
        *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
    }
}

// VEC weights (the arrays are 16-byte aligned).
template <int VEC>
__device__ __forceinline__ void load_weights(const float* p, float (&f)[VEC]) {
    if constexpr (VEC == 1) {
        f[0] = __ldg(p);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; i += 4) {
            const float4 v = __ldg(reinterpret_cast<const float4*>(p + i));
            f[i] = v.x, f[i + 1] = v.y, f[i + 2] = v.z, f[i + 3] = v.w;
        }
    }
}

// Sum over a group of `warps` consecutive warps of the block, the same bits in
// every thread: the shuffle tree inside a warp, then the warps in order.  `red`
// holds one value per warp of the block; two calls with the same `red` have a
// block barrier between them.
__device__ __forceinline__ float group_sum(float v, int warps, float* red) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (warps == 1) return v;
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) red[warp] = v;
    __syncthreads();
    const int w0 = warp / warps * warps;
    float s = red[w0];
    for (int i = 1; i < warps; ++i) s += red[w0 + i];
    return s;
}

// NV vectors of VEC elements per thread; a row is `warps` warps.
template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(kMaxWarps * 32)
    layernorm_kernel(const T* __restrict__ x, const float* __restrict__ gamma, const float* __restrict__ beta,
                     int64_t rows, int d, float eps, int warps, bf16* __restrict__ y, float* __restrict__ mean,
                     float* __restrict__ rstd) {
    __shared__ float red[2][kMaxWarps];
    const int group = warps * 32;
    const int tid = threadIdx.x % group;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / group) + threadIdx.x / group;
    const bool ok = row < rows;
    const T* xr = x + (ok ? row : 0) * d;
    float v[NV][VEC];
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * group + tid) * VEC;
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[i][e] = 0.0f;
        if (ok && c < d) load_vec<T, VEC>(xr + c, v[i]);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) s += v[i][e];
    const float m = group_sum(s, warps, red[0]) / static_cast<float>(d);
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if ((i * group + tid) * VEC < d)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                v[i][e] -= m;
                s = fmaf(v[i][e], v[i][e], s);
            }
    const float r = rsqrtf(group_sum(s, warps, red[1]) / static_cast<float>(d) + eps);
    if (!ok) return;
    if (tid == 0) {
        mean[row] = m;
        rstd[row] = r;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * group + tid) * VEC;
        if (c < d) {
            float g[VEC], b[VEC];
            load_weights<VEC>(gamma + c, g);
            load_weights<VEC>(beta + c, b);
#pragma unroll
            for (int e = 0; e < VEC; ++e) g[e] = fmaf(v[i][e] * r, g[e], b[e]);
            store_vec<bf16, VEC>(y + row * d + c, g);
        }
    }
}

template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(kMaxWarps * 32)
    layernorm_bwd_kernel(const bf16* __restrict__ dy, const T* __restrict__ x, const float* __restrict__ gamma,
                         const float* __restrict__ mean, const float* __restrict__ rstd, const T* __restrict__ dres,
                         int64_t rows, int d, int warps, T* __restrict__ dx, float* __restrict__ part) {
    extern __shared__ float sums[];  // [2][d], only with several row groups per block
    __shared__ float red[2][2][kMaxWarps];
    const int group = warps * 32;
    const int groups = blockDim.x / group;
    const int gid = threadIdx.x / group;
    const int tid = threadIdx.x % group;
    float ag[NV][VEC], ab[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) ag[i][e] = ab[i][e] = 0.0f;
    const float inv_d = 1.0f / static_cast<float>(d);
    int parity = 0;
    for (int64_t base = static_cast<int64_t>(blockIdx.x) * groups; base < rows;
         base += static_cast<int64_t>(gridDim.x) * groups, parity ^= 1) {
        const int64_t row = base + gid;
        const bool ok = row < rows;
        const int64_t at = (ok ? row : 0) * d;
        float xv[NV][VEC], t[NV][VEC];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * group + tid) * VEC;
#pragma unroll
            for (int e = 0; e < VEC; ++e) xv[i][e] = t[i][e] = 0.0f;
            if (ok && c < d) {
                load_vec<T, VEC>(x + at + c, xv[i]);
                load_vec<bf16, VEC>(dy + at + c, t[i]);
            }
        }
        const float m = ok ? __ldg(mean + row) : 0.0f, r = ok ? __ldg(rstd + row) : 0.0f;
        float st = 0.0f, sx = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * group + tid) * VEC;
            if (c < d) {
                float g[VEC];
                load_weights<VEC>(gamma + c, g);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float xh = (xv[i][e] - m) * r;
                    xv[i][e] = xh;
                    ab[i][e] += t[i][e];
                    ag[i][e] = fmaf(t[i][e], xh, ag[i][e]);
                    t[i][e] *= g[e];
                    st += t[i][e];
                    sx = fmaf(t[i][e], xh, sx);
                }
            }
        }
        st = group_sum(st, warps, red[parity][0]) * inv_d;
        sx = group_sum(sx, warps, red[parity][1]) * inv_d;
        if (!ok) continue;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * group + tid) * VEC;
            if (c < d) {
                float o[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) o[e] = r * (t[i][e] - st - xv[i][e] * sx);
                if (dres != nullptr) {
                    float a[VEC];
                    load_vec<T, VEC>(dres + at + c, a);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) o[e] += a[e];
                }
                store_vec<T, VEC>(dx + at + c, o);
            }
        }
    }
    float* pg = part + static_cast<int64_t>(blockIdx.x) * 2 * d;
    if (groups > 1) {  // the groups' sums in group order
        for (int q = 0; q < groups; ++q) {
            if (gid == q) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const int c = (i * group + tid) * VEC + e;
                        if (c < d) {
                            sums[c] = ag[i][e] + (q > 0 ? sums[c] : 0.0f);
                            sums[d + c] = ab[i][e] + (q > 0 ? sums[d + c] : 0.0f);
                        }
                    }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < 2 * d; c += blockDim.x) pg[c] = sums[c];
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * group + tid) * VEC;
            if (c < d)
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    pg[c + e] = ag[i][e];
                    pg[d + c + e] = ab[i][e];
                }
        }
    }
}

// dgamma | dbeta = the blocks' partial rows [blocks][2 d], 32 columns per
// block: 8 slices of every eighth partial row, then the slices in order.
__global__ void __launch_bounds__(256) layernorm_bwd_sum_kernel(const float* __restrict__ part, int blocks, int d,
                                                                float* __restrict__ dgamma,
                                                                float* __restrict__ dbeta) {
    __shared__ float s[8][32];
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float v = 0.0f;
    if (c < 2 * d)
        for (int b = slice; b < blocks; b += 8) v += part[static_cast<int64_t>(b) * 2 * d + c];
    s[slice][lane] = v;
    __syncthreads();
    if (slice == 0 && c < 2 * d) {
#pragma unroll
        for (int i = 1; i < 8; ++i) v += s[i][lane];
        (c < d ? dgamma + c : dbeta + (c - d))[0] = v;
    }
}

// Warps per row and rows per block: 16 elements per thread up to d = 8192, 32
// above (16 warps then).
struct RowShape {
    int warps, rows;
    bool wide;
};
RowShape row_shape(int d) {
    RowShape s;
    s.wide = d > kMaxWarps * 512;
    s.warps = s.wide ? (d + 1023) / 1024 : (d + 511) / 512;
    s.rows = std::max(1, 8 / s.warps);
    return s;
}

unsigned bwd_blocks(int64_t rows, int d) {
    const RowShape s = row_shape(d);
    return static_cast<unsigned>(std::min<int64_t>((rows + s.rows - 1) / s.rows, kBwdBlocks));
}

template <typename T, int VEC>
cudaError_t launch_fwd(const void* x, const float* gamma, const float* beta, int64_t rows, int d, float eps, void* y,
                       float* mean, float* rstd, cudaStream_t s) {
    const RowShape r = row_shape(d);
    auto fn = r.wide ? layernorm_kernel<T, VEC, 32 / VEC> : layernorm_kernel<T, VEC, 16 / VEC>;
    fn<<<static_cast<unsigned>((rows + r.rows - 1) / r.rows), r.rows * r.warps * 32, 0, s>>>(
        static_cast<const T*>(x), gamma, beta, rows, d, eps, r.warps, static_cast<bf16*>(y), mean, rstd);
    return cudaGetLastError();
}

template <typename T, int VEC>
cudaError_t launch_bwd(const void* dy, const void* x, const float* gamma, const float* mean, const float* rstd,
                       const void* dres, int64_t rows, int d, void* dx, float* part, cudaStream_t s) {
    const RowShape r = row_shape(d);
    auto fn = r.wide ? layernorm_bwd_kernel<T, VEC, 32 / VEC> : layernorm_bwd_kernel<T, VEC, 16 / VEC>;
    const size_t smem = r.rows > 1 ? 2 * sizeof(float) * static_cast<size_t>(d) : 0;  // at most 16 KB
    fn<<<bwd_blocks(rows, d), r.rows * r.warps * 32, smem, s>>>(
        static_cast<const bf16*>(dy), static_cast<const T*>(x), gamma, mean, rstd, static_cast<const T*>(dres), rows,
        d, r.warps, static_cast<T*>(dx), part);
    return cudaGetLastError();
}

mk_status check_norm(int64_t T, int d, int x_type) {
    if (T < 0 || d <= 0 || (x_type != MK_TYPE_BF16 && x_type != MK_TYPE_FP32)) return MK_ERR_INVALID_ARG;
    if (d > kMaxD || T >= (int64_t(1) << 31) || T * d >= (int64_t(1) << 40)) return MK_ERR_UNSUPPORTED;
    return MK_OK;
}

}  // namespace
}  // namespace mk

using namespace mk;

extern "C" mk_status mk_moe_layernorm(const void* x, int x_type, const float* gamma, const float* beta, int64_t T,
                                      int d, float eps, void* y, float* mean, float* rstd, void* stream) {
    const mk_status st = check_norm(T, d, x_type);
    if (st != MK_OK) return st;
    if (!(eps >= 0.0f)) return MK_ERR_INVALID_ARG;
    if (T == 0) return MK_OK;
    if (!x || !gamma || !beta || !y || !mean || !rstd) return MK_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(gamma) || !aligned16(beta) || !aligned16(y)) return MK_ERR_INVALID_ARG;
    if (!device_is_sm103()) return MK_ERR_UNSUPPORTED;
    auto run = x_type == MK_TYPE_FP32 ? (d % 4 == 0 ? launch_fwd<float, 4> : launch_fwd<float, 1>)
                                      : (d % 8 == 0 ? launch_fwd<bf16, 8> : launch_fwd<bf16, 1>);
    const cudaError_t err = run(x, gamma, beta, T, d, eps, y, mean, rstd, static_cast<cudaStream_t>(stream));
    return err == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}

extern "C" size_t mk_moe_layernorm_bwd_workspace_size(int64_t T, int d) {
    if (check_norm(T, d, MK_TYPE_BF16) != MK_OK) return 0;
    return 256 + static_cast<size_t>(bwd_blocks(T, d)) * 2 * d * sizeof(float);
}

extern "C" mk_status mk_moe_layernorm_bwd(const void* dy, const void* x, int x_type, const float* gamma,
                                          const float* mean, const float* rstd, const void* dres, int64_t T, int d,
                                          void* dx, float* dgamma, float* dbeta, void* ws, size_t ws_bytes,
                                          void* stream) {
    const mk_status st = check_norm(T, d, x_type);
    if (st != MK_OK) return st;
    if (!dgamma || !dbeta) return MK_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T > 0) {
        if (!dy || !x || !gamma || !mean || !rstd || !dx) return MK_ERR_INVALID_ARG;
        if (!aligned16(dy) || !aligned16(x) || !aligned16(gamma) || !aligned16(dx) || (dres && !aligned16(dres)))
            return MK_ERR_INVALID_ARG;
        if (ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0 ||
            ws_bytes < mk_moe_layernorm_bwd_workspace_size(T, d))
            return MK_ERR_WORKSPACE;
    }
    if (!device_is_sm103()) return MK_ERR_UNSUPPORTED;
    if (T == 0) {  // no rows: the weights' gradients are zero
        if (cudaMemsetAsync(dgamma, 0, sizeof(float) * d, s) != cudaSuccess ||
            cudaMemsetAsync(dbeta, 0, sizeof(float) * d, s) != cudaSuccess)
            return MK_ERR_CUDA;
        return MK_OK;
    }
    float* part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + 256);
    auto run = x_type == MK_TYPE_FP32 ? (d % 4 == 0 ? launch_bwd<float, 4> : launch_bwd<float, 1>)
                                      : (d % 8 == 0 ? launch_bwd<bf16, 8> : launch_bwd<bf16, 1>);
    if (run(dy, x, gamma, mean, rstd, dres, T, d, dx, part, s) != cudaSuccess) return MK_ERR_CUDA;
    layernorm_bwd_sum_kernel<<<static_cast<unsigned>((2 * static_cast<int64_t>(d) + 31) / 32), 256, 0, s>>>(
        part, static_cast<int>(bwd_blocks(T, d)), d, dgamma, dbeta);
    return cudaGetLastError() == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}
