// layernorm.cu -- the layer norm ahead of the MoE layer, forward and backward.
//
//   mean = sum x / d,  var = sum (x - mean)^2 / d,  rstd = 1 / sqrt(var + eps)
//   xh = (x - mean) rstd,  y = xh gamma + beta
//   t = dy gamma
//   dx = rstd (t - sum t / d - xh sum(t xh) / d)  (+ dres)
//   dgamma = sum_rows dy xh,  dbeta = sum_rows dy
//
// x (and dx, dres) bf16 or fp32 (a residual stream), y and dy bf16, the
// weights, statistics and their gradients fp32.  A row is held by a group of
// warps, 16 values per thread, so that the variance is the sum of squared
// differences from the mean (no cancellation) with x read once; everything is
// fp32 and rounded where it is stored.
//
// Both kernels are bound by HBM.  Blocks stay on their SM and walk over the
// rows; each warp copies its own values of the next rows into shared memory
// (cp.async) while the current row is reduced, so no barrier between warps waits
// for memory and a block holds two to three rows in flight.
//
// The backward pass reads x and dy once: each thread keeps its columns' dgamma
// and dbeta in registers over the block's rows, the block writes one partial
// row, and a second kernel adds the partial rows in block order.  The number of
// blocks depends on the sizes and the GPU alone, so the sums have one order
// and repeat bit for bit.
//
// Rows of any length take the same path: a row whose length is no multiple of 8
// starts somewhere inside a 16-byte word, so its words are loaded whole and the
// neighbouring rows' values in its first and last word masked.  A group's rows
// are a multiple of 8 apart, so that place, and with it the columns that a
// thread holds, stay the same.
//
// Measured, and the share of the measured copy rate: 32768 x 7168 bf16 forward
// 146 us (0.96), backward 249 us (0.84); 16384 x 4096 fp32 forward 66 us (0.91),
// backward with dres 146 us (0.96); 16384 x 4095 bf16 67 us (0.59) and 123 us
// (0.49).  At 16384 x 7168 bf16 the backward kernel executes 20.7 instructions per
// value (6.6 integer, 6.1 fp32) on the 14 warps of its 126 registers, with the
// issue slots 50 % busy and DRAM at 67 %; per instruction a warp waits 1.25 cycles
// on fixed latencies, 1.16 on shared memory and shuffles, 0.94 at the row's
// barrier and 0.60 on global memory.
#include <algorithm>

#include "norm_rows.cuh"

namespace mk {
namespace {

using namespace norm_rows;

constexpr int kStages = 3;           // rows of a group in the forward kernel's ring

template <typename T, int NV, bool kAligned>
__global__ void __launch_bounds__(kMaxWarps * 32, NV == 1 ? 2 : 1)
    layernorm_kernel(const T* __restrict__ x, const float* __restrict__ gamma, const float* __restrict__ beta,
                     uint32_t rows, int d, float eps, int warps, bf16* __restrict__ y, float* __restrict__ mean,
                     float* __restrict__ rstd) {
    using X = RingPart<T, NV>;
    extern __shared__ __align__(32) uint4 ring[];
    __shared__ float red[GroupSum<1>::kWords];
    const Place<kAligned> p(d, warps, NV);
    const GroupSum<1> group_sum(smem_u32(red), warps, p.gid);
    const float inv_d = 1.0f / static_cast<float>(d);
    const int64_t stride = static_cast<int64_t>(p.step) * d;
    f2 g[NV][4], b[NV][4];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        p.weights(gamma, v, g[v]);
        p.weights(beta, v, b[v]);
    }
    const uint32_t mine = smem_u32(ring) + (threadIdx.x >> 5) * (kStages * X::kBytes);
    const uint32_t to = mine + X::copy_at(), from = mine + X::read_at();
    const T* ahead = x + p.first(d) - X::before();
    uint32_t row_ahead = p.row0;
    const uint32_t near_end = p.near_end(rows, d);
    bf16* out = y + p.first(d);
    auto fetch = [&](uint32_t slot) {
        if (row_ahead < rows) X::copy(to + slot, ahead, p, row_ahead >= near_end);
        ahead += stride;
        row_ahead += p.step;
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch(i * X::kBytes);
    uint32_t slot = 0;
    for (uint32_t row = p.row0; row < rows; row += p.step, out += stride) {
        fetch(slot == 0 ? (kStages - 1) * X::kBytes : slot - X::kBytes);
        cp_async_wait<kStages - 1>();
        if (X::kShared) __syncwarp();
        const uint32_t stage = after(from + slot);
        f2 f[NV][4], s = both(0.0f), s2 = both(0.0f);
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (p.in(v)) {
                X::read(stage, v, f[v]);
                p.mask(v, f[v]);
                s = add2(s, add2(f[v][0], f[v][1]));
                s2 = add2(s2, add2(f[v][2], f[v][3]));
            }
        slot = slot == (kStages - 1) * X::kBytes ? 0 : slot + X::kBytes;
        s = add2(s, s2);
        float sum[1] = {s.x() + s.y()};
        group_sum(sum, 0);
        const float m = sum[0] * inv_d;
        s = s2 = both(0.0f);
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (p.in(v)) {
#pragma unroll
                for (int e = 0; e < 4; ++e) f[v][e] = add2(f[v][e], both(-m));
                p.mask(v, f[v]);
                s = fma2(f[v][0], f[v][0], fma2(f[v][1], f[v][1], s));
                s2 = fma2(f[v][2], f[v][2], fma2(f[v][3], f[v][3], s2));
            }
        s = add2(s, s2);
        sum[0] = s.x() + s.y();
        group_sum(sum, 1);
        const float rs = rsqrtf(fmaf(sum[0], inv_d, eps));
        if (p.col <= 0 && p.col > -8) {
            mean[row] = m;
            rstd[row] = rs;
        }
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (p.in(v)) {
#pragma unroll
                for (int e = 0; e < 4; ++e) f[v][e] = fma2(mul2(f[v][e], both(rs)), g[v][e], b[v][e]);
                p.store(v, out + kLaneStep * v, f[v], false);
            }
    }
}

// With 2 vectors a lane holds x - mean and r t over the row's sums; with 1 or 4
// x and dy are read from the ring a second time, for the registers go to gamma
// and the columns' sums.
template <typename T, int NV, bool kAligned, int STAGES>
__global__ void __launch_bounds__(kMaxWarps * 32, NV == 1 ? 2 : 1)
    layernorm_bwd_kernel(const bf16* __restrict__ dy, const T* __restrict__ x, const float* __restrict__ gamma,
                         const float* __restrict__ mean, const float* __restrict__ rstd, const T* __restrict__ dres,
                         uint32_t rows, int d, int warps, T* __restrict__ dx, float* __restrict__ part) {
    using X = RingPart<T, NV>;
    using Y = RingPart<bf16, NV>;
    constexpr bool kHold = NV == 2;
    extern __shared__ __align__(32) uint4 ring[];
    __shared__ float red[GroupSum<2>::kWords];
    const Place<kAligned> p(d, warps, NV);
    const GroupSum<2> group_sum(smem_u32(red), warps, p.gid);
    const uint32_t stage_bytes = X::kBytes + Y::kBytes + (dres != nullptr ? X::kBytes : 0);
    const float inv_d = 1.0f / static_cast<float>(d);
    const bool wide = (reinterpret_cast<uintptr_t>(dx) & 31) == 0;
    const int64_t stride = static_cast<int64_t>(p.step) * d;
    const uint32_t mine = smem_u32(ring) + (threadIdx.x >> 5) * (STAGES * stage_bytes);
    const uint32_t to = mine + X::copy_at(), from = mine + X::read_at();
    const uint32_t y_to = X::kBytes + Y::copy_at() - X::copy_at(), y_from = X::kBytes + Y::read_at() - X::read_at();
    int64_t at = p.first(d), ahead = at;
    uint32_t row_ahead = p.row0;
    const uint32_t near_end = p.near_end(rows, d);
    auto fetch = [&](uint32_t slot) {
        if (row_ahead < rows) {
            const bool last = row_ahead >= near_end;
            X::copy(to + slot, x + ahead - X::before(), p, last);
            Y::copy(to + slot + y_to, dy + ahead, p, last);
            if (dres != nullptr) X::copy(to + slot + X::kBytes + Y::kBytes, dres + ahead - X::before(), p, last);
        }
        ahead += stride;
        row_ahead += p.step;
        cp_async_commit();
    };
    f2 ag[NV][4], ab[NV][4], g[NV][4];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
#pragma unroll
        for (int e = 0; e < 4; ++e) ag[v][e] = ab[v][e] = both(0.0f);
        p.weights(gamma, v, g[v]);
    }
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) fetch(i * stage_bytes);
    const uint32_t last_slot = (STAGES - 1) * stage_bytes;
    uint32_t slot = 0;
    int buffer = 0;
    float r_next = p.row0 < rows ? __ldg(rstd + p.row0) : 0.0f, m_next = p.row0 < rows ? __ldg(mean + p.row0) : 0.0f;
    for (uint32_t row = p.row0; row < rows; row += p.step, at += stride) {
        if (X::kShared) __syncwarp();  // the slot was read by all lanes
        fetch(slot == 0 ? last_slot : slot - stage_bytes);
        const float r = r_next, m = -m_next;
        // (row0, step and this index without a sign, too, cost 12 % at 262144 x 256 bf16: registers)
        if (row + p.step < rows)
            r_next = __ldg(rstd + static_cast<int>(row + p.step)), m_next = __ldg(mean + static_cast<int>(row + p.step));
        cp_async_wait<STAGES - 1>();
        if (X::kShared) __syncwarp();
        uint32_t stage = after(from + slot);
        slot = slot == last_slot ? 0 : slot + stage_bytes;
        f2 st = both(0.0f), sc = both(0.0f);  // sums of r t and r t (x - mean)
        f2 cv[kHold ? NV : 1][4], tv[kHold ? NV : 1][4];  // x - mean, then r t
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (p.in(v)) {
                f2 (&c)[4] = cv[kHold ? v : 0];
                f2 y[4];
                X::read(stage, v, c);
                Y::read(stage + y_from, v, y);
#pragma unroll
                for (int e = 0; e < 4; ++e) c[e] = add2(c[e], both(m));
                p.mask(v, c);
                p.mask(v, y);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    ab[v][e] = add2(ab[v][e], y[e]);
                    y[e] = mul2(y[e], both(r));
                    ag[v][e] = fma2(y[e], c[e], ag[v][e]);
                    y[e] = mul2(y[e], g[v][e]);
                    st = add2(st, y[e]);
                    sc = fma2(y[e], c[e], sc);
                    if (kHold) tv[v][e] = y[e];
                }
            }
        float sum[2] = {st.x() + st.y(), sc.x() + sc.y()};
        group_sum(sum, buffer);
        buffer ^= 1;
        stage = after(stage);
        // dx = r t - (x - mean) r^2 sum(r t (x - mean)) / d - sum(r t) / d
        const f2 c0 = both(-sum[0] * inv_d), c1 = both(-r * (r * sum[1]) * inv_d);
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (p.in(v)) {
                f2 (&c)[4] = cv[kHold ? v : 0];
                f2 y[4];
                if (!kHold) {
                    X::read(stage, v, c);
                    Y::read(stage + y_from, v, y);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    c[e] = kHold ? add2(tv[v][e], fma2(c[e], c1, c0))
                                 : fma2(mul2(y[e], g[v][e]), both(r), fma2(add2(c[e], both(m)), c1, c0));
                if (dres != nullptr) {
                    X::read(stage + X::kBytes + Y::kBytes, v, y);
#pragma unroll
                    for (int e = 0; e < 4; ++e) c[e] = add2(c[e], y[e]);
                }
                p.store(v, dx + at + kLaneStep * v, c, wide);
            }
    }
    pdl_launch_dependents();  // the kernel that adds the partial rows
    // The block's partial row [dgamma d | dbeta d]: every group's sums side by
    // side in shared memory, added in group order.
    float* sums = reinterpret_cast<float*>(ring);
    const int groups = (blockDim.x >> 5) / warps;
    __syncthreads();  // the shared memory is no longer a ring
#pragma unroll
    for (int v = 0; v < NV; ++v)
        if (p.in(v))
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (p.has(v, e)) {
                    float* to = sums + p.gid * 2 * d + p.col + kLaneStep * v + e;
                    to[0] = (e & 1) ? ag[v][e >> 1].y() : ag[v][e >> 1].x();
                    to[d] = (e & 1) ? ab[v][e >> 1].y() : ab[v][e >> 1].x();
                }
    __syncthreads();
    float* out = part + static_cast<int64_t>(blockIdx.x) * 2 * d;
    for (int c = threadIdx.x; c < 2 * d; c += blockDim.x) {
        float t = sums[c];
        for (int q = 1; q < groups; ++q) t += sums[q * 2 * d + c];
        out[c] = t;
    }
}

// ------------------------------------------------------------------ host side

struct NormArgs {
    const void* x;
    const float* gamma;
    int rows, d;
    cudaStream_t s;
    // forward
    const float* beta;
    float eps;
    void* y;
    float *mean, *rstd;
    // backward
    const void *dy, *dres;
    void* dx;
    float *part, *dgamma, *dbeta;
};

template <typename T, int NV, bool kAligned>
cudaError_t launch_fwd(const NormArgs& a, RowShape r) {
    const Ring q = ring_shape(r, RingPart<T, NV>::kWords);  // 16384 fp32 values fit three times
    constexpr auto fn = layernorm_kernel<T, NV, kAligned>;
    const cudaError_t err = allow_smem<fn>();
    if (err != cudaSuccess) return err;
    fn<<<grid_blocks(r, a.rows, a.d, q.blocks * device_sm_count()), r.threads(), q.bytes, a.s>>>(
        static_cast<const T*>(a.x), a.gamma, a.beta, a.rows, a.d, a.eps, r.warps, static_cast<bf16*>(a.y), a.mean,
        a.rstd);
    return cudaGetLastError();
}

template <typename T, bool kAligned>
cudaError_t run_fwd(const NormArgs& a) {
    const RowShape r = row_shape(a.rows, a.d, true);
    return r.nv == 1   ? launch_fwd<T, 1, kAligned>(a, r)
           : r.nv == 2 ? launch_fwd<T, 2, kAligned>(a, r)
                       : launch_fwd<T, 4, kAligned>(a, r);
}

template <typename T, int NV, bool kAligned, int STAGES>
cudaError_t launch_bwd(const NormArgs& a, const RowShape& r, const Ring& q) {
    const size_t smem = std::max(q.bytes, 2 * sizeof(float) * static_cast<size_t>(a.d) * r.rows);
    const int most = std::min(q.blocks * device_sm_count(), kMaxBwdBlocks);
    constexpr auto fn = layernorm_bwd_kernel<T, NV, kAligned, STAGES>;
    cudaError_t err = allow_smem<fn>();
    const int64_t piece = piece_rows(r, grid_blocks(r, a.rows, a.d, most));
    for (int64_t row = 0; row < a.rows && err == cudaSuccess; row += piece) {
        const int rows = static_cast<int>(std::min<int64_t>(piece, a.rows - row));
        const int64_t at = row * a.d;
        const int blocks = grid_blocks(r, rows, a.d, most);
        const T* dres = static_cast<const T*>(a.dres);
        fn<<<blocks, r.threads(), smem, a.s>>>(static_cast<const bf16*>(a.dy) + at, static_cast<const T*>(a.x) + at, a.gamma,
                                               a.mean + row, a.rstd + row, dres != nullptr ? dres + at : nullptr, rows, a.d,
                                               r.warps, static_cast<T*>(a.dx) + at, a.part);
        err = cudaGetLastError();
        if (err == cudaSuccess) err = sum_partial_rows(a.part, blocks, 2 * a.d, a.d, a.dgamma, a.dbeta, a.s, row > 0);
    }
    return err;
}

template <typename T, bool kAligned>
cudaError_t run_bwd(const NormArgs& a) {
    RowShape r = row_shape(a.rows, a.d, false);
    const int xs = a.dres != nullptr ? 2 : 1;
    const Ring q = ring_shape(r, r.nv * (RingPart<T, 1>::kWords * xs + RingPart<bf16, 1>::kWords));
    if (q.stages == 1) return launch_bwd<T, 4, kAligned, 1>(a, r, q);  // fp32 rows of over 11000 values with dres
    if (q.stages == 2)
        return r.nv == 1   ? launch_bwd<T, 1, kAligned, 2>(a, r, q)
               : r.nv == 2 ? launch_bwd<T, 2, kAligned, 2>(a, r, q)
                           : launch_bwd<T, 4, kAligned, 2>(a, r, q);
    return r.nv == 1   ? launch_bwd<T, 1, kAligned, 3>(a, r, q)
           : r.nv == 2 ? launch_bwd<T, 2, kAligned, 3>(a, r, q)
                       : launch_bwd<T, 4, kAligned, 3>(a, r, q);
}

// The kernels for x's type and for rows that start a 16-byte word or not.
cudaError_t run(const NormArgs& a, int x_type, bool forward) {
    const bool aligned = a.d % 8 == 0;
    if (x_type == MK_TYPE_FP32)
        return forward ? (aligned ? run_fwd<float, true>(a) : run_fwd<float, false>(a))
                       : (aligned ? run_bwd<float, true>(a) : run_bwd<float, false>(a));
    return forward ? (aligned ? run_fwd<bf16, true>(a) : run_fwd<bf16, false>(a))
                   : (aligned ? run_bwd<bf16, true>(a) : run_bwd<bf16, false>(a));
}

mk_status check_norm(int64_t T, int d, int x_type) {
    if (T < 0 || d <= 0 || (x_type != MK_TYPE_BF16 && x_type != MK_TYPE_FP32)) return MK_ERR_INVALID_ARG;
    if (d > (d % 8 == 0 ? kMaxD : kMaxD - 8) || T >= (int64_t(1) << 31) || T * d >= (int64_t(1) << 40)) return MK_ERR_UNSUPPORTED;
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
    NormArgs a{};
    a.x = x, a.gamma = gamma, a.rows = static_cast<int>(T), a.d = d, a.s = static_cast<cudaStream_t>(stream);
    a.beta = beta, a.eps = eps, a.y = y, a.mean = mean, a.rstd = rstd;
    return run(a, x_type, true) == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}

extern "C" size_t mk_moe_layernorm_bwd_workspace_size(int64_t T, int d) {
    if (check_norm(T, d, MK_TYPE_BF16) != MK_OK) return 0;
    return 256 + static_cast<size_t>(std::min<int64_t>(T, kMaxBwdBlocks)) * 2 * d * sizeof(float);
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
    NormArgs a{};
    a.x = x, a.gamma = gamma, a.rows = static_cast<int>(T), a.d = d, a.s = s;
    a.mean = const_cast<float*>(mean), a.rstd = const_cast<float*>(rstd);
    a.dy = dy, a.dres = dres, a.dx = dx;
    a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + 256);
    a.dgamma = dgamma, a.dbeta = dbeta;
    return run(a, x_type, false) == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}
