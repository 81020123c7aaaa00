// rmsnorm.cu -- root-mean-square norm with the residual's addition, its output in
// bf16 and in 8 bits, and its backward pass.
//
//   h = x + add                    (rounded to x's type; h = x without add)
//   rstd = 1 / sqrt(sum h^2 / d + eps),  y = h rstd gamma
//   codes, scales: y in e4m3 with a scale per 128 values (quant8.cuh)
//   t = dy gamma
//   dx = rstd t - h rstd^3 sum(t h) / d  (+ dres),  dgamma = sum_rows dy h rstd
//
// x (and h, dx, dres) bf16 or fp32 (a residual stream), add (the block's output), y
// and dy bf16, gamma, rstd and dgamma fp32.  The norm is that of the rounded h, which
// the backward pass reads; y is rounded once to each output, from fp32.
//
// Both kernels are bound by HBM and walk over the rows as the layer norm's do
// (norm_rows.cuh): blocks stay on their SM, each warp copies its own values of the
// next rows into shared memory while the current row is reduced, and the row's sum
// is the only point where its warps meet.  A block of 128 values lies in 16
// neighbouring lanes' vectors, so its scale takes four shuffles and no barrier.
// 32768 x 7168 bf16: forward with an addition 302 us (0.91 of the copy rate), with codes
// as well 355 to 368 (0.85 to 0.88; 28 warps with half the values each were up to 5 % slower), with codes
// alone 264 (0.92), backward with a residual 277 (0.98).
#include <algorithm>

#include "norm_rows.cuh"
#include "quant8.cuh"

namespace mk {
namespace {

using namespace norm_rows;

struct RmsOut {
    void* h;         // null: no add
    bf16* y;         // or null
    float* rstd;
    uint8_t* codes;  // or null
    float* scales;
    int pitch;
};

// Rounded to the residual stream's type.
__device__ __forceinline__ f2 rounded(f2 v, const float*) { return v; }
__device__ __forceinline__ f2 rounded(f2 v, const bf16*) {
    const uint32_t w = pack_bf16x2(v.x(), v.y());
    return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

template <typename T, int NV, bool kAligned, int STAGES, bool kQ8>
__global__ void __launch_bounds__(kMaxWarps * 32, NV == 1 ? 2 : 1)
    rmsnorm_kernel(const T* __restrict__ x, const bf16* __restrict__ add, const float* __restrict__ gamma, uint32_t rows,
                   int d, float eps, int warps, const RmsOut out) {
    using X = RingPart<T, NV>;
    using Y = RingPart<bf16, NV>;
    extern __shared__ __align__(32) uint4 ring[];
    __shared__ float red[GroupSum<1>::kWords];
    const Place<kAligned> p(d, warps, NV);
    const GroupSum<1> group_sum(smem_u32(red), warps, p.gid);
    const float inv_d = 1.0f / static_cast<float>(d);
    const int64_t stride = static_cast<int64_t>(p.step) * d;
    const uint32_t stage_bytes = X::kBytes + (add != nullptr ? Y::kBytes : 0);
    const uint32_t last_slot = (STAGES - 1) * stage_bytes;
    const bool wide = (reinterpret_cast<uintptr_t>(out.h) & 31) == 0;
    f2 g[NV][4];
#pragma unroll
    for (int v = 0; v < NV; ++v) p.weights(gamma, v, g[v]);
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
            if (add != nullptr) Y::copy(to + slot + y_to, add + ahead, p, last);
        }
        ahead += stride;
        row_ahead += p.step;
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) fetch(i * stage_bytes);
    uint32_t slot = 0;
    int buffer = 0;
    for (uint32_t row = p.row0; row < rows; row += p.step, at += stride) {
        fetch(slot == 0 ? last_slot : slot - stage_bytes);
        cp_async_wait<STAGES - 1>();
        if (X::kShared) __syncwarp();
        const uint32_t stage = after(from + slot);
        slot = slot == last_slot ? 0 : slot + stage_bytes;
        f2 f[NV][4], s = both(0.0f), s2 = both(0.0f);
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (p.in(v)) {
                X::read(stage, v, f[v]);
                if (add != nullptr) {
                    f2 a[4];
                    Y::read(stage + y_from, v, a);
#pragma unroll
                    for (int e = 0; e < 4; ++e) f[v][e] = rounded(add2(f[v][e], a[e]), x);
                    p.store(v, static_cast<T*>(out.h) + at + kLaneStep * v, f[v], wide);
                }
                p.mask(v, f[v]);
                s = fma2(f[v][0], f[v][0], fma2(f[v][1], f[v][1], s));
                s2 = fma2(f[v][2], f[v][2], fma2(f[v][3], f[v][3], s2));
            }
        s = add2(s, s2);
        float sum[1] = {s.x() + s.y()};
        group_sum(sum, buffer);
        buffer ^= 1;
        const float rs = rsqrtf(fmaf(sum[0], inv_d, eps));
        if (p.col <= 0 && p.col > -8) out.rstd[row] = rs;
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (p.in(v)) {
#pragma unroll
                for (int e = 0; e < 4; ++e) f[v][e] = mul2(mul2(f[v][e], both(rs)), g[v][e]);
                if (out.y != nullptr) p.store(v, out.y + at + kLaneStep * v, f[v], false);
            }
        if constexpr (kQ8) {
            float q[NV][8], scale[NV];
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    q[v][2 * e] = p.in(v) ? f[v][e].x() : 0.0f;
                    q[v][2 * e + 1] = p.in(v) ? f[v][e].y() : 0.0f;
                }
            quant8::block_scales<NV, 8, 16>(q, scale);
#pragma unroll
            for (int v = 0; v < NV; ++v)
                if (p.in(v)) {
                    uint32_t c[2];
                    quant8::encode(q[v], scale[v], c);
                    *reinterpret_cast<uint2*>(out.codes + at + kLaneStep * v) = make_uint2(c[0], c[1]);
                    if ((threadIdx.x & 15) == 0)
                        out.scales[static_cast<int64_t>(row) * out.pitch + ((p.col + kLaneStep * v) / kScaleBlock)] = scale[v];
                }
        }
        if (kQ8 && p.col == 0)
            for (int b = (d + kScaleBlock - 1) / kScaleBlock; b < out.pitch; ++b)
                out.scales[static_cast<int64_t>(row) * out.pitch + b] = 0.0f;
    }
}

// With 2 vectors a lane holds h and r t over the row's sum; with 1 or 4 h and dy are
// read from the ring a second time (as in the layer norm's backward kernel).
template <typename T, int NV, bool kAligned, int STAGES>
__global__ void __launch_bounds__(kMaxWarps * 32, NV == 1 ? 2 : 1)
    rmsnorm_bwd_kernel(const bf16* __restrict__ dy, const T* __restrict__ h, const float* __restrict__ gamma,
                       const float* __restrict__ rstd, const T* __restrict__ dres, uint32_t rows, int d, int warps,
                       T* __restrict__ dx, float* __restrict__ part) {
    using X = RingPart<T, NV>;
    using Y = RingPart<bf16, NV>;
    constexpr bool kHold = NV == 2;
    extern __shared__ __align__(32) uint4 ring[];
    __shared__ float red[GroupSum<1>::kWords];
    const Place<kAligned> p(d, warps, NV);
    const GroupSum<1> group_sum(smem_u32(red), warps, p.gid);
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
            X::copy(to + slot, h + ahead - X::before(), p, last);
            Y::copy(to + slot + y_to, dy + ahead, p, last);
            if (dres != nullptr) X::copy(to + slot + X::kBytes + Y::kBytes, dres + ahead - X::before(), p, last);
        }
        ahead += stride;
        row_ahead += p.step;
        cp_async_commit();
    };
    f2 ag[NV][4], g[NV][4];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
#pragma unroll
        for (int e = 0; e < 4; ++e) ag[v][e] = both(0.0f);
        p.weights(gamma, v, g[v]);
    }
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) fetch(i * stage_bytes);
    const uint32_t last_slot = (STAGES - 1) * stage_bytes;
    uint32_t slot = 0;
    int buffer = 0;
    float r_next = p.row0 < rows ? __ldg(rstd + p.row0) : 0.0f;
    for (uint32_t row = p.row0; row < rows; row += p.step, at += stride) {
        if (X::kShared) __syncwarp();  // the slot was read by all lanes
        fetch(slot == 0 ? last_slot : slot - stage_bytes);
        const float r = r_next;
        if (row + p.step < rows) r_next = __ldg(rstd + static_cast<int>(row + p.step));
        cp_async_wait<STAGES - 1>();
        if (X::kShared) __syncwarp();
        uint32_t stage = after(from + slot);
        slot = slot == last_slot ? 0 : slot + stage_bytes;
        f2 sc = both(0.0f);  // sum of r t h
        f2 cv[kHold ? NV : 1][4], tv[kHold ? NV : 1][4];  // h, and r t
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (p.in(v)) {
                f2 (&c)[4] = cv[kHold ? v : 0];
                f2 y[4];
                X::read(stage, v, c);
                Y::read(stage + y_from, v, y);
                p.mask(v, c);
                p.mask(v, y);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    y[e] = mul2(y[e], both(r));
                    ag[v][e] = fma2(y[e], c[e], ag[v][e]);
                    y[e] = mul2(y[e], g[v][e]);
                    sc = fma2(y[e], c[e], sc);
                    if (kHold) tv[v][e] = y[e];
                }
            }
        float sum[1] = {sc.x() + sc.y()};
        group_sum(sum, buffer);
        buffer ^= 1;
        stage = after(stage);
        // dx = r t - h r^2 sum(r t h) / d
        const f2 c1 = both(-r * (r * sum[0]) * inv_d);
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
                    c[e] = fma2(c[e], c1, kHold ? tv[v][e] : mul2(mul2(y[e], both(r)), g[v][e]));
                if (dres != nullptr) {
                    X::read(stage + X::kBytes + Y::kBytes, v, y);
#pragma unroll
                    for (int e = 0; e < 4; ++e) c[e] = add2(c[e], y[e]);
                }
                p.store(v, dx + at + kLaneStep * v, c, wide);
            }
    }
    pdl_launch_dependents();  // the kernel that adds the partial rows
    // The block's partial row of dgamma: every group's sums side by side in shared
    // memory, added in group order.
    float* sums = reinterpret_cast<float*>(ring);
    const int groups = (blockDim.x >> 5) / warps;
    __syncthreads();  // the shared memory is no longer a ring
#pragma unroll
    for (int v = 0; v < NV; ++v)
        if (p.in(v))
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (p.has(v, e))
                    sums[p.gid * d + p.col + kLaneStep * v + e] = (e & 1) ? ag[v][e >> 1].y() : ag[v][e >> 1].x();
    __syncthreads();
    float* out = part + static_cast<int64_t>(blockIdx.x) * d;
    for (int c = threadIdx.x; c < d; c += blockDim.x) {
        float t = sums[c];
        for (int q = 1; q < groups; ++q) t += sums[q * d + c];
        out[c] = t;
    }
}

// ------------------------------------------------------------------ host side

struct RmsArgs {
    const void* x;  // backward: h
    const float* gamma;
    int rows, d;
    cudaStream_t s;
    // forward
    const void* add;
    float eps;
    RmsOut out;
    // backward
    const float* rstd;
    const void *dy, *dres;
    void* dx;
    float *part, *dgamma;
};

// A ring of three stages, with fewer rows per block where they do not fit; two for
// fp32 rows of over 12000 values with an addition, which do not fit three times.
Ring forward_ring(RowShape& s, int words) {
    const auto stage = [&] { return 16 * static_cast<size_t>(words) * s.warps * s.rows; };
    Ring r;
    r.blocks = s.nv == 1 && stage() * 3 * 2 <= kSmSmem ? 2 : 1;
    while (s.rows > 1 && stage() * 3 * r.blocks > kSmSmem) --s.rows;
    r.stages = stage() * 3 * r.blocks <= kSmSmem ? 3 : 2;
    r.bytes = stage() * r.stages;
    return r;
}

template <typename T, int NV, bool kAligned, int STAGES, bool kQ8>
cudaError_t launch_fwd_kernel(const RmsArgs& a, const RowShape& r, const Ring& q) {
    constexpr auto fn = rmsnorm_kernel<T, NV, kAligned, STAGES, kQ8>;
    const cudaError_t err = allow_smem<fn>();
    if (err != cudaSuccess) return err;
    fn<<<grid_blocks(r, a.rows, a.d, q.blocks * device_sm_count()), r.threads(), q.bytes, a.s>>>(
        static_cast<const T*>(a.x), static_cast<const bf16*>(a.add), a.gamma, a.rows, a.d, a.eps, r.warps, a.out);
    return cudaGetLastError();
}

template <typename T, int NV, bool kAligned, bool kQ8>
cudaError_t launch_fwd(const RmsArgs& a, RowShape r) {
    const Ring q = forward_ring(r, RingPart<T, NV>::kWords + (a.add != nullptr ? RingPart<bf16, NV>::kWords : 0));
    if constexpr (sizeof(T) == 4 && NV == 4)  // others fit three times
        if (q.stages == 2) return launch_fwd_kernel<T, NV, kAligned, 2, kQ8>(a, r, q);
    return launch_fwd_kernel<T, NV, kAligned, 3, kQ8>(a, r, q);
}

template <typename T, bool kAligned, bool kQ8>
cudaError_t run_fwd(const RmsArgs& a) {
    const RowShape r = row_shape(a.rows, a.d, true);
    return r.nv == 1   ? launch_fwd<T, 1, kAligned, kQ8>(a, r)
           : r.nv == 2 ? launch_fwd<T, 2, kAligned, kQ8>(a, r)
                       : launch_fwd<T, 4, kAligned, kQ8>(a, r);
}

template <typename T>
cudaError_t run_fwd(const RmsArgs& a) {
    if (a.out.codes != nullptr) return run_fwd<T, true, true>(a);  // d is a multiple of 64
    return a.d % 8 == 0 ? run_fwd<T, true, false>(a) : run_fwd<T, false, false>(a);
}

template <typename T, int NV, bool kAligned, int STAGES>
cudaError_t launch_bwd(const RmsArgs& a, const RowShape& r, const Ring& q) {
    const size_t smem = std::max(q.bytes, sizeof(float) * static_cast<size_t>(a.d) * r.rows);
    const int most = std::min(q.blocks * device_sm_count(), kMaxBwdBlocks);
    constexpr auto fn = rmsnorm_bwd_kernel<T, NV, kAligned, STAGES>;
    cudaError_t err = allow_smem<fn>();
    const int64_t piece = piece_rows(r, grid_blocks(r, a.rows, a.d, most));
    for (int64_t row = 0; row < a.rows && err == cudaSuccess; row += piece) {
        const int rows = static_cast<int>(std::min<int64_t>(piece, a.rows - row));
        const int64_t at = row * a.d;
        const int blocks = grid_blocks(r, rows, a.d, most);
        const T* dres = static_cast<const T*>(a.dres);
        fn<<<blocks, r.threads(), smem, a.s>>>(static_cast<const bf16*>(a.dy) + at, static_cast<const T*>(a.x) + at, a.gamma,
                                               a.rstd + row, dres != nullptr ? dres + at : nullptr, rows, a.d, r.warps,
                                               static_cast<T*>(a.dx) + at, a.part);
        err = cudaGetLastError();
        if (err == cudaSuccess) err = sum_partial_rows(a.part, blocks, a.d, a.d, a.dgamma, nullptr, a.s, row > 0);
    }
    return err;
}

template <typename T, bool kAligned>
cudaError_t run_bwd(const RmsArgs& a) {
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

template <typename T>
cudaError_t run_bwd(const RmsArgs& a) {
    return a.d % 8 == 0 ? run_bwd<T, true>(a) : run_bwd<T, false>(a);
}

mk_status check_rms(int64_t T, int d, int x_type) {
    if (T < 0 || d <= 0 || (x_type != MK_TYPE_BF16 && x_type != MK_TYPE_FP32)) return MK_ERR_INVALID_ARG;
    if (d > (d % 8 == 0 ? kMaxD : kMaxD - 8) || T >= (int64_t(1) << 31) || T * d >= (int64_t(1) << 40)) return MK_ERR_UNSUPPORTED;
    return MK_OK;
}

}  // namespace
}  // namespace mk

using namespace mk;

extern "C" mk_status mk_moe_rmsnorm(const void* x, int x_type, const void* add, const float* gamma, int64_t T, int d,
                                    float eps, void* h, void* y, float* rstd, uint8_t* codes, float* scales,
                                    void* stream) {
    const mk_status st = check_rms(T, d, x_type);
    if (st != MK_OK) return st;
    if (!(eps >= 0.0f) || (codes == nullptr) != (scales == nullptr) || (codes != nullptr && d % 64 != 0))
        return MK_ERR_INVALID_ARG;
    if (T == 0) return MK_OK;
    if (!x || !gamma || !rstd || (!y && !codes) || (add == nullptr) != (h == nullptr)) return MK_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(add) || !aligned16(gamma) || !aligned16(h) || !aligned16(y) || !aligned16(codes))
        return MK_ERR_INVALID_ARG;
    if (!device_is_sm103()) return MK_ERR_UNSUPPORTED;
    RmsArgs a{};
    a.x = x, a.gamma = gamma, a.rows = static_cast<int>(T), a.d = d, a.s = static_cast<cudaStream_t>(stream);
    a.add = add, a.eps = eps;
    a.out = RmsOut{h, static_cast<bf16*>(y), rstd, codes, scales, scale_pitch(d)};
    const cudaError_t err = x_type == MK_TYPE_FP32 ? run_fwd<float>(a) : run_fwd<bf16>(a);
    return err == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}

extern "C" size_t mk_moe_rmsnorm_bwd_workspace_size(int64_t T, int d) {
    if (check_rms(T, d, MK_TYPE_BF16) != MK_OK) return 0;
    return 256 + static_cast<size_t>(std::min<int64_t>(T, kMaxBwdBlocks)) * d * sizeof(float);
}

extern "C" mk_status mk_moe_rmsnorm_bwd(const void* dy, const void* h, int x_type, const float* gamma,
                                        const float* rstd, const void* dres, int64_t T, int d, void* dx, float* dgamma,
                                        void* ws, size_t ws_bytes, void* stream) {
    const mk_status st = check_rms(T, d, x_type);
    if (st != MK_OK) return st;
    if (!dgamma) return MK_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T > 0) {
        if (!dy || !h || !gamma || !rstd || !dx) return MK_ERR_INVALID_ARG;
        if (!aligned16(dy) || !aligned16(h) || !aligned16(gamma) || !aligned16(dx) || !aligned16(dres))
            return MK_ERR_INVALID_ARG;
        if (ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0 ||
            ws_bytes < mk_moe_rmsnorm_bwd_workspace_size(T, d))
            return MK_ERR_WORKSPACE;
    }
    if (!device_is_sm103()) return MK_ERR_UNSUPPORTED;
    if (T == 0)  // no rows: the weight's gradient is zero
        return cudaMemsetAsync(dgamma, 0, sizeof(float) * d, s) == cudaSuccess ? MK_OK : MK_ERR_CUDA;
    RmsArgs a{};
    a.x = h, a.gamma = gamma, a.rows = static_cast<int>(T), a.d = d, a.s = s;
    a.rstd = rstd, a.dy = dy, a.dres = dres, a.dx = dx;
    a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + 256);
    a.dgamma = dgamma;
    return (x_type == MK_TYPE_FP32 ? run_bwd<float>(a) : run_bwd<bf16>(a)) == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}
