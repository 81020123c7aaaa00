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
// rows; each thread copies its own values of the next rows into shared memory
// (cp.async) while the current row is reduced, so no barrier waits for memory
// and a block holds two to three rows in flight.
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
#include <algorithm>
#include <numeric>

#include "mk_device.cuh"
#include "mk_internal.h"

namespace mk {
namespace {

constexpr int kMaxD = 16384;  // 16 warps of 4 vectors; 8 less where a row's first word may start before it
constexpr int kMaxWarps = 16;    // per block and per row
constexpr int kStages = 3;           // rows of a group in the forward kernel's ring
constexpr int kMaxBwdBlocks = 304;  // partial rows

// ---------------------------------------------------------------- packed fp32 pairs

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

// ---------------------------------------------------------------- eight values

// 16-byte words of eight values, and the values.
template <typename T>
constexpr int kWords8 = 8 * sizeof(T) / 16;

__device__ __forceinline__ void unpack(const uint4 (&w)[1], f2 (&f)[4]) {  // bf16
    const uint32_t q[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = f2(__uint_as_float(q[i] << 16), __uint_as_float(q[i] & 0xffff0000u));
}
__device__ __forceinline__ void unpack(const uint4 (&w)[2], f2 (&f)[4]) {  // fp32
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        f[2 * i] = f2(__uint_as_float(w[i].x), __uint_as_float(w[i].y));
        f[2 * i + 1] = f2(__uint_as_float(w[i].z), __uint_as_float(w[i].w));
    }
}

__device__ __forceinline__ void store8(bf16* p, const f2 (&f)[4]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0].x(), f[0].y()), pack_bf16x2(f[1].x(), f[1].y()),
                                              pack_bf16x2(f[2].x(), f[2].y()), pack_bf16x2(f[3].x(), f[3].y()));
}
__device__ __forceinline__ void store8(float* p, const f2 (&f)[4]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0].x(), f[0].y(), f[1].x(), f[1].y());
    reinterpret_cast<float4*>(p)[1] = make_float4(f[2].x(), f[2].y(), f[3].x(), f[3].y());
}
__device__ __forceinline__ void store1(bf16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }

// ---------------------------------------------------------------- sums over a row

template <int N>
__device__ __forceinline__ void warp_sums(float (&v)[N]) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
}

// Sums of N values over a group of `warps` consecutive warps (group `gid` of
// the block), the same bits in every thread: a shuffle tree inside each warp,
// then the same tree over the warps' sums (a chain over up to 16 warps took
// longer than all the rest of a row).  The group alone meets at its named
// barrier.  `red` holds N values per warp of the group and is not written again
// before the barrier of another call with another `red`.
template <int N>
__device__ __forceinline__ void group_sums(float (&v)[N], int warps, int gid, float (*red)[kMaxWarps]) {
    warp_sums(v);
    if (warps == 1) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) red[i][warp] = v[i];
    asm volatile("bar.sync %0, %1;" ::"r"(gid + 1), "r"(warps * 32) : "memory");
    const int w0 = gid * warps;
    const int tree = warps > 8 ? 16 : warps > 4 ? 8 : warps > 2 ? 4 : 2;  // every lane sums `tree` of them
    const int q = lane & (tree - 1);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = q < warps ? red[i][w0 + q] : 0.0f;
    for (int o = tree >> 1; o >= 1; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
}

// ---------------------------------------------------------------- rows
//
// A warp owns 256 NV consecutive columns of its row; lane l's vector v is the
// eight values from column 256 v + 8 l of them (shifted by the row's start in
// its first word), so every offset below is a constant.  One stage of the ring
// holds a row per group: per warp and tensor, NV vectors of 32 lanes, each
// thread reading only what it copied itself.

constexpr int kLaneStep = 256;  // columns between a lane's vectors

// Where a thread stands: its row group, its first vector's first column (from
// -7: the first word may start in the row before), and its group's rows row0,
// row0 + step, ... below `rows`.  kAligned: d is a multiple of 8, every row
// starts a word.
template <bool kAligned>
struct Place {
    int gid, col, left, row0, step, steps;  // left: columns from the first vector to the row's end
    __device__ __forceinline__ Place(int rows, int d, int warps, int nv) {
        const int warp = threadIdx.x >> 5;
        const int groups = (blockDim.x >> 5) / warps;
        gid = warp / warps;
        row0 = blockIdx.x * groups + gid;
        step = gridDim.x * groups;
        steps = row0 < rows ? (rows - row0 + step - 1) / step : 0;
        const int start = kAligned ? 0 : static_cast<int>((static_cast<int64_t>(row0) * d) & 7);
        col = (warp - gid * warps) * (kLaneStep * nv) + 8 * (threadIdx.x & 31) - start;
        left = d - col;
    }
    __device__ __forceinline__ int64_t first(int d) const { return static_cast<int64_t>(row0) * d + col; }
    __device__ __forceinline__ bool in(int v) const { return kLaneStep * v < left; }
    __device__ __forceinline__ bool whole(int v) const {
        return kAligned || ((v > 0 || col >= 0) && kLaneStep * v + 8 <= left);
    }
    __device__ __forceinline__ bool has(int v, int e) const {  // value e of vector v is the row's
        return kAligned ? kLaneStep * v < left : (v > 0 || col + e >= 0) && kLaneStep * v + e < left;
    }
    // Values outside the row become zero (NaN of another row included).
    __device__ __forceinline__ void mask(int v, f2 (&f)[4]) const {
        if (whole(v)) return;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            f[e] = f2(has(v, 2 * e) ? f[e].x() : 0.0f, has(v, 2 * e + 1) ? f[e].y() : 0.0f);
        }
    }
    // The row's values of vector v to p[0..7].
    template <typename T>
    __device__ __forceinline__ void store(int v, T* p, const f2 (&f)[4]) const {
        if (whole(v)) {
            store8(p, f);
            return;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (has(v, 2 * e)) store1(p + 2 * e, f[e].x());
            if (has(v, 2 * e + 1)) store1(p + 2 * e + 1, f[e].y());
        }
    }
    // The weights of vector v, zeros outside the row.  Away from the row's ends they are read
    // as the aligned words around them and shifted into place.
    __device__ __forceinline__ void weights(const float* w, int v, f2 (&f)[4]) const {
        const int c = col + kLaneStep * v;
        const int sh = kAligned ? 0 : c & 3;
        if (kAligned ? in(v) : c - sh >= 0 && c - sh + 12 <= col + left) {
            float q[12];
#pragma unroll
            for (int i = 0; i < (kAligned ? 2 : 3); ++i) {
                const float4 t = __ldg(reinterpret_cast<const float4*>(w + (c - sh)) + i);
                q[4 * i] = t.x, q[4 * i + 1] = t.y, q[4 * i + 2] = t.z, q[4 * i + 3] = t.w;
            }
            if (!kAligned) {
#pragma unroll
                for (int i = 0; i < 11; ++i) q[i] = (sh & 1) ? q[i + 1] : q[i];
#pragma unroll
                for (int i = 0; i < 9; ++i) q[i] = (sh & 2) ? q[i + 2] : q[i];
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = f2(q[2 * e], q[2 * e + 1]);
            return;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            f[e] = f2(has(v, 2 * e) ? __ldg(w + c + 2 * e) : 0.0f, has(v, 2 * e + 1) ? __ldg(w + c + 2 * e + 1) : 0.0f);
    }
};

template <typename T, int NV>
struct RingPart {
    static constexpr int kW = kWords8<T>;
    static constexpr int kWords = NV * kW * 32;  // 16-byte words per warp and stage

    // `slot`: this lane's first word; `row`: its first vector.  The tensor's last
    // word is read up to the tensor's end only.
    template <bool kAligned>
    static __device__ __forceinline__ void copy(uint4* slot, const T* row, const Place<kAligned>& p, bool last) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (p.in(v)) {
                const int bytes = (p.left - kLaneStep * v) * static_cast<int>(sizeof(T));
#pragma unroll
                for (int q = 0; q < kW; ++q) {
                    const uint4* src = reinterpret_cast<const uint4*>(row + kLaneStep * v) + q;
                    if (kAligned || !last || bytes >= 16 * (q + 1))
                        cp_async16(slot + (v * kW + q) * 32, src);
                    else if (bytes > 16 * q)
                        cp_async16_part(slot + (v * kW + q) * 32, src, bytes - 16 * q);
                }
            }
    }
    static __device__ __forceinline__ void read(const uint4* slot, int v, f2 (&f)[4]) {
        uint4 w[kW];
#pragma unroll
        for (int q = 0; q < kW; ++q) w[q] = slot[(v * kW + q) * 32];
        unpack(w, f);
    }
};

template <typename T, int NV, bool kAligned>
__global__ void __launch_bounds__(kMaxWarps * 32, NV == 1 ? 2 : 1)
    layernorm_kernel(const T* __restrict__ x, const float* __restrict__ gamma, const float* __restrict__ beta,
                     int rows, int d, float eps, int warps, bf16* __restrict__ y, float* __restrict__ mean,
                     float* __restrict__ rstd) {
    using X = RingPart<T, NV>;
    extern __shared__ uint4 ring[];
    __shared__ float red[2][kMaxWarps];
    const Place<kAligned> p(rows, d, warps, NV);
    const float inv_d = 1.0f / static_cast<float>(d);
    const int64_t stride = static_cast<int64_t>(p.step) * d;
    f2 g[NV][4], b[NV][4];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        p.weights(gamma, v, g[v]);
        p.weights(beta, v, b[v]);
    }
    uint4* mine = ring + (threadIdx.x >> 5) * (kStages * X::kWords) + (threadIdx.x & 31);
    const T* ahead = x + p.first(d);
    bf16* out = y + p.first(d);
    auto fetch = [&](int i, int slot) {
        if (i < p.steps) X::copy(mine + slot * X::kWords, ahead, p, p.row0 + i * p.step == rows - 1);
        ahead += stride;
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch(i, i);
    int slot = 0;
    for (int i = 0; i < p.steps; ++i, out += stride) {
        fetch(i + kStages - 1, slot == 0 ? kStages - 1 : slot - 1);
        cp_async_wait<kStages - 1>();
        f2 f[NV][4], s = both(0.0f), s2 = both(0.0f);
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (p.in(v)) {
                X::read(mine + slot * X::kWords, v, f[v]);
                p.mask(v, f[v]);
                s = add2(s, add2(f[v][0], f[v][1]));
                s2 = add2(s2, add2(f[v][2], f[v][3]));
            }
        if (++slot == kStages) slot = 0;
        s = add2(s, s2);
        float sum[1] = {s.x() + s.y()};
        group_sums(sum, warps, p.gid, &red[0]);
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
        group_sums(sum, warps, p.gid, &red[1]);
        const float rs = rsqrtf(fmaf(sum[0], inv_d, eps));
        if (p.col <= 0 && p.col > -8) {
            mean[p.row0 + i * p.step] = m;
            rstd[p.row0 + i * p.step] = rs;
        }
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (p.in(v)) {
#pragma unroll
                for (int e = 0; e < 4; ++e) f[v][e] = fma2(mul2(f[v][e], both(rs)), g[v][e], b[v][e]);
                p.store(v, out + kLaneStep * v, f[v]);
            }
    }
}

// x and dy are read from the ring twice, before and after the row's sums,
// rather than held: the registers go to gamma and the columns' sums.
template <typename T, int NV, bool kAligned, int STAGES>
__global__ void __launch_bounds__(kMaxWarps * 32, NV == 1 ? 2 : 1)
    layernorm_bwd_kernel(const bf16* __restrict__ dy, const T* __restrict__ x, const float* __restrict__ gamma,
                         const float* __restrict__ mean, const float* __restrict__ rstd, const T* __restrict__ dres,
                         int rows, int d, int warps, T* __restrict__ dx, float* __restrict__ part) {
    using X = RingPart<T, NV>;
    using Y = RingPart<bf16, NV>;
    extern __shared__ uint4 ring[];
    __shared__ float red[2][2][kMaxWarps];
    const Place<kAligned> p(rows, d, warps, NV);
    const int words = X::kWords + Y::kWords + (dres != nullptr ? X::kWords : 0);
    const float inv_d = 1.0f / static_cast<float>(d);
    const int64_t stride = static_cast<int64_t>(p.step) * d;
    int64_t at = p.first(d);
    uint4* mine = ring + (threadIdx.x >> 5) * (STAGES * words) + (threadIdx.x & 31);
    auto fetch = [&](int i, int slot) {
        if (i < p.steps) {
            uint4* s = mine + slot * words;
            const bool last = p.row0 + i * p.step == rows - 1;
            const int64_t ahead = p.first(d) + i * stride;
            X::copy(s, x + ahead, p, last);
            Y::copy(s + X::kWords, dy + ahead, p, last);
            if (dres != nullptr) X::copy(s + X::kWords + Y::kWords, dres + ahead, p, last);
        }
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
    for (int i = 0; i < STAGES - 1; ++i) fetch(i, i);
    int slot = 0, row = p.row0;
    float r_next = p.steps > 0 ? __ldg(rstd + row) : 0.0f, m_next = p.steps > 0 ? __ldg(mean + row) : 0.0f;
    for (int i = 0; i < p.steps; ++i, at += stride) {
        fetch(i + STAGES - 1, slot == 0 ? STAGES - 1 : slot - 1);
        const float r = r_next, m = -m_next;
        row += p.step;
        if (i + 1 < p.steps) r_next = __ldg(rstd + row), m_next = __ldg(mean + row);
        cp_async_wait<STAGES - 1>();
        const uint4* stage = mine + slot * words;
        if (++slot == STAGES) slot = 0;
        f2 st = both(0.0f), sc = both(0.0f);  // sums of t and t (x - mean)
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (p.in(v)) {
                f2 c[4], y[4];
                X::read(stage, v, c);
                Y::read(stage + X::kWords, v, y);
#pragma unroll
                for (int e = 0; e < 4; ++e) c[e] = add2(c[e], both(m));
                p.mask(v, c);
                p.mask(v, y);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const f2 t = mul2(y[e], g[v][e]);
                    ab[v][e] = add2(ab[v][e], y[e]);
                    ag[v][e] = fma2(mul2(y[e], both(r)), c[e], ag[v][e]);
                    st = add2(st, t);
                    sc = fma2(t, c[e], sc);
                }
            }
        float sum[2] = {st.x() + st.y(), sc.x() + sc.y()};
        group_sums(sum, warps, p.gid, red[i & 1]);
        // dx = r t - (x - mean) (r^3 sum(t (x - mean)) / d) - r sum t / d
        const f2 c0 = both(-r * sum[0] * inv_d), c1 = both(-r * (r * (r * sum[1])) * inv_d);
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (p.in(v)) {
                f2 c[4], y[4];
                X::read(stage, v, c);
                Y::read(stage + X::kWords, v, y);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    c[e] = fma2(mul2(y[e], g[v][e]), both(r), fma2(add2(c[e], both(m)), c1, c0));
                if (dres != nullptr) {
                    X::read(stage + X::kWords + Y::kWords, v, y);
#pragma unroll
                    for (int e = 0; e < 4; ++e) c[e] = add2(c[e], y[e]);
                }
                p.store(v, dx + at + kLaneStep * v, c);
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

// dgamma | dbeta = the blocks' partial rows [blocks][2 d], 32 columns per
// block: 8 slices of every eighth partial row, then the slices in order.
__global__ void __launch_bounds__(256) layernorm_bwd_sum_kernel(const float* __restrict__ part, int blocks, int d,
                                                                float* __restrict__ dgamma,
                                                                float* __restrict__ dbeta) {
    __shared__ float s[8][32];
    pdl_wait();  // the partial rows come from the kernel before
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float v = 0.0f;
    if (c < 2 * d)
#pragma unroll 8
        for (int b = slice; b < blocks; b += 8) v += part[static_cast<int64_t>(b) * 2 * d + c];
    s[slice][lane] = v;
    __syncthreads();
    if (slice == 0 && c < 2 * d) {
#pragma unroll
        for (int i = 1; i < 8; ++i) v += s[i][lane];
        (c < d ? dgamma + c : dbeta + (c - d))[0] = v;
    }
}

// ------------------------------------------------------------------ host side

// Warps per row, rows per block, and vectors of 8 values per lane.
struct RowShape {
    int warps, rows, nv;
    int threads() const { return warps * rows * 32; }
};
// A block has up to 16 warps.  Of 4, 2 and 1 vectors per lane the one is taken
// that uses most of them: the share of the lanes' vectors that lie in the row,
// times the share of 16 warps that whole row groups fill, times a weight from
// measurements.  Forward, 4 vectors share a thread's fixed work per row (sums,
// copies) best (32768 x 7168 bf16: 155 us, with 2 vectors 232); backward, the
// columns' sums of 4 vectors do not fit the registers (307 us, with 2 262).
RowShape row_shape(int64_t rows, int d, bool forward) {
    const int n = d % 8 == 0 ? d : d + 7;  // the row's words may start up to 7 values before it
    RowShape best{};
    double most = 0.0;
    for (const int nv : {4, 2, 1}) {
        RowShape s;
        s.nv = nv;
        s.warps = (n + kLaneStep * nv - 1) / (kLaneStep * nv);
        if (s.warps > kMaxWarps) continue;
        s.rows = kMaxWarps / s.warps;
        const double use = static_cast<double>(n) * s.rows / (kLaneStep * nv * kMaxWarps) *
                           (forward ? (nv == 4 ? 1.0 : nv == 2 ? 0.9 : 0.75) : (nv == 4 ? 0.8 : nv == 2 ? 1.0 : 0.8));
        if (use > most) {
            most = use;
            best = s;
        }
    }
    // few rows: spread over all SMs
    best.rows = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(best.rows, (rows + device_sm_count() - 1) / device_sm_count())));
    return best;
}

constexpr size_t kSmSmem = 216 * 1024;  // of an SM's shared memory, for the rings of its blocks

// Blocks per SM (two of 16 warps with one vector per lane, for which the kernels'
// registers are bounded; one with more) and ring
// stages for `words` 16-byte words per warp and stage: three where they fit, two
// with fewer rows per block where not (the row ahead of 16 warps covers the
// latency; fewer warps do not keep up with the copies).
struct Ring {
    int blocks, stages;
    size_t bytes;
};
Ring ring_shape(RowShape& s, int words) {
    const auto stage = [&] { return 16 * static_cast<size_t>(words) * s.warps * s.rows; };
    Ring r;
    r.blocks = s.nv == 1 && stage() * 2 * 2 <= kSmSmem ? 2 : 1;
    while (s.rows > 1 && stage() * 2 * r.blocks > kSmSmem) --s.rows;
    r.stages = static_cast<int>(std::min<size_t>(3, kSmSmem / r.blocks / stage()));
    r.bytes = stage() * r.stages;
    return r;
}

// Blocks for `rows` rows, at most `most` (> 0): where a group takes more than
// one row, its rows are a multiple of 8 / gcd(d, 8) apart.
int grid_blocks(const RowShape& s, int64_t rows, int d, int most) {
    const int64_t chunks = (rows + s.rows - 1) / s.rows;
    if (chunks <= most) return static_cast<int>(chunks);
    const int apart = 8 / std::gcd(d, 8), unit = apart / std::gcd(s.rows, apart);
    return std::max(unit, most / unit * unit);
}

template <typename F>
cudaError_t allow_smem(F fn, size_t bytes) {
    return bytes <= 40 * 1024 ? cudaSuccess  // 48 KB with the static part need no leave
                              : cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                     static_cast<int>(bytes));
}

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
    float* part;
    int blocks;  // out: partial rows written
};

template <typename T, int NV>
cudaError_t launch_fwd(const NormArgs& a, RowShape r) {
    const Ring q = ring_shape(r, RingPart<T, NV>::kWords);  // 16384 fp32 values fit three times
    auto fn = a.d % 8 == 0 ? layernorm_kernel<T, NV, true> : layernorm_kernel<T, NV, false>;
    const cudaError_t err = allow_smem(fn, q.bytes);
    if (err != cudaSuccess) return err;
    fn<<<grid_blocks(r, a.rows, a.d, q.blocks * device_sm_count()), r.threads(), q.bytes, a.s>>>(
        static_cast<const T*>(a.x), a.gamma, a.beta, a.rows, a.d, a.eps, r.warps, static_cast<bf16*>(a.y), a.mean,
        a.rstd);
    return cudaGetLastError();
}

template <typename T>
cudaError_t run_fwd(const NormArgs& a) {
    const RowShape r = row_shape(a.rows, a.d, true);
    return r.nv == 1 ? launch_fwd<T, 1>(a, r) : r.nv == 2 ? launch_fwd<T, 2>(a, r) : launch_fwd<T, 4>(a, r);
}

template <typename T, int NV, int STAGES>
cudaError_t launch_bwd(NormArgs& a, const RowShape& r, const Ring& q) {
    const size_t smem = std::max(q.bytes, 2 * sizeof(float) * static_cast<size_t>(a.d) * r.rows);
    a.blocks = grid_blocks(r, a.rows, a.d, std::min(q.blocks * device_sm_count(), kMaxBwdBlocks));
    auto fn = a.d % 8 == 0 ? layernorm_bwd_kernel<T, NV, true, STAGES> : layernorm_bwd_kernel<T, NV, false, STAGES>;
    const cudaError_t err = allow_smem(fn, smem);
    if (err != cudaSuccess) return err;
    fn<<<a.blocks, r.threads(), smem, a.s>>>(static_cast<const bf16*>(a.dy), static_cast<const T*>(a.x), a.gamma,
                                             a.mean, a.rstd, static_cast<const T*>(a.dres), a.rows, a.d, r.warps,
                                             static_cast<T*>(a.dx), a.part);
    return cudaGetLastError();
}

template <typename T>
cudaError_t run_bwd(NormArgs& a) {
    RowShape r = row_shape(a.rows, a.d, false);
    const int xs = a.dres != nullptr ? 2 : 1;
    const Ring q = ring_shape(r, r.nv * (RingPart<T, 1>::kWords * xs + RingPart<bf16, 1>::kWords));
    if (q.stages == 1) return launch_bwd<T, 4, 1>(a, r, q);  // fp32 rows of over 11000 values with dres
    if (q.stages == 2)
        return r.nv == 1   ? launch_bwd<T, 1, 2>(a, r, q)
               : r.nv == 2 ? launch_bwd<T, 2, 2>(a, r, q)
                           : launch_bwd<T, 4, 2>(a, r, q);
    return r.nv == 1   ? launch_bwd<T, 1, 3>(a, r, q)
           : r.nv == 2 ? launch_bwd<T, 2, 3>(a, r, q)
                       : launch_bwd<T, 4, 3>(a, r, q);
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
    const cudaError_t err = x_type == MK_TYPE_FP32 ? run_fwd<float>(a) : run_fwd<bf16>(a);
    return err == cudaSuccess ? MK_OK : MK_ERR_CUDA;
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
    if ((x_type == MK_TYPE_FP32 ? run_bwd<float>(a) : run_bwd<bf16>(a)) != cudaSuccess) return MK_ERR_CUDA;
    const LaunchCfg lc(dim3(static_cast<unsigned>((2 * static_cast<int64_t>(d) + 31) / 32)), dim3(256), 0, s, true);
    if (cudaLaunchKernelEx(&lc.cfg, layernorm_bwd_sum_kernel, static_cast<const float*>(a.part), a.blocks, d, dgamma,
                           dbeta) != cudaSuccess)
        return MK_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}
