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
#include <atomic>
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

__device__ __forceinline__ void store8(bf16* p, const f2 (&f)[4], bool) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0].x(), f[0].y()), pack_bf16x2(f[1].x(), f[1].y()),
                                              pack_bf16x2(f[2].x(), f[2].y()), pack_bf16x2(f[3].x(), f[3].y()));
}
// One store of 32 bytes (whole sectors) where the tensor starts on a multiple of 32, else two.
__device__ __forceinline__ void store8(float* p, const f2 (&f)[4], bool wide) {
    if (wide) {
        asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(f[0].x()), "f"(f[0].y()),
                     "f"(f[1].x()), "f"(f[1].y()), "f"(f[2].x()), "f"(f[2].y()), "f"(f[3].x()), "f"(f[3].y())
                     : "memory");
        return;
    }
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0].x(), f[0].y(), f[1].x(), f[1].y());
    reinterpret_cast<float4*>(p)[1] = make_float4(f[2].x(), f[2].y(), f[3].x(), f[3].y());
}
__device__ __forceinline__ void store1(bf16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }

// ---------------------------------------------------------------- sums over a row

__device__ __forceinline__ void st_shared(uint32_t addr, float v) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ float ld_shared(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
// A read that the compiler may place freely between the point that `addr` comes
// from (see after()) and its use.
__device__ __forceinline__ uint4 ld_shared16(uint32_t addr) {
    uint4 v;
    asm("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}
// `addr` for reads that come after everything before this point, and are not
// shared with reads from before it.
__device__ __forceinline__ uint32_t after(uint32_t addr) {
    asm volatile("" : "+r"(addr)::"memory");
    return addr;
}

// Sums of N values over a group of `warps` consecutive warps (group `gid` of
// the block), the same bits in every thread: a shuffle tree inside each warp,
// then the same tree over the warps' sums (a chain over up to 16 warps took
// longer than all the rest of a row).  The group alone meets at its named
// barrier.  There are two buffers, used in turn: a buffer is written again only
// after the barrier of the sum between.
template <int N>
struct GroupSum {
    static constexpr uint32_t kBuffer = kMaxWarps * N * 4;
    static constexpr int kWords = 2 * kMaxWarps * N;
    uint32_t put, get;
    int tree, barrier, threads;
    bool takes;

    __device__ __forceinline__ GroupSum(uint32_t buffers, int warps, int gid) {
        tree = warps > 8 ? 16 : warps > 4 ? 8 : warps > 2 ? 4 : warps > 1 ? 2 : 1;
        const int q = threadIdx.x & (tree - 1);
        barrier = gid + 1;
        threads = warps * 32;
        takes = q < warps;
        put = buffers + (threadIdx.x >> 5) * (N * 4);
        get = buffers + (gid * warps + q) * (N * 4);
    }
    static __device__ __forceinline__ void round(float (&v)[N], int o) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    }
    __device__ __forceinline__ void operator()(float (&v)[N], int buffer) const {
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) round(v, o);
        if (tree == 1) return;
        const uint32_t shift = buffer * kBuffer;
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) st_shared(put + shift + 4 * i, v[i]);
        asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(threads) : "memory");
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = takes ? ld_shared(get + shift + 4 * i) : 0.0f;
        if (tree > 8) round(v, 8);
        if (tree > 4) round(v, 4);
        if (tree > 2) round(v, 2);
        round(v, 1);
    }
};

// ---------------------------------------------------------------- rows
//
// A warp owns 256 NV consecutive columns of its row; lane l's vector v is the
// eight values from column 256 v + 8 l of them (shifted by the row's start in
// its first word), so every offset below is a constant.  One stage of the ring
// holds a row per group: per warp and tensor, NV vectors of 32 lanes, read by the
// warp that copied them.

constexpr int kLaneStep = 256;  // columns between a lane's vectors

// Where a thread stands: its row group, its first vector's first column (from
// -7: the first word may start in the row before), and its group's rows row0,
// row0 + step, ... below `rows`.  Rows are counted without a sign: a group looks up
// to three steps (of 16 rows per block) past the last of up to 2^31 - 1 rows.
// kAligned: d is a multiple of 8, every row starts a word.
template <bool kAligned>
struct Place {
    int gid, col, left, row0, step;  // left: columns from the first vector to the row's end
    __device__ __forceinline__ Place(int d, int warps, int nv) {
        const int warp = threadIdx.x >> 5;
        const int groups = (blockDim.x >> 5) / warps;
        gid = warp / warps;
        row0 = blockIdx.x * groups + gid;
        step = gridDim.x * groups;
        const int start = kAligned ? 0 : static_cast<int>((static_cast<int64_t>(row0) * d) & 7);
        col = (warp - gid * warps) * (kLaneStep * nv) + 8 * (threadIdx.x & 31) - start;
        left = d - col;
    }
    // The rows from this one on may share their last word with the tensor's end.
    static __device__ __forceinline__ uint32_t near_end(uint32_t rows, int d) { return rows - min(rows, 1u + 7u / d); }
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
        if constexpr (!kAligned) {
            if (whole(v)) return;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                f[e] = f2(has(v, 2 * e) ? f[e].x() : 0.0f, has(v, 2 * e + 1) ? f[e].y() : 0.0f);
        }
    }
    // The row's values of vector v to p[0..7].
    template <typename T>
    __device__ __forceinline__ void store(int v, T* p, const f2 (&f)[4], bool wide) const {
        if constexpr (kAligned) {
            store8(p, f, wide);
        } else if (whole(v)) {
            store8(p, f, wide);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (has(v, 2 * e)) store1(p + 2 * e, f[e].x());
                if (has(v, 2 * e + 1)) store1(p + 2 * e + 1, f[e].y());
            }
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

// A warp's part of a ring stage for one tensor.  fp32: a lane's eight values are
// two words; copied and read by that lane they would be accesses of 16 bytes, 32
// apart (half of each sector, and two lanes on a bank).  So lane l copies words l
// and 32 + l of a vector's 64, word w goes to place w ^ (w / 8 & 1), and the lane
// that holds words 2l and 2l + 1 reads them without conflicts, after a warp barrier.
// (16384 x 4096 forward 66 us, with each lane's own words 95; backward with dres
// 146 and 214, there with dx in stores of 32 bytes, too.)
template <typename T, int NV>
struct RingPart {
    static constexpr int kW = kWords8<T>;
    static constexpr bool kShared = kW > 1;         // a lane reads what others of its warp copied
    static constexpr int kWords = NV * kW * 32;     // 16-byte words per warp and stage
    static constexpr uint32_t kBytes = 16 * kWords;

    // Bytes from a stage's start to the lane's first word, to copy and to read.
    static __device__ __forceinline__ uint32_t copy_at() {
        const uint32_t lane = threadIdx.x & 31;
        return 16 * (kShared ? lane ^ (lane >> 3 & 1) : lane);
    }
    static __device__ __forceinline__ uint32_t read_at() {
        const uint32_t lane = threadIdx.x & 31;
        return kShared ? 32 * lane + 16 * (lane >> 2 & 1) : 16 * lane;
    }
    // Values that the word a lane copies first lies before the first that it holds.
    static __device__ __forceinline__ int before() { return kShared ? 4 * (threadIdx.x & 31) : 0; }

    // `slot`: shared address of the first word that this lane copies; `row`: where it lies in
    // the row.  The tensor's last word is read up to the tensor's end only.
    template <bool kAligned>
    static __device__ __forceinline__ void copy(uint32_t slot, const T* row, const Place<kAligned>& p, bool last) {
        const int left = p.left + before();
#pragma unroll
        for (int v = 0; v < NV; ++v) {
#pragma unroll
            for (int q = 0; q < kW; ++q) {
                const int off = kLaneStep * v + 128 * q;
                if (off >= left) continue;
                const uint32_t dst = slot + (v * kW + q) * 512;
                const int bytes = (left - off) * static_cast<int>(sizeof(T));
                if (kAligned || !last || bytes >= 16)
                    cp_async16_at(dst, row + off);
                else
                    cp_async16_part(dst, row + off, bytes);
            }
        }
    }
    // `slot`: shared address of the first word that this lane reads.
    static __device__ __forceinline__ void read(uint32_t slot, int v, f2 (&f)[4]) {
        uint4 w[kW];
#pragma unroll
        for (int q = 0; q < kW; ++q) w[q] = ld_shared16((q == 0 ? slot : slot ^ 16) + v * kW * 512);
        unpack(w, f);
    }
};

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
// columns' sums of 4 vectors do not fit the registers (307 us, with 2 262).  (When
// the choice was made; now 146 us forward, 249 backward.)
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
                           (forward ? (nv == 4 ? 1.0 : nv == 2 ? 0.9 : 0.75) : (nv == 4 ? 0.6 : nv == 2 ? 1.0 : 0.8));
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

// Leave for `fn`'s launches to use up to kSmSmem of shared memory, once per device.
// The attribute is the function's, not the launch's: set to each call's own need, a
// call in another thread could lower it between this call's leave and its launch.
template <auto fn>
cudaError_t allow_smem() {
    static std::atomic<int> configured[64];
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev >= 64 || !configured[dev].load(std::memory_order_acquire)) {
        err = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmSmem));
        if (err != cudaSuccess) return err;
        if (dev < 64) configured[dev].store(1, std::memory_order_release);
    }
    return cudaSuccess;
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
cudaError_t launch_bwd(NormArgs& a, const RowShape& r, const Ring& q) {
    const size_t smem = std::max(q.bytes, 2 * sizeof(float) * static_cast<size_t>(a.d) * r.rows);
    a.blocks = grid_blocks(r, a.rows, a.d, std::min(q.blocks * device_sm_count(), kMaxBwdBlocks));
    constexpr auto fn = layernorm_bwd_kernel<T, NV, kAligned, STAGES>;
    const cudaError_t err = allow_smem<fn>();
    if (err != cudaSuccess) return err;
    fn<<<a.blocks, r.threads(), smem, a.s>>>(static_cast<const bf16*>(a.dy), static_cast<const T*>(a.x), a.gamma,
                                             a.mean, a.rstd, static_cast<const T*>(a.dres), a.rows, a.d, r.warps,
                                             static_cast<T*>(a.dx), a.part);
    return cudaGetLastError();
}

template <typename T, bool kAligned>
cudaError_t run_bwd(NormArgs& a) {
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
cudaError_t run(NormArgs& a, int x_type, bool forward) {
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
    if (run(a, x_type, false) != cudaSuccess) return MK_ERR_CUDA;
    const LaunchCfg lc(dim3(static_cast<unsigned>((2 * static_cast<int64_t>(d) + 31) / 32)), dim3(256), 0, s, true);
    if (cudaLaunchKernelEx(&lc.cfg, layernorm_bwd_sum_kernel, static_cast<const float*>(a.part), a.blocks, d, dgamma,
                           dbeta) != cudaSuccess)
        return MK_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}
