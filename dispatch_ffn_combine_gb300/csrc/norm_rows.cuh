// norm_rows.cuh -- what the norms over rows of a tensor share: where a thread
// stands in its row, the ring of rows copied ahead, sums over a row's warps, and
// the choice of a block's shape.
#pragma once

#include <algorithm>
#include <atomic>
#include <numeric>

#include "f32x2.cuh"
#include "mk_device.cuh"
#include "mk_internal.h"

namespace mk {
namespace norm_rows {

constexpr int kMaxD = 16384;  // 16 warps of 4 vectors; 8 less where a row's first word may start before it
constexpr int kMaxWarps = 16;    // per block and per row
constexpr int kMaxBwdBlocks = 304;  // partial rows of a backward pass

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

// ---------------------------------------------------------------- partial rows

// The blocks' partial rows [blocks][n] added, 32 columns per block: 8 slices of
// every eighth partial row, then the slices in order.  Columns below `split` go
// to `first`, the others to `second`; with `add` onto what is there.
static __global__ void __launch_bounds__(256) sum_partial_rows_kernel(const float* __restrict__ part, int blocks, int n,
                                                                      int split, float* __restrict__ first,
                                                                      float* __restrict__ second, bool add) {
    __shared__ float s[8][32];
    pdl_wait();  // the partial rows come from the kernel before
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float v = 0.0f;
    if (c < n)
#pragma unroll 8
        for (int b = slice; b < blocks; b += 8) v += part[static_cast<int64_t>(b) * n + c];
    s[slice][lane] = v;
    __syncthreads();
    if (slice == 0 && c < n) {
#pragma unroll
        for (int i = 1; i < 8; ++i) v += s[i][lane];
        float* to = c < split ? first + c : second + (c - split);
        *to = add ? *to + v : v;
    }
}

// ------------------------------------------------------------------ host side

// Behind the kernel that writes the partial rows, as its programmatic dependent.
static inline cudaError_t sum_partial_rows(const float* part, int blocks, int n, int split, float* first, float* second,
                                           cudaStream_t s, bool add = false) {
    const LaunchCfg lc(dim3(static_cast<unsigned>((static_cast<int64_t>(n) + 31) / 32)), dim3(256), 0, s, true);
    const cudaError_t err = cudaLaunchKernelEx(&lc.cfg, sum_partial_rows_kernel, part, blocks, n, split, first, second, add);
    return err != cudaSuccess ? err : cudaGetLastError();
}

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
inline RowShape row_shape(int64_t rows, int d, bool forward) {
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
inline Ring ring_shape(RowShape& s, int words) {
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
inline int grid_blocks(const RowShape& s, int64_t rows, int d, int most) {
    const int64_t chunks = (rows + s.rows - 1) / s.rows;
    if (chunks <= most) return static_cast<int>(chunks);
    const int apart = 8 / std::gcd(d, 8), unit = apart / std::gcd(s.rows, apart);
    return std::max(unit, most / unit * unit);
}

// Rows that a row group of a backward pass adds up in one fp32 sum per column.  A chain of n additions is off by up to n
// 2^-24 of its terms' magnitudes, so more rows than that per group (0.6 million for long rows, 20 for short ones) go through the
// kernel in pieces, whose sums are added: 2^-12 for a piece and 2^-24 for each.  The rows of a piece are a multiple of 8, so that it
// starts on a 16-byte word as the tensor does.
constexpr int kMaxChain = 4096;
inline int64_t piece_rows(const RowShape& s, int blocks) { return static_cast<int64_t>(kMaxChain) * s.rows * blocks; }

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

}  // namespace norm_rows
}  // namespace mk
