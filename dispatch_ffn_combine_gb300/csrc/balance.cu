// balance.cu -- the router's balance and z losses with the experts' counts, and the
// gradient of the gate logits.
//
// Over sequences s of n_s tokens (N in all, B' of them not empty), with p[t] the
// softmax of token t's logits over all E experts, c[s, e] how often e was chosen in s:
//
//   P[s, e] = sum_{t in s} p[t, e] / n_s,   F[s, e] = E c[s, e] / (k n_s)
//   balance = sum_s sum_e F[s, e] P[s, e] / B',   z = sum_t lse(l[t])^2 / N
//
//   dl[t, e] = bc p[t, e] (G[e] - sum_i G[i] p[t, i])   with G = F[s] / (B' n_s)
//            + zc 2 lse(l[t]) p[t, e] / N
//            + w[t, j] (dw[t, j] - sum_i w[t, i] dw[t, i])   where e is t's j-th expert
//
// c is constant to the gradient, as usual; the last line is the softmax over the
// chosen logits that gives the routing weights.  A token whose logits are all -inf has
// p = 0 and no part in z.
//
// Both are one pass over the logits: the gradient needs c (known from the forward
// pass) but not P.  A token's logits are held by eight lanes, 4 to 32 each, so a warp
// takes four tokens at a time: three shuffles per reduction serve four tokens, and a
// warp has four rows of loads in flight.  Sums over tokens: a lane keeps its experts' p
// in registers over its block's tokens of a sequence, the block adds its warps and
// writes one partial row per sequence it meets (the pairs (block, sequence) met form a
// staircase, so block + sequence numbers them), and a second kernel adds the partial
// rows in block order.  Counts are integers.  The number of blocks depends on the
// sizes alone: results repeat bit for bit.
//
// 32768 tokens of 256 experts in 23 sequences: the losses 18.6 us (two launches; 34 MB,
// 5 us at the copy rate), the gradient 16.2 us (72 MB, 11 us).  Few warps are resident, with
// 32 logits and 32 sums or factors per lane, and each waits for its rows' loads: with 32
// lanes per token, in earlier forms, 26 and 40 us, with a branch around each load 34 and 39.
#include <algorithm>

#include "mk_device.cuh"
#include "mk_internal.h"

namespace mk {
namespace {

constexpr int kLanes = 8;        // of a token
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kPass = kThreads / kLanes;  // tokens a block takes at a time
constexpr int kManyBlocks = 608;  // partial rows, and blocks of the backward kernel: four per SM
// Tokens whose p a lane adds up in one fp32 sum: a chain of n additions is off by up to n 2^-24, so beyond 20 million
// tokens there are more blocks rather than longer chains (65536 of them at most, whose partial rows the sums' kernel
// adds in slices of 2048 at most).
constexpr int kMaxChain = 2048;
constexpr int kMaxSlices = 32;   // of a sequence's partial rows, a warp each
constexpr int kMaxSeqs = 65535;

int tokens_per_block(int64_t T) {
    return static_cast<int>(std::min<int64_t>(kPass * kMaxChain, std::max<int64_t>(kPass, (T + kManyBlocks - 1) / kManyBlocks)));
}

struct Seqs {
    const int32_t* offsets;  // [B + 1] or null: one sequence of all T tokens
    int B;
    int64_t T;
    // Whether sequence i's bounds are out of order or outside the tokens, or the first one does not start at 0.
    __device__ __forceinline__ bool bad(int i) const {
        if (offsets == nullptr) return false;
        const int32_t a = __ldg(offsets + i), b = __ldg(offsets + i + 1);
        return a < 0 || b < a || b > T || (i == 0 && a != 0);
    }
    // Clamped to the tokens, so that no offset leads outside the tensors.
    __device__ __forceinline__ int64_t at(int s) const {
        if (offsets == nullptr) return s == 0 ? 0 : T;
        return max(static_cast<int64_t>(0), min(static_cast<int64_t>(__ldg(offsets + s)), T));
    }
};

// The first sequence that ends behind token t (B: none), how many are not empty, and whether any has bad bounds.  All
// threads of the block.
struct Place {
    int seq, filled;
    bool bad;
};
__device__ __forceinline__ Place find_place(const Seqs& seqs, int64_t t, uint32_t (&s_part)[kWarps]) {
    static_assert(kMaxSeqs < 1 << 16, "two counts in a word");
    uint32_t n = 0;
    bool bad = false;
    for (int i = threadIdx.x; i < seqs.B; i += kThreads) {
        const int64_t end = seqs.at(i + 1);
        n += (end <= t ? 0x10000u : 0u) + (end > seqs.at(i) ? 1u : 0u);
        bad |= seqs.bad(i);
    }
    n = __reduce_add_sync(0xffffffffu, n);
    if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = n;
    bad = __syncthreads_or(bad ? 1 : 0) != 0;
    n = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) n += s_part[i];
    return {static_cast<int>(n >> 16), static_cast<int>(n & 0xffffu), bad};
}

// A lane's VALS of a token's E logits.  kVec: E is a multiple of four, loaded 16 bytes at a time.
template <int VALS, bool kVec>
struct Row {
    static __device__ __forceinline__ int expert(int lane, int i) {
        return kVec ? 4 * (lane + kLanes * (i / 4)) + i % 4 : lane + kLanes * i;
    }
    template <typename V>
    static __device__ __forceinline__ void load(const V* row, int lane, int E, V pad, V (&v)[VALS]) {
        // Lanes behind the last expert load the first ones again: loads without branches, all in flight together.
        if constexpr (kVec) {
            uint4 w[VALS / 4];
#pragma unroll
            for (int q = 0; q < VALS / 4; ++q) {
                const int e = 4 * (lane + kLanes * q);
                w[q] = __ldg(reinterpret_cast<const uint4*>(row + (e < E ? e : 0)));
            }
#pragma unroll
            for (int q = 0; q < VALS / 4; ++q) {
                const uint32_t u[4] = {w[q].x, w[q].y, w[q].z, w[q].w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[4 * q + i] = 4 * (lane + kLanes * q) < E ? reinterpret_cast<const V&>(u[i]) : pad;
            }
        } else {
#pragma unroll
            for (int i = 0; i < VALS; ++i) v[i] = __ldg(row + (expert(lane, i) < E ? expert(lane, i) : 0));
#pragma unroll
            for (int i = 0; i < VALS; ++i) v[i] = expert(lane, i) < E ? v[i] : pad;
        }
    }
    static __device__ __forceinline__ void store(float* row, int lane, int E, const float (&v)[VALS]) {
        if constexpr (kVec) {
#pragma unroll
            for (int q = 0; q < VALS / 4; ++q)
                if (4 * (lane + kLanes * q) < E)
                    reinterpret_cast<float4*>(row)[lane + kLanes * q] =
                        make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
        } else {
#pragma unroll
            for (int i = 0; i < VALS; ++i)
                if (expert(lane, i) < E) row[expert(lane, i)] = v[i];
        }
    }
};

__device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int o = kLanes / 2; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = kLanes / 2; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// e^x for x <= 0 as 2^(x log2 e), below 2^-126 zero: off by (1.25 |x| + 4) 2^-24 of itself, the
// product's rounding and log2 e's, and ex2's 2^-22.  x, the difference of two fp32 logits, is off by |x| 2^-24
// already, which expf does not mend; with it the losses take 20.4 us for 18.6, the gradient 17.7 for 16.2.
__device__ __forceinline__ float exp_down(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
    return y;
}

// Softmax of a token's logits, v becoming p = exp(v - base) inv, and their log-sum-exp; a
// token whose logits are all -inf has inv = p = lse = 0.  A NaN or +inf among them gives NaN.
struct Softmax {
    float base, inv, lse;
    template <int VALS>
    __device__ __forceinline__ explicit Softmax(float (&v)[VALS]) {
        constexpr float kNegInf = -__builtin_huge_valf();
        float m = v[0];
#pragma unroll
        for (int i = 1; i < VALS; ++i) m = fmaxf(m, v[i]);
        m = group_max(m);
        base = m == kNegInf ? 0.0f : m;  // NaN logits keep NaN: v - base is
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < VALS; ++i) {
            v[i] = exp_down(v[i] - base);
            s += v[i];
        }
        s = group_sum(s);
        inv = s != 0.0f ? 1.0f / s : 0.0f;
        lse = s != 0.0f ? base + logf(s) : 0.0f;
#pragma unroll
        for (int i = 0; i < VALS; ++i) v[i] *= inv;
    }
};

struct LossPart {
    float* p;         // [slots, E]
    int32_t* counts;  // [slots, E]
    float* z;         // [slots]
    int32_t* bad;     // [slots] an expert id was out of range
};

template <int VALS, bool kVec>
__global__ void __launch_bounds__(kThreads, 4) balance_part_kernel(const float* __restrict__ logits,
                                                                const int32_t* __restrict__ ids, const Seqs seqs, int E,
                                                                int k, int per_block, const LossPart out,
                                                                uint32_t* status) {
    __shared__ float s_p[kWarps][kMaxExperts];
    __shared__ float s_z[kWarps];
    __shared__ int32_t s_counts[kMaxExperts];
    __shared__ uint32_t s_part[kWarps];
    using R = Row<VALS, kVec>;
    const int warp = threadIdx.x >> 5, wl = threadIdx.x & 31, lane = wl % kLanes, group = threadIdx.x / kLanes;
    const int64_t t1 = min(seqs.T, static_cast<int64_t>(blockIdx.x + 1) * per_block);
    int64_t t = static_cast<int64_t>(blockIdx.x) * per_block;
    pdl_launch_dependents();
    // For the sums' kernel, which reports what is bad and counts its blocks: with a launch of its own for these words
    // a call of 256 or 32768 tokens took 4 us longer on the host.
    if (blockIdx.x == 0 && threadIdx.x < kControlWords) status[threadIdx.x] = 0u;
    const Place place = find_place(seqs, t, s_part);
    for (int s = place.seq; s < seqs.B && t < t1; ++s) {
        const int64_t end = min(seqs.at(s + 1), t1);
        if (end <= t) continue;
        bool bad = false;
        for (int e = threadIdx.x; e < E; e += kThreads) s_counts[e] = 0;
        __syncthreads();
        for (int64_t i = t * k + threadIdx.x; i < end * k; i += kThreads) {
            const int e = __ldg(ids + i);
            if (e >= 0 && e < E)
                atomicAdd(s_counts + e, 1);
            else
                bad = true;
        }
        float sum[VALS], z = 0.0f;
#pragma unroll
        for (int i = 0; i < VALS; ++i) sum[i] = 0.0f;
#pragma unroll(VALS <= 8 ? 4 : 1)
        for (int64_t q = t; q < end; q += kPass) {  // the same passes for all lanes of the block
            const bool live = q + group < end;
            float v[VALS];
            R::load(logits + (live ? q + group : t) * E, lane, E, -__builtin_huge_valf(), v);
            const Softmax soft(v);
            if (live) {
#pragma unroll
                for (int i = 0; i < VALS; ++i) sum[i] += v[i];
                z = fmaf(soft.lse, soft.lse, z);
            }
        }
#pragma unroll
        for (int o = 16; o >= kLanes; o >>= 1) {
#pragma unroll
            for (int i = 0; i < VALS; ++i) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
            z += __shfl_xor_sync(0xffffffffu, z, o);
        }
        if (wl < kLanes) {
#pragma unroll
            for (int i = 0; i < VALS; ++i)
                if (R::expert(lane, i) < E) s_p[warp][R::expert(lane, i)] = sum[i];
        }
        if (wl == 0) s_z[warp] = z;
        const int any_bad = __syncthreads_or(bad ? 1 : 0);
        const int64_t slot = blockIdx.x + static_cast<int64_t>(s);
        for (int e = threadIdx.x; e < E; e += kThreads) {
            float a = s_p[0][e];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) a += s_p[w][e];
            out.p[slot * E + e] = a;
            out.counts[slot * E + e] = s_counts[e];
        }
        if (threadIdx.x == 0) {
            float a = s_z[0];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) a += s_z[w];
            out.z[slot] = a;
            out.bad[slot] = any_bad;
        }
        __syncthreads();
        t = end;
    }
}

// 32 experts of one sequence per block: its partial rows in block order (a slice per
// warp, each every so manieth row, then the slices), P, c, and the block's part of the
// losses; the last block adds those.
__global__ void __launch_bounds__(32 * kMaxSlices) balance_sum_kernel(const LossPart part, const Seqs seqs, int E, int k,
                                                               int per_block, float* __restrict__ loss,
                                                               int32_t* __restrict__ counts, float* __restrict__ probs,
                                                               float* __restrict__ terms, uint32_t* status) {
    __shared__ float s_p[kMaxSlices][32];
    __shared__ int32_t s_c[kMaxSlices][32];
    __shared__ float s_z[kMaxSlices];
    __shared__ int s_last, s_filled[kMaxSlices];
    __shared__ float s_sum[2][kMaxSlices];
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5, slices = blockDim.x >> 5, s = blockIdx.y;
    const int e = blockIdx.x * 32 + lane;
    const int64_t t0 = seqs.at(s), n = max(seqs.at(s + 1) - t0, static_cast<int64_t>(0));
    pdl_wait();
    if (threadIdx.x == 0 && blockIdx.x == 0 && seqs.bad(s)) report_error(status, MK_ERR_BOUNDS, kSiteBalanceOffsets);
    float p = 0.0f, z = 0.0f;
    int32_t c = 0;
    if (n > 0) {
        const int64_t b0 = t0 / per_block + s, b1 = (t0 + n - 1) / per_block + s;
        if (e < E)
#pragma unroll 8
            for (int64_t b = b0 + slice; b <= b1; b += slices) {
                p += part.p[b * E + e];
                c += part.counts[b * E + e];
            }
        if (blockIdx.x == 0)
            for (int64_t b = b0 + threadIdx.x; b <= b1; b += blockDim.x) {
                z += part.z[b];
                if (part.bad[b] != 0) report_error(status, MK_ERR_BOUNDS, kSiteBalanceIds);
            }
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    s_p[slice][lane] = p;
    s_c[slice][lane] = c;
    if (lane == 0) s_z[slice] = z;
    __syncthreads();
    if (slice == 0) {
        for (int i = 1; i < slices; ++i) {
            p += s_p[i][lane];
            c += s_c[i][lane];
        }
        const float inv_n = n > 0 ? 1.0f / static_cast<float>(n) : 0.0f;
        p *= inv_n;
        if (e < E) {
            counts[static_cast<int64_t>(s) * E + e] = c;
            probs[static_cast<int64_t>(s) * E + e] = p;
        }
        float term = static_cast<float>(E) * inv_n / static_cast<float>(k) * static_cast<float>(c) * p;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) term += __shfl_xor_sync(0xffffffffu, term, o);
        if (lane == 0) {
            const int64_t at = static_cast<int64_t>(s) * gridDim.x + blockIdx.x;
            terms[2 * at] = term;
            float a = s_z[0];
            for (int i = 1; i < slices; ++i) a += s_z[i];
            terms[2 * at + 1] = a;
            __threadfence();
            s_last = atomicAdd(status + 4, 1u) == gridDim.x * gridDim.y - 1 ? 1 : 0;
        }
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    // every thread a strided part of the terms, then a fixed tree
    float balance = 0.0f, zsum = 0.0f;
    int filled = 0;
    for (int64_t i = threadIdx.x; i < static_cast<int64_t>(gridDim.x) * gridDim.y; i += blockDim.x) {
        balance += __ldcg(terms + 2 * i);
        zsum += __ldcg(terms + 2 * i + 1);
    }
    for (int i = threadIdx.x; i < seqs.B; i += blockDim.x) filled += seqs.at(i + 1) > seqs.at(i) ? 1 : 0;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        balance += __shfl_xor_sync(0xffffffffu, balance, o);
        zsum += __shfl_xor_sync(0xffffffffu, zsum, o);
        filled += __shfl_xor_sync(0xffffffffu, filled, o);
    }
    if (lane == 0) s_sum[0][slice] = balance, s_sum[1][slice] = zsum, s_filled[slice] = filled;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < slices; ++i) balance += s_sum[0][i], zsum += s_sum[1][i], filled += s_filled[i];
        const bool bad = *static_cast<volatile uint32_t*>(status) != 0u;
        const float tokens = static_cast<float>(seqs.at(seqs.B));
        loss[0] = bad ? __uint_as_float(0x7fc00000u) : filled > 0 ? balance / static_cast<float>(filled) : 0.0f;
        loss[1] = bad ? __uint_as_float(0x7fc00000u) : tokens > 0.0f ? zsum / tokens : 0.0f;
    }
}

struct RouteBwd {
    const float* logits;
    const int32_t* ids;
    const float* w;          // null: no part of the weights
    const float* dw;         // [T, k], or [T k] rows with slot_row
    const int32_t* slot_row;
    const int32_t* counts;   // null: no balance part
    float balance_coef, z_coef;
    int E, k, per_block;
    float* dlogits;
    uint32_t* status;
};

// The chosen experts' part is a lane's per choice: it works its expert's whole value out
// again (the same operations on the same logit) and writes it over the row's.  Choosing
// each value's part from all the choices instead is 2 k instructions per value and lane.
template <int VALS, bool kVec>
__global__ void __launch_bounds__(kThreads, 4) route_bwd_kernel(const RouteBwd a, const Seqs seqs) {
    __shared__ uint32_t s_part[kWarps];
    using R = Row<VALS, kVec>;
    const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
    const int E = a.E, k = a.k;
    const int64_t t1 = min(seqs.T, static_cast<int64_t>(blockIdx.x + 1) * a.per_block);
    int64_t t = static_cast<int64_t>(blockIdx.x) * a.per_block;
    const Place place = find_place(seqs, t, s_part);
    const int64_t all = seqs.at(seqs.B);
    const float z_scale = all > 0 ? 2.0f * a.z_coef / static_cast<float>(all) : 0.0f;
    pdl_wait();  // the status was cleared by the kernel before
    if (place.bad && blockIdx.x == 0 && threadIdx.x == 0) report_error(a.status, MK_ERR_BOUNDS, kSiteBalanceOffsets);
    for (int s = place.bad ? seqs.B : place.seq; t < t1; ++s) {
        // else the tokens behind the last sequence, or all of them where the bounds are bad: the weights' part only
        const bool in_seq = s < seqs.B;
        const int64_t end = in_seq ? min(seqs.at(s + 1), t1) : t1;
        if (end <= t) continue;
        const float n = in_seq ? static_cast<float>(seqs.at(s + 1) - seqs.at(s)) : 1.0f;
        float per_count = 0.0f;
        float g[VALS];
        if (in_seq && a.counts != nullptr)
            per_count =
                a.balance_coef * static_cast<float>(E) / (static_cast<float>(k) * n * n * static_cast<float>(place.filled));
        const int32_t* counts = a.counts + static_cast<int64_t>(s) * E;  // read only where per_count is not 0
        {
            int32_t c[VALS];
            if (per_count != 0.0f) R::template load<int32_t>(counts, lane, E, 0, c);
#pragma unroll
            for (int i = 0; i < VALS; ++i) g[i] = per_count != 0.0f ? per_count * static_cast<float>(c[i]) : 0.0f;
        }
        const float z_seq = in_seq ? z_scale : 0.0f;
        const bool needs_p = per_count != 0.0f || z_seq != 0.0f;
#pragma unroll(VALS <= 8 ? 4 : 1)
        for (int64_t q = t; q < end; q += kPass) {  // the same passes for all lanes of the block
            const bool live = q + group < end;
            const int64_t tok = live ? q + group : t;
            float v[VALS];
            if (needs_p) {
                R::load(a.logits + tok * E, lane, E, -__builtin_huge_valf(), v);
            } else {
#pragma unroll
                for (int i = 0; i < VALS; ++i) v[i] = 0.0f;
            }
            // this lane's choice: its expert, weight, the weight's gradient, and the expert's logit and count
            int e = -1;
            float w = 0.0f, dw = 0.0f, l = 0.0f, g_e = 0.0f;
            if (a.w != nullptr && lane < k) {
                const int64_t i = tok * k + lane;
                e = __ldg(a.ids + i);
                const int64_t at = a.slot_row != nullptr ? static_cast<int64_t>(__ldg(a.slot_row + i)) : i;
                if (e >= 0 && e < E && at >= 0 && at < seqs.T * k) {
                    w = __ldg(a.w + i);
                    dw = __ldg(a.dw + at);
                    if (needs_p) l = __ldg(a.logits + tok * E + e);
                    if (per_count != 0.0f) g_e = per_count * static_cast<float>(__ldg(counts + e));
                } else {
                    e = -1;
                    if (live) report_error(a.status, MK_ERR_BOUNDS, kSiteRouteBwd);
                }
            }
            float p = 0.0f, shift = 0.0f;
            if (needs_p) {
                const Softmax soft(v);
                float dot = 0.0f;
#pragma unroll
                for (int i = 0; i < VALS; ++i) dot = fmaf(g[i], v[i], dot);
                shift = fmaf(z_seq, soft.lse, -group_sum(dot));
#pragma unroll
                for (int i = 0; i < VALS; ++i) v[i] *= g[i] + shift;
                p = exp_down(l - soft.base) * soft.inv;
            }
            float* row = a.dlogits + tok * E;
            if (live) R::store(row, lane, E, v);
            if (a.w != nullptr) {
                const float dl = w * (dw - group_sum(w * dw));
                float part = 0.0f;  // of all choices of the expert
                for (int j = 0; j < k; ++j) {
                    const int ej = __shfl_sync(0xffffffffu, e, j, kLanes);
                    const float dlj = __shfl_sync(0xffffffffu, dl, j, kLanes);
                    if (ej == e) part += dlj;
                }
                __syncwarp();  // the row's stores come first
                if (live && e >= 0) row[e] = fmaf(p, g_e + shift, part);
            }
        }
        t = end;
    }
}

// ------------------------------------------------------------------ host side

mk_status check_balance(int64_t T, int E, int k, int B, bool offsets) {
    if (T < 0 || E <= 0 || k <= 0 || B <= 0 || E > kMaxExperts || k > kMaxTopK || k > E || (!offsets && B != 1))
        return MK_ERR_INVALID_ARG;
    if (B > kMaxSeqs || T * k >= (int64_t(1) << 31)) return MK_ERR_UNSUPPORTED;
    return MK_OK;
}

int blocks_of(int64_t T, int per_block) { return static_cast<int>((T + per_block - 1) / per_block); }

// f(values per lane, vec) with both as compile-time constants.
template <typename F>
cudaError_t with_row(int E, F f) {
    const bool vec = E % 4 == 0;
#define MK_VALS(n) \
    if (E <= kLanes * n) return vec ? f(std::integral_constant<int, n>(), std::true_type()) : f(std::integral_constant<int, n>(), std::false_type())
    MK_VALS(4);
    MK_VALS(8);
    MK_VALS(16);
    MK_VALS(32);
#undef MK_VALS
    return cudaErrorInvalidValue;
}
static_assert(kMaxExperts <= 32 * kLanes && kMaxTopK <= kLanes, "a token's logits and choices fit its lanes");

}  // namespace
}  // namespace mk

using namespace mk;

extern "C" size_t mk_moe_balance_workspace_size(int64_t T, int E, int k, int B) {
    if (check_balance(T, E, k, B, true) != MK_OK) return 0;
    const size_t slots = static_cast<size_t>(blocks_of(T, tokens_per_block(T))) + B;
    return 256 + 4 * (slots * (2 * static_cast<size_t>(E) + 2) + 2 * static_cast<size_t>(B) * ((E + 31) / 32));
}

extern "C" mk_status mk_moe_balance_loss(const float* logits, const int32_t* topk_ids, const int32_t* seq_offsets,
                                         int64_t T, int E, int k, int B, float* loss, int32_t* counts, float* probs,
                                         void* ws, size_t ws_bytes, void* stream) {
    const mk_status st = check_balance(T, E, k, B, seq_offsets != nullptr);
    if (st != MK_OK) return st;
    if (!loss || !counts || !probs || (T > 0 && (!logits || !topk_ids))) return MK_ERR_INVALID_ARG;
    if (!aligned16(logits)) return MK_ERR_INVALID_ARG;
    if (ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0 ||
        ws_bytes < mk_moe_balance_workspace_size(T, E, k, B))
        return MK_ERR_WORKSPACE;
    if (!device_is_sm103()) return MK_ERR_UNSUPPORTED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint32_t* status = static_cast<uint32_t*>(ws);
    const int per_block = tokens_per_block(T);
    const int blocks = blocks_of(T, per_block);
    const size_t slots = static_cast<size_t>(blocks) + B;
    LossPart part;
    part.p = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + 256);
    part.counts = reinterpret_cast<int32_t*>(part.p + slots * E);
    part.z = reinterpret_cast<float*>(part.counts + slots * E);
    part.bad = reinterpret_cast<int32_t*>(part.z + slots);
    float* terms = part.z + 2 * slots;
    const Seqs seqs{seq_offsets, B, T};
    cudaError_t err;
    if (blocks == 0)
        err = launch_clear_control(status, s);
    else
        err = with_row(E, [&](auto vals, auto vec) {
            LaunchCfg lc(dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, s, false);
            return cudaLaunchKernelEx(&lc.cfg, balance_part_kernel<decltype(vals)::value, decltype(vec)::value>, logits,
                                      topk_ids, seqs, E, k, per_block, part, status);
        });
    if (err != cudaSuccess) return MK_ERR_CUDA;
    // With few long sequences a block's own walk is the time (32768 tokens of 256 experts in one: 29 us with 8 slices,
    // 19 with 32), with many the blocks (512 sequences of 256 tokens, 64 experts: 21 and 30).
    // So many blocks may be one sequence's that eight slices would be longer chains than a lane's.
    const unsigned slices = blocks > std::min(64 * B, 8 * kMaxChain) ? kMaxSlices : 8;
    LaunchCfg lc(dim3(static_cast<unsigned>((E + 31) / 32), static_cast<unsigned>(B)), dim3(32u * slices), 0, s, true);
    if (cudaLaunchKernelEx(&lc.cfg, balance_sum_kernel, part, seqs, E, k, per_block, loss, counts, probs, terms, status) !=
        cudaSuccess)
        return MK_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}

extern "C" mk_status mk_moe_route_bwd(const float* logits, const int32_t* topk_ids, const float* topk_w,
                                      const float* dweight, const int32_t* slot_row, const int32_t* counts,
                                      const int32_t* seq_offsets, int64_t T, int E, int k, int B, float balance_coef,
                                      float z_coef, float* dlogits, void* ws, size_t ws_bytes, void* stream) {
    const mk_status st = check_balance(T, E, k, B, seq_offsets != nullptr);
    if (st != MK_OK) return st;
    if ((topk_w == nullptr) != (dweight == nullptr) || (slot_row != nullptr && dweight == nullptr)) return MK_ERR_INVALID_ARG;
    if (balance_coef != 0.0f && counts == nullptr) return MK_ERR_INVALID_ARG;
    if (T == 0) return MK_OK;
    if (!dlogits || !aligned16(dlogits) || !aligned16(logits) || !aligned16(counts)) return MK_ERR_INVALID_ARG;
    if (topk_w != nullptr && !topk_ids) return MK_ERR_INVALID_ARG;
    if ((balance_coef != 0.0f || z_coef != 0.0f) && !logits) return MK_ERR_INVALID_ARG;
    if (ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0 || ws_bytes < 256) return MK_ERR_WORKSPACE;
    if (!device_is_sm103()) return MK_ERR_UNSUPPORTED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    RouteBwd a;
    a.logits = logits;
    a.ids = topk_ids;
    a.w = topk_w;
    a.dw = dweight;
    a.slot_row = slot_row;
    a.counts = balance_coef != 0.0f ? counts : nullptr;
    a.balance_coef = balance_coef;
    a.z_coef = z_coef;
    a.E = E;
    a.k = k;
    a.per_block = tokens_per_block(T);
    a.dlogits = dlogits;
    a.status = static_cast<uint32_t*>(ws);
    if (launch_clear_control(a.status, s) != cudaSuccess) return MK_ERR_CUDA;
    const Seqs seqs{seq_offsets, B, T};
    const cudaError_t err = with_row(E, [&](auto vals, auto vec) {
        LaunchCfg lc(dim3(static_cast<unsigned>(blocks_of(T, a.per_block))), dim3(kThreads), 0, s, true);
        return cudaLaunchKernelEx(&lc.cfg, route_bwd_kernel<decltype(vals)::value, decltype(vec)::value>, a, seqs);
    });
    if (err != cudaSuccess) return MK_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}
