// gemm_wgrad.cu -- weight gradient of the grouped expert GEMM, on CTA pairs.
//
//   dW_e[i, j] (+)= sum over rows r of expert e of  dout[r, i] * x[r, j]
//
// for every expert, dout [S, n] and x [S, d] bf16 with expert e's rows
// [off[e], off[e + 1]), fp32 accumulation, dW [E, n, d] fp32 (stored, or added
// to what is there) or bf16 (stored).  The sum runs over an expert's rows, so
// its length is ragged: none, one, or tens of thousands.
//
//   tile        256 rows of dW_e (dout columns, the M side) x 256 columns (x
//               columns, the N side; the last tile of a row takes the 64 to
//               192 that are left).  CTA r of the pair holds 128 dout columns
//               and half of the x columns of a k-block of 64 rows, and its 128
//               rows of the accumulator in its own TMEM.
//   operands    both run along the sum's rows in memory, so both are read
//               MN-major: a TMA box of 64 columns x 64 rows lands as 64 rows
//               of 128 bytes (128-byte swizzle), 8 KB, two boxes per operand
//               half; no transposed copy of either tensor is made.
//   ragged end  an expert's last k-block holds rows of the next expert too.
//               Only its own rows are loaded, in boxes of 32, 16, 8, 4, 2 and 1
//               rows, and the last MMA step of 16 rows is filled up with boxes
//               past the tensor's end, which read as zeros: both operands are
//               zero there, so that a NaN of the next expert is not multiplied
//               by zero.  (The 128-byte swizzle follows the shared-memory
//               address, so boxes of any height make up one tile.  Clearing the
//               foreign rows with a warp after the copy cost 5 to 25 % at 8
//               k-blocks per tile.)
//   long sums   the tensor core's fp32 accumulator truncates, so its error grows
//               with the number of MMA steps: over 38000 rows it was 2.5e-5 of
//               the result's norm (1.4e-6 with rounded fp32 sums).  So a tile is
//               summed kWChunkRows rows at a time: each chunk has a TMEM
//               accumulator of its own, and eight epilogue warps keep the tile's
//               sums in registers (128 each) and add the chunks in row order,
//               rounded to nearest, while the next chunk is multiplied.
//   few tiles   where the tiles do not fill the GPU, an expert's rows are cut
//               into pieces; each piece's tiles are a sum of their own, stored
//               to the workspace, and a second kernel adds an expert's pieces
//               in row order.  (131072 rows of one 64 x 64 expert: 535 us as one
//               tile.)
//   order       a scheduler warp claims tiles from one ticket, experts with
//               the most rows first, so that the last tiles are the shortest.
//   store       the epilogue warps pass 32 x 128 bytes at a time through
//               swizzled shared memory to TMA stores (adding: TMA reductions
//               in L2, each element once per call, so the result does not
//               depend on timing; such additions may take subnormal values as
//               zero, though a GB300 was seen to keep them).  An expert without
//               rows gets zeros.
//
// Bound by the tensor cores where experts have many rows, by storing dW where they
// have few.  Measured, 20 calls in a row after a rest, of the measured burst bf16
// rate (R) or copy rate (C): 131072 skewed rows over 64 experts of 1536 x 4096 fp32
// 980 us (0.86 R), adding 1127 (0.75 R: the additions read the gradient too, 1.6 GB;
// for 3 s without a rest, at the power cap's clock, 1131 and 1208); 16384 rows over
// 32 of 1408 x 2048 fp32 105 to 111 us (0.68 to 0.65 C; what holds it was not
// measured), adding 141 (0.90 C), bf16 88 to 94 (0.55 to 0.51 R; nor here); 8191
// rows over 256 of them, bf16 303 us (0.76 C; the MMA warp and the epilogue wait on
// each other for accumulators, not for stores), fp32 adding 880 (1.01 C).
//
// Every wait is bounded, as in the other pair kernels.
#include <algorithm>
#include <atomic>

#include "gemm_impl.cuh"

namespace mk {
namespace {

using namespace gemm_detail;

// Stages of the operand ring and store buffers per epilogue warp, which share
// the 224 KB beside the control block: tiles with long sums take a sixth stage,
// short ones (bound by their stores) a second buffer.
constexpr int kLongStages = 6, kLongBufs = 1;
constexpr int kShortStages = 5, kShortBufs = 2;
constexpr int kMaxStages = 6;
constexpr uint32_t WBOX_BYTES = 64 * BK * 2;             // 64 columns of 64 rows
constexpr uint32_t WHALF_BYTES = 2 * WBOX_BYTES;         // 128 columns
constexpr uint32_t WSTAGE_BYTES = 2 * WHALF_BYTES;       // this CTA's dout and x columns
constexpr int kWEpiWarps = 8;                            // two per TMEM quarter, half of the columns each
constexpr uint32_t WSTORE_BYTES = 32 * 128;              // one store of an epilogue warp
// The other one of an epilogue warp's two store buffers, wherever the pair lies (dynamic
// shared memory is aligned to 1024 bytes here, not to the pair's size); `both` is the sum
// of their addresses.
__host__ __device__ constexpr uint32_t both_bufs(uint32_t first) { return 2 * first + WSTORE_BYTES; }
__host__ __device__ constexpr uint32_t other_buf(uint32_t buf, uint32_t both) { return both - buf; }
constexpr bool swaps_at(uint32_t first) {
    return other_buf(first, both_bufs(first)) == first + WSTORE_BYTES &&
           other_buf(first + WSTORE_BYTES, both_bufs(first)) == first;
}
static_assert(swaps_at(0) && swaps_at(1024) && swaps_at(WSTORE_BYTES) && swaps_at(WSTORE_BYTES + 1024),
              "the store buffers swap at any base");
constexpr int kWSchedWarp = 2;
constexpr int kWEpiWarp0 = 4;  // registers move between warpgroups; warp 3 only fills up the first
constexpr int WNUM_THREADS = 32 * (kWEpiWarp0 + kWEpiWarps);
constexpr int kWSlots = 8;  // most tiles claimed ahead
// Readers of a tile slot: CTA 0 its producer, MMA and epilogue warps plus CTA
// 1's slot relay; CTA 1 its producer, accumulator relay and epilogue warps.
constexpr uint32_t kWSlotReaders0 = 3 + kWEpiWarps;
constexpr uint32_t kWSlotReaders1 = 2 + kWEpiWarps;
// Rows summed in one accumulator (a multiple of 64).  Measured on 131072 rows
// over 64 experts of 1536 x 4096, the largest with 38360 (error of the fp32
// gradient against 64 bits, time): 256 rows 2.7e-7, 1298 us; 512 4.7e-7, 1080;
// 1024 9.2e-7, 1039; 2048 1.8e-6, 1035; all rows in one 2.5e-5.  (Times as of the
// choice; now 768 rows: 6.3e-7, 980 us.)
constexpr int kWChunkRows = 768;
// A tile's four (bf16: two) stores per epilogue warp are spread over the next
// tile's main loop, this many SM cycles per k-block of the last chunk apart:
// bursts of stores hold up the operand loads.  Measured (32 experts of about
// 512 rows, 1408 x 2048 fp32): 0: 116 us, 100: 115, 200: 107, 300: 130; 64
// experts of 2048 x 7168 bf16 with 1024 rows: 1262, 1232, 1217, 1199 us.
constexpr int kStorePace = 200;
constexpr int kClusters = 76;  // what the splitting and pacing rules assume resident
constexpr int kWGroupM = 8;  // M tiles walked together: tiles claimed together share operand columns in L2

struct WgradCtl {
    uint64_t full[kMaxStages];   // CTA 0: both CTAs' copies of the stage landed
    uint64_t empty[kMaxStages];  // each CTA: the MMAs that read the stage are done
    uint64_t tmem_full[2];
    uint64_t tmem_empty[2];  // each CTA: its epilogue warps have read the accumulator (CTA 0: and CTA 1's)
    // the accumulator
    uint64_t drain;
    uint64_t slot_full[kWSlots];
    uint64_t slot_empty[kWSlots];
    int4 slot[kWSlots];  // {expert or piece (< 0 ends the list), first row, rows, kLastChunk | m tile << 15 | n tile}
    uint32_t tmem_base;
    uint32_t abort_flag;
    uint32_t zero;
    int32_t offsets[kMaxExperts + 1];
    uint16_t index[kMaxExperts + 1];  // experts by falling row count; split sums: prefix over experts of their pieces
};

static_assert(WNUM_THREADS > kMaxExperts, "the prologue has a thread per offset");
constexpr size_t wgrad_smem(int stages, int bufs) {
    return static_cast<size_t>(stages) * WSTAGE_BYTES + static_cast<size_t>(kWEpiWarps * bufs) * WSTORE_BYTES +
           sizeof(WgradCtl) + 1024;
}
static_assert(wgrad_smem(kLongStages, kLongBufs) <= 227u * 1024u && wgrad_smem(kShortStages, kShortBufs) <= 227u * 1024u,
              "weight-gradient shared memory exceeds the per-CTA limit");

// One operand [S, columns] in boxes of 64 columns x 64, 32, 16, 8, 4, 2 and 1 rows.
constexpr int kBoxes = 7;
struct OperandMaps {
    CUtensorMap m[kBoxes];
};

struct WgradParams {
    const int32_t* offsets;  // [E + 1]
    int64_t S;
    int E, n, d;
    int m_tiles, n_tiles;
    int accumulate;
    int pace;         // cycles per k-block between the stores of a tile
    int split_rows;   // 0, or the most rows of a piece (a multiple of 64)
    int slots, batch;  // tiles claimed ahead (<= kWSlots), and at a time
    uint32_t* status;
    uint32_t* ticket;
    uint64_t timeout_ns;
};

__device__ __forceinline__ uint32_t wgrad_idesc(int N) {
    return idesc_bf16_f32(PAIR_M, static_cast<uint32_t>(N)) | kIdescAMnMajor | kIdescBMnMajor;
}

__device__ __forceinline__ void fence_proxy_async_shared() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, int32_t c0, int32_t c1, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1), "r"(src)
                 : "memory");
}

__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap* map, int32_t c0, int32_t c1) {  // into L2
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1)
                 : "memory");
}

__device__ __forceinline__ void tma_reduce_add_2d(const CUtensorMap* map, int32_t c0, int32_t c1, uint32_t src) {
    asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1), "r"(src)
                 : "memory");
}

__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}

__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void bulk_wait_read() {  // at most N stores have still to read their shared memory
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

__device__ __forceinline__ void raise_abort(WgradCtl* ctl, uint32_t peer) {
    ctl->abort_flag = 1u;
    st_shared_cluster_u32(mapa_shared(smem_u32(&ctl->abort_flag), peer), 1u);
}

// A slot reader's position in the ring.
struct SlotCursor {
    uint32_t slot = 0, phase = 0;
    __device__ __forceinline__ void next(int slots) {
        if (static_cast<int>(++slot) == slots) {
            slot = 0;
            phase ^= 1u;
        }
    }
};

// The next tile of the list, for a whole warp: false if the wait ran out.
__device__ __forceinline__ bool take_slot(WgradCtl* ctl, SlotCursor& cur, int4& info, const volatile uint32_t* abort_word,
                                          const WgradParams& p) {
    if (!__all_sync(0xffffffffu, mbar_wait_bounded_cluster(smem_u32(&ctl->slot_full[cur.slot]), cur.phase, abort_word,
                                                           p.timeout_ns)))
        return false;
    info = ctl->slot[cur.slot];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&ctl->slot_empty[cur.slot]));
    cur.next(p.slots);
    return true;
}

template <int kStages>
struct StageCursor {
    uint32_t stage = 0, phase = 0;
    __device__ __forceinline__ void next() {
        if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
        }
    }
};

__host__ __device__ __forceinline__ int pieces_of(int rows, int split_rows) {
    return (max(rows, 0) + split_rows - 1) / split_rows;
}

// A chunk's place in its expert's gradient, as packed in a tile slot.
constexpr int kLastChunk = 1 << 30;
__device__ __forceinline__ int slot_m(int w) { return (w >> 15) & 0x7fff; }
__device__ __forceinline__ int slot_n(int w) { return w & 0x7fff; }

__device__ __forceinline__ int k_blocks_of(int rows) { return (rows + BK - 1) / BK; }
__device__ __forceinline__ int tile_cols(int n_tile, const WgradParams& p) {
    return min(MMA_N, p.d - n_tile * MMA_N);  // a multiple of 64
}

constexpr int kHalfCols = MMA_N / 2;

template <bool kBf16Out, int kStages, int kBufs>
__global__ void __launch_bounds__(WNUM_THREADS, 1)
    grouped_wgrad_kernel(const __grid_constant__ OperandMaps tmA, const __grid_constant__ OperandMaps tmB,
                         const __grid_constant__ CUtensorMap tmOut, const WgradParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* store_smem = smem + kStages * WSTAGE_BYTES;
    WgradCtl* ctl = reinterpret_cast<WgradCtl*>(store_smem + kWEpiWarps * kBufs * WSTORE_BYTES);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const uint32_t peer = rank ^ 1u;

    // The experts' offsets, checked, and the experts by falling row count
    // (a thread per expert).
    const int my_e = threadIdx.x;
    if (my_e <= p.E) ctl->offsets[my_e] = p.offsets[my_e];
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_u32(&ctl->full[s]), 1);
            mbar_init(smem_u32(&ctl->empty[s]), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(smem_u32(&ctl->tmem_full[a]), 1);
            mbar_init(smem_u32(&ctl->tmem_empty[a]), rank == 0 ? kWEpiWarps + 1 : kWEpiWarps);
        }
        for (int i = 0; i < kWSlots; ++i) {
            mbar_init(smem_u32(&ctl->slot_full[i]), 1);
            mbar_init(smem_u32(&ctl->slot_empty[i]), rank == 0 ? kWSlotReaders0 : kWSlotReaders1);
        }
        mbar_init(smem_u32(&ctl->drain), 1);
        ctl->abort_flag = 0;
        ctl->zero = 0;
        fence_mbar_init();
        for (int i = 0; i < kBoxes; ++i) {
            prefetch_tensormap(&tmA.m[i]);
            prefetch_tensormap(&tmB.m[i]);
        }
        prefetch_tensormap(&tmOut);
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(&ctl->tmem_base), TMEM_COLS);
        tmem_relinquish_pair();
    }
    __syncthreads();
    bool bad = false;
    if (my_e < p.E) {
        const int cnt = ctl->offsets[my_e + 1] - ctl->offsets[my_e];
        bad = cnt < 0 || ctl->offsets[my_e] < 0;
        int rank_e = 0;
        for (int q = 0; q < p.E; ++q) {
            const int c = ctl->offsets[q + 1] - ctl->offsets[q];
            rank_e += (c > cnt || (c == cnt && q < my_e)) ? 1 : 0;
        }
        if (p.split_rows == 0) ctl->index[rank_e] = static_cast<uint16_t>(my_e);
    }
    if (p.split_rows != 0 && my_e <= p.E) {
        int before = 0;
        for (int q = 0; q < my_e; ++q) before += pieces_of(ctl->offsets[q + 1] - ctl->offsets[q], p.split_rows);
        ctl->index[my_e] = static_cast<uint16_t>(min(before, 0xffff));  // few: fewer tiles than clusters are split
    }
    if (my_e == 0) bad = bad || ctl->offsets[0] != 0 || ctl->offsets[p.E] != p.S;
    pdl_wait();  // the control words come from the kernel before
    const bool rejected = __syncthreads_or(bad ? 1 : 0) != 0;
    if (rejected && blockIdx.x == 0 && threadIdx.x == 0) report_error(p.status, MK_ERR_BOUNDS, kSiteWgradOffsets);
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // both CTAs' barriers exist before any copy, commit or arrive targets them
    tc_fence_after();
    const uint32_t tmem_base = ctl->tmem_base;
    volatile uint32_t* abort_word = &ctl->abort_flag;
    const volatile uint32_t* never = &ctl->zero;
    const int tiles_per_expert = p.m_tiles * p.n_tiles;
    const int total_tiles = rejected ? 0 : (p.split_rows != 0 ? ctl->index[p.E] : p.E) * tiles_per_expert;

    // The epilogue warps take the registers (their sums) that the other four give up: 40 + 2 x 232 of the
    // 3 x 168 per warp that the block is launched with.
    if (warp < kWEpiWarp0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp == 0) {
            // ---------------------------------------------------- TMA producer (both CTAs)
            const bool leader = elect_one();
            const uint32_t full0 = mapa_shared(smem_u32(&ctl->full[0]), 0);
            StageCursor<kStages> st;
            SlotCursor cur;
            uint32_t issued = 0, last_par = 0;
            bool ok = true;
            for (;;) {
                int4 info;
                if (!(ok = take_slot(ctl, cur, info, abort_word, p))) break;
                if (info.x < 0) break;
                const int kb_n = k_blocks_of(info.z);
                const int a_col = slot_m(info.w) * PAIR_M + static_cast<int>(rank) * BM;
                const int cols = tile_cols(slot_n(info.w), p);
                const int b_col = slot_n(info.w) * MMA_N + static_cast<int>(rank) * (cols >> 1);
                const int b_boxes = cols > 2 * 64 ? 2 : 1;
                for (int kb = 0; kb < kb_n; ++kb) {
                    if (!__all_sync(0xffffffffu, mbar_wait_bounded_cluster(smem_u32(&ctl->empty[st.stage]),
                                                                          st.phase ^ 1u, abort_word, p.timeout_ns))) {
                        ok = false;
                        break;
                    }
                    if (leader) {
                        const uint32_t sa = smem_u32(smem + st.stage * WSTAGE_BYTES);
                        const uint32_t fb = full0 + st.stage * 8u;
                        const int row = info.y + kb * BK;
                        const int left = min(BK, info.z - kb * BK);
                        const int filled = (left + UMMA_K - 1) / UMMA_K * UMMA_K;
                        if (rank == 0)
                            mbar_arrive_expect_tx(smem_u32(&ctl->full[st.stage]),
                                                  2u * static_cast<uint32_t>((2 + b_boxes) * filled * 128));
                        // `h` rows from row r of both tensors to row `at` of the stage
                        auto load = [&](int box, int at, int r) {
                            const uint32_t a = sa + static_cast<uint32_t>(at) * 128u, b = a + WHALF_BYTES;
                            tma_load_2d_pair(a, &tmA.m[box], a_col, r, fb);
                            tma_load_2d_pair(a + WBOX_BYTES, &tmA.m[box], a_col + 64, r, fb);
                            tma_load_2d_pair(b, &tmB.m[box], b_col, r, fb);
                            if (b_boxes == 2) tma_load_2d_pair(b + WBOX_BYTES, &tmB.m[box], b_col + 64, r, fb);
                        };
                        if (left == BK) {
                            load(0, 0, row);
                        } else {
                            int at = 0;
#pragma unroll 1
                            for (int box = 1; box < kBoxes; ++box)
                                if (left & (BK >> box)) {
                                    load(box, at, row + at);
                                    at += BK >> box;
                                }
                            const int fill = filled - left;
#pragma unroll 1
                            for (int box = kBoxes - 1; box > 2; --box)
                                if (fill & (BK >> box)) {
                                    load(box, at, static_cast<int>(p.S));  // past the last row: zeros
                                    at += BK >> box;
                                }
                        }
                    }
                    __syncwarp();
                    if (rank == 0) {
                        issued |= 1u << st.stage;
                        last_par = (last_par & ~(1u << st.stage)) | (st.phase << st.stage);
                    }
                    st.next();
                }
                if (!ok) break;
            }
            if (leader) {
                if (!ok) {
                    raise_abort(ctl, peer);
                    report_error(p.status, MK_ERR_TIMEOUT, kSiteGemmProducer);
                }
                // CTA 0: every stage it armed completes (or times out) before the CTA exits
                for (int s = 0; s < kStages; ++s)
                    if ((issued >> s) & 1u)
                        mbar_wait_bounded_cluster(smem_u32(&ctl->full[s]), (last_par >> s) & 1u, never, p.timeout_ns);
            }
            __syncwarp();
        } else if (warp == 1) {
            if (rank == 0) {
                // ------------------------------------------------ MMA issuer (CTA 0 only)
                const bool leader = elect_one();
                StageCursor<kStages> st;
                SlotCursor cur;
                uint32_t acc = 0, acc_phase = 0;
                bool ok = true;
                for (;;) {
                    int4 info;
                    if (!(ok = take_slot(ctl, cur, info, abort_word, p))) break;
                    if (info.x < 0) break;
                    if (info.z == 0) continue;
                    const uint32_t idesc = wgrad_idesc(tile_cols(slot_n(info.w), p));
                    if (!__all_sync(0xffffffffu, mbar_wait_bounded_cluster(smem_u32(&ctl->tmem_empty[acc]),
                                                                          acc_phase ^ 1u, abort_word, p.timeout_ns))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t d_tmem = tmem_base + acc * MMA_N;
                    const int kb_n = k_blocks_of(info.z);
                    for (int kb = 0; kb < kb_n; ++kb) {
                        if (!__all_sync(0xffffffffu, mbar_wait_bounded_cluster(smem_u32(&ctl->full[st.stage]), st.phase,
                                                                              abort_word, p.timeout_ns))) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        if (leader) {
                            const uint32_t sa = smem_u32(smem + st.stage * WSTAGE_BYTES);
                            const uint32_t sb = sa + WHALF_BYTES;
                            const int steps = (min(BK, info.z - kb * BK) + UMMA_K - 1) / UMMA_K;
    #pragma unroll
                            for (int kk = 0; kk < BK / UMMA_K; ++kk)
                                if (kk < steps)
                                    mma_bf16_ss_pair(d_tmem, sw128_mnmajor_desc(sa + kk * UMMA_K * 128, WBOX_BYTES),
                                                     sw128_mnmajor_desc(sb + kk * UMMA_K * 128, WBOX_BYTES), idesc,
                                                     (kb | kk) != 0 ? 1u : 0u);
                            mma_commit_pair_mc(smem_u32(&ctl->empty[st.stage]), 0x3);
                        }
                        __syncwarp();
                        st.next();
                    }
                    if (!ok) break;
                    if (leader) mma_commit_pair_mc(smem_u32(&ctl->tmem_full[acc]), 0x3);
                    __syncwarp();
                    acc ^= 1u;
                    if (acc == 0) acc_phase ^= 1u;
                }
                if (leader) {
                    if (!ok) {
                        raise_abort(ctl, peer);
                        report_error(p.status, MK_ERR_TIMEOUT, kSiteGemmMma);
                    }
                    // All MMAs issued complete before either CTA frees TMEM or shared memory.
                    mma_commit_pair_mc(smem_u32(&ctl->drain), 0x1);
                    if (!mbar_wait_bounded_cluster(smem_u32(&ctl->drain), 0u, never, p.timeout_ns))
                        report_error(p.status, MK_ERR_TIMEOUT, kSiteGemmDrain);
                }
            } else {
                // ------------------------------------------------ accumulator-release relay (CTA 1)
                // Once this CTA's epilogue warps have read an accumulator, one arrive (release at
                // cluster scope, cumulative over theirs) frees it on CTA 0.  The epilogue warps do
                // not arrive there themselves: a cluster-scope release waits for the stores its
                // warp has in flight (measured 2100 to 7400 cycles of each tile).
                const uint32_t tmem_empty0 = mapa_shared(smem_u32(&ctl->tmem_empty[0]), 0);
                SlotCursor cur;
                uint32_t acc = 0, acc_phase = 0;
                bool ok = true;
                for (;;) {
                    int4 info;
                    if (!(ok = take_slot(ctl, cur, info, abort_word, p))) break;
                    if (info.x < 0) break;
                    if (info.z == 0) continue;
                    if (!__all_sync(0xffffffffu, mbar_wait_bounded_cluster(smem_u32(&ctl->tmem_empty[acc]), acc_phase,
                                                                          abort_word, p.timeout_ns))) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) mbar_arrive_cluster(tmem_empty0 + acc * 8u);
                    acc ^= 1u;
                    if (acc == 0) acc_phase ^= 1u;
                }
                if (!ok && lane == 0) {
                    raise_abort(ctl, peer);
                    report_error(p.status, MK_ERR_TIMEOUT, kSiteGemmEpilogue);
                }
            }
            __syncwarp();
        } else if (warp == kWSchedWarp) {
            const bool leader = elect_one();
            const int lead = __ffs(__ballot_sync(0xffffffffu, leader)) - 1;
            SlotCursor cur;
            bool ok = true;
            if (rank == 0) {
                // ------------------------------------------------ tile scheduler (CTA 0)
                const uint32_t peer_slot0 = mapa_shared(smem_u32(&ctl->slot[0]), peer);
                const uint32_t peer_slot_full0 = mapa_shared(smem_u32(&ctl->slot_full[0]), peer);
                int4 nfo = make_int4(0, 0, 0, 0);
                int row_end = 0;  // of the tile's expert
                uint32_t tk = 0;
                int batch_left = 0;
                for (;;) {
                    if (!__all_sync(0xffffffffu, mbar_wait_bounded_cluster(smem_u32(&ctl->slot_empty[cur.slot]),
                                                                          cur.phase ^ 1u, abort_word, p.timeout_ns))) {
                        ok = false;
                        break;
                    }
                    if (nfo.y + nfo.z < row_end) {  // the tile's next chunk, in this cluster too
                        nfo.y += nfo.z;
                        nfo.z = min(kWChunkRows, row_end - nfo.y);
                    } else {
                        if (batch_left == 0) {
                            if (leader) tk = atomicAdd(p.ticket, static_cast<uint32_t>(p.batch));
                            tk = __shfl_sync(0xffffffffu, tk, lead);
                            batch_left = p.batch;
                        } else {
                            ++tk;
                        }
                        --batch_left;
                        nfo = make_int4(-1, 0, 0, 0);
                        row_end = 0;
                        if (tk < static_cast<uint32_t>(total_tiles)) {
                            const int piece = tk / tiles_per_expert;
                            const int l = tk % tiles_per_expert;
                            const int q = l / (kWGroupM * p.n_tiles);  // group of M tiles, walked M first
                            const int gm = min(kWGroupM, p.m_tiles - q * kWGroupM);
                            const int r = l - q * kWGroupM * p.n_tiles;
                            int out = 0, row = 0;
                            if (p.split_rows != 0) {
                                int lo = 0, hi = p.E - 1;  // largest e with index[e] <= piece
                                while (lo < hi) {
                                    const int mid = (lo + hi + 1) >> 1;
                                    if (ctl->index[mid] <= piece)
                                        lo = mid;
                                    else
                                        hi = mid - 1;
                                }
                                out = piece;
                                row = ctl->offsets[lo] + (piece - ctl->index[lo]) * p.split_rows;
                                row_end = min(row + p.split_rows, ctl->offsets[lo + 1]);
                            } else {
                                out = ctl->index[piece];
                                row = ctl->offsets[out];
                                row_end = ctl->offsets[out + 1];
                            }
                            nfo = make_int4(out, row, min(kWChunkRows, row_end - row),
                                            ((q * kWGroupM + r % gm) << 15) | (r / gm));
                        }
                    }
                    if (nfo.y + nfo.z >= row_end) nfo.w |= kLastChunk;
                    if (leader) {
                        ctl->slot[cur.slot] = nfo;
                        st_shared_cluster_v4(peer_slot0 + cur.slot * static_cast<uint32_t>(sizeof(int4)), nfo);
                        mbar_arrive(smem_u32(&ctl->slot_full[cur.slot]));
                        mbar_arrive_cluster(peer_slot_full0 + cur.slot * 8u);
                    }
                    __syncwarp();
                    cur.next(p.slots);
                    if (nfo.x < 0) break;
                }
            } else {
                // ------------------------------------------------ slot-release relay (CTA 1)
                const uint32_t slot_empty0 = mapa_shared(smem_u32(&ctl->slot_empty[0]), 0);
                for (;;) {
                    if (!__all_sync(0xffffffffu, mbar_wait_bounded_cluster(smem_u32(&ctl->slot_empty[cur.slot]), cur.phase,
                                                                          abort_word, p.timeout_ns))) {
                        ok = false;
                        break;
                    }
                    const int e = ctl->slot[cur.slot].x;
                    __syncwarp();
                    if (leader) mbar_arrive_cluster(slot_empty0 + cur.slot * 8u);
                    cur.next(p.slots);
                    if (e < 0) break;
                }
            }
            if (!ok && leader) {
                raise_abort(ctl, peer);
                report_error(p.status, MK_ERR_TIMEOUT, kSiteGemmProducer);
            }
            __syncwarp();
        }
    } else {
        // ---------------------------------------------------- epilogue (both CTAs, warps 4-11)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
        const int sub = warp & 3;            // TMEM lanes [32 sub, 32 sub + 32) are this warp's
        const int half = (warp - kWEpiWarp0) >> 2;  // and columns [128 half, 128 half + 128)
        uint32_t buf = smem_u32(store_smem + (warp - kWEpiWarp0) * (kBufs * WSTORE_BYTES));
        const uint32_t bufs = both_bufs(buf);
        SlotCursor cur;
        const uint32_t buf_row = lane * 128 + (lane & 7) * 16;
        uint32_t acc = 0, acc_phase = 0;
        bool ok = true;
        float sum[kHalfCols];  // zero between tiles
#pragma unroll
        for (int i = 0; i < kHalfCols; ++i) sum[i] = 0.0f;
        for (;;) {
            int4 info;
            if (!(ok = take_slot(ctl, cur, info, abort_word, p))) break;
            if (info.x < 0) break;
            const bool rows = info.z != 0;
            const int m_row = slot_m(info.w) * PAIR_M + static_cast<int>(rank) * BM + sub * 32;
            const int cols = tile_cols(slot_n(info.w), p) - half * kHalfCols;  // <= 0: none for this warp
            const int col0 = slot_n(info.w) * MMA_N + half * kHalfCols;
            const int out_row = info.x * p.n + m_row;
            const bool in = m_row < p.n;  // n is a multiple of 64: all 32 rows or none
            constexpr int kCols = kBf16Out ? 64 : 32;  // columns per 128-byte row of a store
            const bool last = (info.w & kLastChunk) != 0;
            const bool store = in && (rows || !p.accumulate);
            if (!kBf16Out && p.accumulate && last && store && lane == 0)
                for (int c = 0; c < kHalfCols && c < cols; c += kCols) tma_prefetch_2d(&tmOut, col0 + c, out_row);
            if (rows) {
                if (!__all_sync(0xffffffffu, mbar_wait_bounded_cluster(smem_u32(&ctl->tmem_full[acc]), acc_phase,
                                                                      abort_word, p.timeout_ns))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                // the chunk joins the tile's sums, then its accumulator is free
                const uint32_t tbase =
                    tmem_base + (static_cast<uint32_t>(sub * 32) << 16) + acc * MMA_N + half * kHalfCols;
#pragma unroll
                for (int c = 0; c < kHalfCols; c += 32) {
                    uint32_t v[32];
                    tmem_ld_32x32b_x32(tbase + c, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 32; ++i) sum[c + i] += __uint_as_float(v[i]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&ctl->tmem_empty[acc]));
                acc ^= 1u;
                if (acc == 0) acc_phase ^= 1u;
            }
            if (!last) continue;
            const int pace = k_blocks_of(info.z) * p.pace * (kCols / 32);
            const long long t0 = clock64();
#pragma unroll
            for (int c = 0; c < kHalfCols; c += kCols) {
                if (store && c < cols) {
                    if (c != 0)
                        while (clock64() - t0 < static_cast<long long>(c / kCols) * pace) __nanosleep(64);
                    if (lane == 0) bulk_wait_read<kBufs - 1>();  // the last store from this buffer has read it
                    __syncwarp();
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        uint4 o;
                        if (kBf16Out)
                            o = make_uint4(pack_bf16x2(sum[c + 8 * q], sum[c + 8 * q + 1]),
                                           pack_bf16x2(sum[c + 8 * q + 2], sum[c + 8 * q + 3]),
                                           pack_bf16x2(sum[c + 8 * q + 4], sum[c + 8 * q + 5]),
                                           pack_bf16x2(sum[c + 8 * q + 6], sum[c + 8 * q + 7]));
                        else
                            o = make_uint4(__float_as_uint(sum[c + 4 * q]), __float_as_uint(sum[c + 4 * q + 1]),
                                           __float_as_uint(sum[c + 4 * q + 2]), __float_as_uint(sum[c + 4 * q + 3]));
                        st_shared_v4(buf + (buf_row ^ (q * 16)), o);
                    }
                    fence_proxy_async_shared();
                    __syncwarp();
                    if (lane == 0) {
                        if (!kBf16Out && p.accumulate)
                            tma_reduce_add_2d(&tmOut, col0 + c, out_row, buf);
                        else
                            tma_store_2d(&tmOut, col0 + c, out_row, buf);
                        bulk_commit();
                    }
                    if (kBufs == 2) buf = other_buf(buf, bufs);
                }
#pragma unroll
                for (int i = 0; i < kCols; ++i) sum[c + i] = 0.0f;
            }
        }
        if (lane == 0) {
            bulk_wait_all();
            if (!ok) {
                raise_abort(ctl, peer);
                report_error(p.status, MK_ERR_TIMEOUT, kSiteGemmEpilogue);
            }
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // neither CTA leaves while the other may still use its shared memory
    if (*abort_word != 0u && threadIdx.x == 0) {
        // After a timeout, copies the peer started may still complete on this CTA's
        // barriers: keep both CTAs resident a little longer (bounded) before exit.
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 200000ull) {
        }
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, TMEM_COLS);
    }
}

// ------------------------------------------------------------------ host side

// 2-D row-major tensor [rows, inner], box {box_cols, box_rows} of 128-byte rows, 128-byte swizzle.
bool make_map_box(CUtensorMap* m, const void* base, bool fp32, uint64_t inner, uint64_t rows, uint32_t box_rows) {
    auto fn = encode_fn();
    if (fn == nullptr) return false;
    const uint32_t size = fp32 ? 4 : 2;
    const cuuint64_t dims[2] = {inner, rows};
    const cuuint64_t strides[1] = {inner * size};
    const cuuint32_t box[2] = {128u / size, box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return fn(m, fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
              const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Adds an expert's pieces, part [pieces, n, d] fp32, in row order into dw (+=
// with `accumulate`): a block per 1024 values of one expert.
template <bool kBf16Out>
__global__ void __launch_bounds__(256) wgrad_join_kernel(const float* __restrict__ part,
                                                         const int32_t* __restrict__ offsets, int split_rows,
                                                         int64_t size, void* dw, int accumulate,
                                                         const uint32_t* __restrict__ status) {
    __shared__ int first;
    if (*status != 0u) return;  // rejected offsets, or a wait that ran out: dw stays as it is
    const int e = blockIdx.y;
    if (threadIdx.x == 0) first = 0;
    __syncthreads();
    int before = 0;
    for (int q = threadIdx.x; q < e; q += 256) before += pieces_of(offsets[q + 1] - offsets[q], split_rows);
    if (before != 0) atomicAdd(&first, before);
    __syncthreads();
    const int n = pieces_of(offsets[e + 1] - offsets[e], split_rows);
    const int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
    if (i >= size) return;
    const float* src = part + static_cast<int64_t>(first) * size + i;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int q = 0; q < n; ++q) {
        const float4 t = __ldcs(reinterpret_cast<const float4*>(src + q * size));
        v.x += t.x, v.y += t.y, v.z += t.z, v.w += t.w;
    }
    if (kBf16Out) {
        *reinterpret_cast<uint2*>(static_cast<bf16*>(dw) + e * size + i) =
            make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
    } else {
        float4* out = reinterpret_cast<float4*>(static_cast<float*>(dw) + e * size + i);
        if (accumulate) {
            const float4 t = *out;
            v.x += t.x, v.y += t.y, v.z += t.z, v.w += t.w;
        }
        *out = v;
    }
}

// Rows of a piece, or 0 where the experts are summed whole.  Pieces make about
// two tiles per cluster and have at least 512 rows.  They pay where the tiles
// are too few: whole sums take the k-blocks of an expert (half as many again
// for uneven ones) per wave of tiles, at 512 cycles (0.27 us) each; pieces share
// the k-blocks out, but are stored and read back (about 8 TB/s through L2) and
// cost a second kernel.  Measured, fp32: 30000 rows of 4 experts of 256 x 256:
// whole 43 us, in pieces 23; 131072 rows of one 64 x 64: 535 and 35; 20000 rows
// of 8 experts of 1024 x 512 (64 tiles): 34 and 44.
int split_rows_of(int64_t S, int d, int E, int n) {
    const int64_t per_expert = static_cast<int64_t>((n + PAIR_M - 1) / PAIR_M) * ((d + MMA_N - 1) / MMA_N);
    if (per_expert * E >= 2 * kClusters) return 0;
    const int64_t rows = std::max<int64_t>(512, (S * per_expert / (2 * kClusters) + BK - 1) / BK * BK);
    if (rows >= S) return 0;
    const double block_us = 0.27;
    const double waves = static_cast<double>((per_expert * E + kClusters - 1) / kClusters);
    const double whole = 1.5 * waves * S / E / BK * block_us;
    const double shared = static_cast<double>(S) * per_expert / BK / kClusters * block_us;
    const double join = 2.0 * (S / rows + E) * n * d * sizeof(float) / 8e6 + 5.0;
    return shared + join < whole ? static_cast<int>(rows) : 0;
}

template <bool kBf16Out, int kStages, int kBufs>
cudaError_t launch_wgrad(const OperandMaps& a, const OperandMaps& b, const CUtensorMap& out, const WgradParams& p,
                         cudaStream_t s) {
    static std::atomic<int> max_clusters[64];  // per device, 0 until configured
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    auto fn = grouped_wgrad_kernel<kBf16Out, kStages, kBufs>;
    constexpr size_t smem = wgrad_smem(kStages, kBufs);
    LaunchCfg lc(dim3(2 * std::max(1, device_sm_count() / 2)), dim3(WNUM_THREADS), smem, s, true, 2);
    int n = dev < 64 ? max_clusters[dev].load(std::memory_order_acquire) : 0;
    if (n == 0) {
        err = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (err != cudaSuccess) return err;
        err = cudaOccupancyMaxActiveClusters(&n, fn, &lc.cfg);
        if (err != cudaSuccess) return err;
        if (n < 1) return cudaErrorInvalidConfiguration;
        if (dev < 64) max_clusters[dev].store(n, std::memory_order_release);
    }
    // with pieces: an upper bound (every expert adds at most one partial piece)
    const int64_t tiles = (p.split_rows != 0 ? p.S / p.split_rows + p.E : p.E) * static_cast<int64_t>(p.m_tiles) * p.n_tiles;
    lc.cfg.gridDim = dim3(2 * static_cast<unsigned>(std::min<int64_t>(n, tiles)));
    err = cudaLaunchKernelEx(&lc.cfg, fn, a, b, out, p);
    if (err != cudaSuccess) return err;
    return cudaGetLastError();
}

}  // namespace
}  // namespace mk

using namespace mk;

extern "C" size_t mk_moe_grouped_wgrad_workspace_size(int64_t S, int d, int E, int n) {
    if (check_sizes(S, d, E, 1, n) != MK_OK) return 0;
    const int rows = split_rows_of(S, d, E, n);
    return 256 + (rows == 0 ? 0 : static_cast<size_t>(S / rows + E) * n * d * sizeof(float));
}

extern "C" mk_status mk_moe_grouped_wgrad(const void* dout, const int32_t* expert_offsets, const void* x_perm,
                                          int64_t S, int d, int E, int n, void* dw, int dw_type, int accumulate,
                                          void* ws, size_t ws_bytes, void* stream) {
    const mk_status st = check_sizes(S, d, E, 1, n);
    if (st != MK_OK) return st;
    const int64_t m_tiles = (n + PAIR_M - 1) / PAIR_M, n_tiles = (d + MMA_N - 1) / MMA_N;
    if (m_tiles > 0x7fff || n_tiles > 0x7fff || m_tiles * n_tiles * E >= (int64_t(1) << 31)) return MK_ERR_UNSUPPORTED;
    if (dw_type != MK_TYPE_BF16 && dw_type != MK_TYPE_FP32) return MK_ERR_INVALID_ARG;
    if (accumulate && dw_type != MK_TYPE_FP32) return MK_ERR_INVALID_ARG;
    if (!dw || !aligned16(dw)) return MK_ERR_INVALID_ARG;
    if (S > 0 && (!dout || !expert_offsets || !x_perm || !aligned16(dout) || !aligned16(x_perm)))
        return MK_ERR_INVALID_ARG;
    if (ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0 || ws_bytes < 256) return MK_ERR_WORKSPACE;
    if (!device_is_sm103()) return MK_ERR_UNSUPPORTED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint32_t* status = static_cast<uint32_t*>(ws);
    if (launch_clear_control(status, s) != cudaSuccess) return MK_ERR_CUDA;
    const bool fp32 = dw_type == MK_TYPE_FP32;
    if (S == 0) {  // no rows: every expert's gradient is zero
        if (!accumulate &&
            cudaMemsetAsync(dw, 0, static_cast<size_t>(E) * n * d * (fp32 ? 4 : 2), s) != cudaSuccess)
            return MK_ERR_CUDA;
        return MK_OK;
    }
    OperandMaps a, b;
    // Pieces need room for their sums; a caller with the least workspace gets whole experts.
    const int split =
        ws_bytes >= mk_moe_grouped_wgrad_workspace_size(S, d, E, n) ? split_rows_of(S, d, E, n) : 0;
    float* part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + 256);
    const bool sums = fp32 || split != 0;  // the tiles' type
    CUtensorMap out;
    for (int i = 0; i < kBoxes; ++i)
        if (!make_map_box(&a.m[i], dout, false, n, S, BK >> i) || !make_map_box(&b.m[i], x_perm, false, d, S, BK >> i))
            return MK_ERR_CUDA;
    if (!make_map_box(&out, split != 0 ? part : dw, sums, d,
                      static_cast<uint64_t>(split != 0 ? S / split + E : E) * n, 32))
        return MK_ERR_CUDA;
    WgradParams p;
    p.offsets = expert_offsets;
    p.S = S;
    p.E = E;
    p.n = n;
    p.d = d;
    p.m_tiles = static_cast<int>(m_tiles);
    p.n_tiles = static_cast<int>(n_tiles);
    p.accumulate = accumulate && split == 0 ? 1 : 0;
    p.split_rows = split;
    // A ticket takes about 1 us, a tile of an expert with few rows little more: then tiles are
    // claimed four at a time and eight ahead.  Otherwise three ahead, so that a cluster holds few
    // at the end.  Measured, 256 experts of 1408 x 2048 bf16 with 32 rows: 332 us, one at a time
    // 385; 32 experts of 512 rows: eight ahead 125 us, three 108.
    const bool short_tiles = S <= 128 * static_cast<int64_t>(E);
    const int64_t tiles = m_tiles * n_tiles * E;
    p.slots = short_tiles ? kWSlots : 3;
    p.batch = short_tiles && tiles >= 64 * kClusters ? 4 : 1;
    p.pace = tiles >= 8 * kClusters ? kStorePace : 0;
    p.status = status;
    p.ticket = status + 4;
    p.timeout_ns = kDefaultTimeoutNs;
    auto run = sums ? (short_tiles ? launch_wgrad<false, kShortStages, kShortBufs>
                                   : launch_wgrad<false, kLongStages, kLongBufs>)
                    : (short_tiles ? launch_wgrad<true, kShortStages, kShortBufs>
                                   : launch_wgrad<true, kLongStages, kLongBufs>);
    cudaError_t err = run(a, b, out, p, s);
    if (err == cudaSuccess && split != 0) {
        const int64_t size = static_cast<int64_t>(n) * d;
        const dim3 grid(static_cast<unsigned>((size + 1023) / 1024), static_cast<unsigned>(E));
        if (fp32)
            wgrad_join_kernel<false><<<grid, 256, 0, s>>>(part, expert_offsets, split, size, dw, accumulate, status);
        else
            wgrad_join_kernel<true><<<grid, 256, 0, s>>>(part, expert_offsets, split, size, dw, 0, status);
        err = cudaGetLastError();
    }
    return err == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}
