// gemm8.cu -- the grouped expert GEMM on 8-bit operands with a scale per block
// of 128, on CTA pairs.
//
//   out[r, j] = wr[r] * sum over blocks b of 128 columns of
//                   xs[r, b] * ws[e, j / 128, b] * sum over i in b of x[r, i] * w[e, j, i]
//
// for the rows r of expert e: x [S, d] and w [E, n, d] e4m3 codes, xs a scale
// per row and block, ws a scale per 128 x 128 block, wr an optional row weight,
// out bf16 or fp32.
//
//   products    tcgen05.mma kind::f8f6f4 (M = 256 over both CTAs, N = up to 128,
//               K = 32): a block of 128 columns is four MMAs into an accumulator of
//               its own for each half of the tile's columns, since the scales change
//               with every block.
//   sums        the scales are fp32 numbers of any value, so the blocks' products
//               are joined outside the tensor core: eight epilogue warps keep
//               the tile's sums in registers (128 per thread) and add each
//               block's accumulators, times its scales, rounded to nearest, while
//               the next block is multiplied into the half's other accumulator.
//   tile        256 rows x 256 columns (the last tile of a row takes the 64 to 192
//               that are left); CTA r holds rows [128 r, 128 r + 128) and half of
//               the weight rows and receives its rows of the accumulator.  A thread
//               of the epilogue has one row and half of the columns, so one product
//               of two scales per block.  A block of rows that is not full takes the
//               time of a full one, but loads only its rows (in boxes of 16, 32,
//               64 or 128), and the warps without rows read nothing: with few rows
//               per expert the weights' stream is the bound.  (With the operands
//               exchanged for such blocks, as in the bf16 kernel, a thread needs
//               a scale per column; such tiles took longer than full ones.)
//   scales      come through shared memory by TMA, sixteen blocks to a slot, by a thread
//               of their own that runs ahead of the operands; a thread of the epilogue
//               reads and multiplies four blocks' at a time.  With the producer issuing
//               them in slots of four, and two reads per block, they came late and cost
//               100 cycles of a block's 1030 (131072 skewed rows of 4096 to 1536 columns:
//               731 us, in that form without any scales 619; from then on 700, with slots of sixteen
//               679).  Loads from global memory in the epilogue warps held up their other waits.
//   roles       the producer, the issuer and the scales' thread are single threads: per block of
//               columns their waits and issues are one after the other, and with
//               a whole warp voting on each wait they took longer than the MMAs.
//   hand-over   each half of the tile's columns has two accumulators and four warps per CTA
//               that read them, so a half is read while the other one is multiplied.
//               With both halves in one MMA of N = 256 a warp saw its block 750 cycles after
//               the issue, and two accumulators could not cover that and the reads: 667 us,
//               so 653.  An accumulator is freed by arrives without memory order (see free_acc).
//               What bounds the kernel with many rows is the epilogue warps' own
//               time per block, one step after the other: a wait takes 150 to 200 cycles
//               though the phase is long complete, so the next one is tested while the last
//               additions run (653 us, so 620; it was no gain with N = 256).  Reads and additions
//               take 350, what is around them 150, scales 30, with 512 of MMAs beside them (clocks
//               read in a copy of the form with N = 256).
//               Uniform waits, predicated arrives and additions in pairs: 700 us to 662.
//               Waits with acquire at cluster scope, since the peer's copies and commits complete
//               the barriers: 629 us to 637.
//               Sixteen epilogue warps of 64 columns, reads ahead of the additions, scales a block
//               ahead, and one lane waiting for its warp were slower.
//   store       32 rows of 128 bytes at a time through swizzled shared memory to
//               TMA stores; the rows at an expert's end, whose 32-row group the
//               next expert's rows share, in plain stores from there.
//   schedule    tile-slot and stage rings, relays and bounded waits as in the
//               weight-gradient kernel.
//
// Times above are of captured calls, four in a row after a rest, with codes of normal values.  Called for
// seconds, at the power cap, the skewed case takes 732 us.  65536 rows over 16 equal experts, 7168 to 4096:
// 2970 TFLOP/s after a rest, 2620 for seconds (codes drawn evenly from 0 to 119: 3070 and 2760).
#include <algorithm>
#include <atomic>

#include "pair_ring.cuh"

namespace mk {
namespace {

using namespace gemm_detail;

constexpr int kBlockK = 128;                             // columns per scale, and per stage
constexpr int kBlockN = 128;                             // weight rows per scale
constexpr uint32_t kHalfBytes = BM * kBlockK;            // 128 rows of 128 codes
constexpr uint32_t kStageBytes = 2 * kHalfBytes;         // this CTA's M and N rows
constexpr int kUmmaK8 = 32;                              // columns per MMA
constexpr int kEpiWarps = 8;                             // two per TMEM quarter
constexpr int kEpiWarp0 = 4;
constexpr int kSchedWarp = 2;
constexpr int kScaleWarp = 3;
constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);
constexpr int kSlots = 3;
constexpr int kStages = 5;
constexpr int kNGroup = 4;  // N tiles walked together over an expert's row blocks
// Readers of a tile slot: CTA 0 its producer, issuer and epilogue warps plus CTA
// 1's slot relay; CTA 1 its producer and epilogue warps.
constexpr uint32_t kSlotReaders0 = 4 + kEpiWarps;
constexpr uint32_t kSlotReaders1 = 2 + kEpiWarps;
constexpr uint32_t kAccCols = 128;               // TMEM columns of an accumulator
constexpr uint32_t kPartBytes = kHalfBytes / 2;  // 64 weight rows: this CTA's of a half of the tile's columns
constexpr int kPartWarps = kEpiWarps / 2;  // epilogue warps of each half of a tile's columns
// Scales reach the epilogue warps through shared memory in groups of four blocks of columns
// (16 bytes of a scale row): the CTA's 128 rows' and its two blocks of weight rows'.
constexpr int kScaleGroup = 4;
constexpr int kScaleSpan = 16;  // blocks per slot
constexpr int kScaleSlots = 2;
constexpr uint32_t kXScaleBytes = BM * 16;
constexpr uint32_t kWScaleBytes = 2 * 16;
constexpr uint32_t kScaleGroupBytes = kXScaleBytes + 128;  // TMA writes start on 128 bytes
constexpr uint32_t kScaleSlotBytes = kScaleSpan / kScaleGroup * kScaleGroupBytes;

struct Ctl8 {
    uint64_t full[kStages];   // CTA 0: both CTAs' copies of the stage landed
    uint64_t empty[kStages];  // each CTA: the MMAs that read the stage are done
    uint64_t tmem_full[4];    // each CTA: the accumulator (two for each half of the columns) is complete
    uint64_t tmem_empty[4];   // CTA 0: both CTAs' epilogue warps of the half have read it
    uint64_t scale_full[kScaleSlots];   // each CTA: a group's scales landed
    uint64_t scale_empty[kScaleSlots];  // each CTA: its epilogue warps have read them
    uint64_t drain;
    uint64_t slot_full[kSlots];
    uint64_t slot_empty[kSlots];
    int4 slot[kSlots];  // {e, row0, rows, n0}; e < 0 ends the list
    uint32_t tmem_base;
    uint32_t abort_flag;
    uint32_t zero;
    int32_t pstart[kMaxExperts + 1];  // prefix over experts of their 256-row blocks
};

constexpr size_t kSmem8 = kStages * kStageBytes + kEpiWarps * kStoreBytes + kScaleSlots * kScaleSlotBytes + sizeof(Ctl8) + 1024;
static_assert(kSmem8 <= 227u * 1024u, "8-bit GEMM shared memory exceeds the per-CTA limit");

struct Params8 {
    const int32_t* offsets;      // [E+1]
    const int32_t* mtile_start;  // [E+1] prefix of ceil(rows / 128); all zero when offsets were rejected
    const float* row_weight;     // [S] or null
    void* out;                   // [S, n]
    int E, n, n_tiles, n_blocks, k_blocks;
    int slots;
    uint32_t* status;
    uint32_t* ticket;
    uint64_t timeout_ns;
};

// Instruction descriptor, kind::f8f6f4: D fp32, A and B e4m3 (format 0), both K-major, M x N.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(uint32_t M, uint32_t N) {
    return (1u << 4) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

__device__ __forceinline__ void mma_e4m3_ss_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                                 uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Rows of the box that covers `rows` (> 0) of a CTA's rows.
__device__ __forceinline__ int box_rows(int rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128; }

// Tile t -> {expert, first row, rows, first column}: an expert's tiles in groups
// of kNGroup N tiles, each group over all the expert's row blocks, N fastest.
__device__ __forceinline__ int4 decode_tile(int tile, const Ctl8* ctl, const Params8& p) {
    const int g = tile / p.n_tiles;
    int lo = 0, hi = p.E - 1;  // largest e with pstart[e] <= g
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (ctl->pstart[mid] <= g)
            lo = mid;
        else
            hi = mid - 1;
    }
    const int blocks = ctl->pstart[lo + 1] - ctl->pstart[lo];
    const int l = tile - ctl->pstart[lo] * p.n_tiles;
    const int q = l / (blocks * kNGroup);
    const int nb = min(kNGroup, p.n_tiles - q * kNGroup);
    const int r = l - q * blocks * kNGroup;
    const int j = r / nb;
    const int nt = q * kNGroup + (r - j * nb);
    const int off = __ldg(p.offsets + lo);
    const int cnt = __ldg(p.offsets + lo + 1) - off;
    return make_int4(lo, off + j * PAIR_M, min(PAIR_M, cnt - j * PAIR_M), nt * MMA_N);
}

__device__ __forceinline__ float4 lds4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
    return v;
}
// A cursor over the two accumulators of a half of the columns.  Every waiter sees every phase of a barrier: one
// that left some out could take an old phase for the one it waits for.
struct AccCursor {
    uint32_t acc, phase = 0;
    __device__ __forceinline__ explicit AccCursor(int part) : acc(2u * part) {}
    __device__ __forceinline__ void next() {
        acc ^= 1u;
        if ((acc & 1u) == 0u) phase ^= 1u;
    }
};

// take_slot for a single thread.
__device__ __forceinline__ bool take_slot_one(Ctl8* ctl, SlotCursor& cur, int4& info, const volatile uint32_t* abort_word,
                                              const Params8& p) {
    if (!mbar_wait_bounded_cluster(smem_u32(&ctl->slot_full[cur.slot]), cur.phase, abort_word, p.timeout_ns)) return false;
    info = ctl->slot[cur.slot];
    mbar_arrive(smem_u32(&ctl->slot_empty[cur.slot]));
    cur.next(p.slots);
    return true;
}

// A whole warp's bounded wait, with one uniform branch where the phase is complete already; _cluster: for barriers that
// the peer CTA's threads, copies or commits complete.
template <typename Try>
__device__ __forceinline__ bool warp_wait_with(Try try_wait, const volatile uint32_t* abort_word, uint64_t timeout_ns) {
    if (__all_sync(0xffffffffu, try_wait())) return true;
    const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
    for (uint32_t it = 1;; ++it) {
        if (__all_sync(0xffffffffu, try_wait())) return true;
        if ((it & 31u) == 0u && __any_sync(0xffffffffu, *abort_word != 0u || globaltimer_ns() - t0 > timeout_ns)) return false;
    }
}
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const volatile uint32_t* abort_word,
                                          uint64_t timeout_ns) {
    return warp_wait_with([&] { return mbar_try_wait(bar, parity); }, abort_word, timeout_ns);
}
__device__ __forceinline__ bool warp_wait_cluster(uint32_t bar, uint32_t parity, const volatile uint32_t* abort_word,
                                                  uint64_t timeout_ns) {
    return warp_wait_with([&] { return mbar_try_wait_cluster(bar, parity); }, abort_word, timeout_ns);
}

// Whether a phase is complete, without waiting.
__device__ __forceinline__ bool mbar_test_cluster(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0u;
}

// Arrive of the lanes with `go`, predicated rather than branched around.
__device__ __forceinline__ void mbar_arrive_if(bool go, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar),
        "r"(go ? 1u : 0u)
        : "memory");
}

// (s0, s1) += (v0, v1) * scale, each rounded to nearest as by fmaf.
__device__ __forceinline__ void fma2(float& s0, float& s1, uint32_t v0, uint32_t v1, uint64_t scale2) {
    asm("{\n\t.reg .b64 s, v;\n\tmov.b64 s, {%0, %1};\n\tmov.b64 v, {%2, %3};\n\t"
        "fma.rn.f32x2 s, v, %4, s;\n\tmov.b64 {%0, %1}, s;\n\t}"
        : "+f"(s0), "+f"(s1)
        : "r"(v0), "r"(v1), "l"(scale2));
}

// Frees an accumulator on CTA 0's barrier.  Relaxed: nothing is handed over through
// memory.  The reads of the accumulator are complete (tcgen05.wait::ld), and
// the tcgen05 fences on both sides order them before the MMAs that follow the wait.  A
// release at cluster scope waits for every copy that this SM has in flight (measured:
// 2000 cycles per arrive, 1.0 us per block of columns instead of 0.6).
__device__ __forceinline__ void free_acc(bool go, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "@p mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n\t}" ::"r"(bar),
        "r"(go ? 1u : 0u)
        : "memory");
}

struct Maps8 {
    CUtensorMap x128, x64, x32, x16;  // activations
    CUtensorMap w;                    // weights
    CUtensorMap xs, ws;               // their scales
};

template <bool kF32Out>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_gemm8_kernel(const __grid_constant__ Maps8 tm, const __grid_constant__ CUtensorMap tmOut, const Params8 p) {
    using Out = typename std::conditional<kF32Out, float, bf16>::type;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* store_smem = smem + kStages * kStageBytes;
    uint8_t* scale_smem = store_smem + kEpiWarps * kStoreBytes;
    Ctl8* ctl = reinterpret_cast<Ctl8*>(scale_smem + kScaleSlots * kScaleSlotBytes);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const uint32_t peer = rank ^ 1u;

    pdl_wait();  // the table, the ticket and the status come from the kernel before
    if (warp == 0) {
        int cnt[kMaxExperts / 32], sum = 0;
#pragma unroll
        for (int i = 0; i < kMaxExperts / 32; ++i) {
            const int e = lane * (kMaxExperts / 32) + i;
            cnt[i] = (e < p.E) ? (p.mtile_start[e + 1] - p.mtile_start[e] + 1) / 2 : 0;
            sum += cnt[i];
        }
        int inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += u;
        }
        int run = inc - sum;
#pragma unroll
        for (int i = 0; i < kMaxExperts / 32; ++i) {
            const int e = lane * (kMaxExperts / 32) + i;
            if (e < p.E) ctl->pstart[e] = run;
            run += cnt[i];
        }
        if (lane == 31) ctl->pstart[p.E] = inc;
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_u32(&ctl->full[s]), 1);
            mbar_init(smem_u32(&ctl->empty[s]), 1);
        }
        for (int a = 0; a < 4; ++a) {
            mbar_init(smem_u32(&ctl->tmem_full[a]), 1);
            mbar_init(smem_u32(&ctl->tmem_empty[a]), 2 * kPartWarps);
        }
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(smem_u32(&ctl->slot_full[i]), 1);
            mbar_init(smem_u32(&ctl->slot_empty[i]), rank == 0 ? kSlotReaders0 : kSlotReaders1);
        }
        for (int i = 0; i < kScaleSlots; ++i) {
            mbar_init(smem_u32(&ctl->scale_full[i]), 1);
            mbar_init(smem_u32(&ctl->scale_empty[i]), kEpiWarps);
        }
        mbar_init(smem_u32(&ctl->drain), 1);
        ctl->abort_flag = 0;
        ctl->zero = 0;
        fence_mbar_init();
        prefetch_tensormap(&tm.x128);
        prefetch_tensormap(&tm.x64);
        prefetch_tensormap(&tm.x32);
        prefetch_tensormap(&tm.x16);
        prefetch_tensormap(&tm.w);
        prefetch_tensormap(&tm.xs);
        prefetch_tensormap(&tm.ws);
        prefetch_tensormap(&tmOut);
    }
    // The stages' rows start as zero.  Rows that no copy has written are multiplied all the same, and zeros take
    // less power than what lay there (1024 rows over 256 experts, 7168 to 2048: 636 us after a rest, so 603; for
    // seconds at the power cap 730, so 660).
    for (uint32_t i = threadIdx.x; i < kStages * (kHalfBytes / 16); i += kThreads)
        st_shared_v4(smem_u32(smem + i / (kHalfBytes / 16) * kStageBytes + i % (kHalfBytes / 16) * 16), make_uint4(0u, 0u, 0u, 0u));
    fence_proxy_async_shared();
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(&ctl->tmem_base), TMEM_COLS);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // both CTAs' barriers exist before any copy, commit or arrive targets them
    tc_fence_after();
    const uint32_t tmem_base = ctl->tmem_base;
    volatile uint32_t* abort_word = &ctl->abort_flag;
    const volatile uint32_t* never = &ctl->zero;
    const int total_tiles = ctl->pstart[p.E] * p.n_tiles;

    // The epilogue warps take the registers (their sums) that the other four give up: 56 + 2 x 224 of the
    // 3 x 168 per warp that the block is launched with (with 72 and 216 they spill: 640 us for 618).
    if (warp < kEpiWarp0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == 0) {
            // ---------------------------------------------------- TMA producer (both CTAs)
            if (elect_one()) {
                const uint32_t full0 = mapa_shared(smem_u32(&ctl->full[0]), 0);
                StageCursor<kStages> st;
                SlotCursor cur;
                uint32_t issued = 0, last_par = 0;
                bool ok = true;
                for (;;) {
                    int4 info;
                    if (!(ok = take_slot_one(ctl, cur, info, abort_word, p))) break;
                    if (info.x < 0) break;
                    // this CTA's rows (the second CTA may have none) and its part of each half's weight rows, in
                    // boxes of 64 (rows past a half of 64 are not multiplied)
                    const int cols = min(MMA_N, p.n - info.w);
                    const int m_row = info.y + static_cast<int>(rank) * BM;
                    const int box0 = box_rows(min(BM, info.z)), box1 = info.z > BM ? box_rows(info.z - BM) : 0;
                    const int box = rank == 0 ? box0 : box1;
                    const int size0 = min(128, cols), size1 = cols - 128, parts = cols > 128 ? 2 : 1;
                    const CUtensorMap* mm = box == 16 ? &tm.x16 : box == 32 ? &tm.x32 : box == 64 ? &tm.x64 : &tm.x128;
                    const int w_row = info.x * p.n + info.w;
                    const int n_row0 = w_row + static_cast<int>(rank) * (size0 >> 1);
                    const int n_row1 = w_row + 128 + static_cast<int>(rank) * (size1 >> 1);
                    const uint32_t stage_tx = static_cast<uint32_t>(box0 + box1 + 2 * 64 * parts) * kBlockK;
                    for (int kb = 0; kb < p.k_blocks; ++kb) {
                        if (!(ok = mbar_wait_bounded_cluster(smem_u32(&ctl->empty[st.stage]), st.phase ^ 1u, abort_word, p.timeout_ns)))
                            break;
                        const uint32_t sa = smem_u32(smem + st.stage * kStageBytes);
                        const uint32_t fb = full0 + st.stage * 8u;
                        if (rank == 0) mbar_arrive_expect_tx(smem_u32(&ctl->full[st.stage]), stage_tx);
                        if (box != 0) tma_load_2d_pair(sa, mm, kb * kBlockK, m_row, fb);
                        tma_load_2d_pair(sa + kHalfBytes, &tm.w, kb * kBlockK, n_row0, fb);
                        if (parts == 2) tma_load_2d_pair(sa + kHalfBytes + kPartBytes, &tm.w, kb * kBlockK, n_row1, fb);
                        issued |= 1u << st.stage;
                        last_par = (last_par & ~(1u << st.stage)) | (st.phase << st.stage);
                        st.next();
                    }
                    if (!ok) break;
                }
                if (!ok) {
                    raise_abort(ctl, peer);
                    report_error(p.status, MK_ERR_TIMEOUT, kSiteGemmProducer);
                }
                // Every stage that CTA 0 armed completes, and the commits that free the stages arrive (or
                // time out) before the CTA exits.
                for (int s = 0; s < kStages; ++s)
                    if ((issued >> s) & 1u) {
                        if (rank == 0)
                            mbar_wait_bounded_cluster(smem_u32(&ctl->full[s]), (last_par >> s) & 1u, never, p.timeout_ns);
                        if (ok)
                            mbar_wait_bounded_cluster(smem_u32(&ctl->empty[s]), (last_par >> s) & 1u, abort_word, p.timeout_ns);
                    }
            }
            __syncwarp();
        } else if (warp == 1) {
            if (rank == 0 && elect_one()) {
                // ------------------------------------------------ MMA issuer (CTA 0 only)
                const uint64_t desc0 = sw128_kmajor_desc(smem_u32(smem));  // + bytes / 16
                SlotCursor cur;
                StageCursor<kStages> st;
                AccCursor acc[2] = {AccCursor(0), AccCursor(1)};
                bool ok = true;
                while (ok) {
                    int4 info;
                    if (!(ok = take_slot_one(ctl, cur, info, abort_word, p))) break;
                    if (info.x < 0) break;
                    const int cols = min(MMA_N, p.n - info.w), parts = cols > 128 ? 2 : 1;
                    const uint32_t idesc0 = idesc_e4m3_f32(PAIR_M, static_cast<uint32_t>(min(128, cols)));
                    const uint32_t idesc1 = idesc_e4m3_f32(PAIR_M, static_cast<uint32_t>(parts == 2 ? cols - 128 : 128));
                    for (int kb = 0; kb < p.k_blocks && ok; ++kb) {
                        if (!(ok = mbar_wait_bounded_cluster(smem_u32(&ctl->full[st.stage]), st.phase, abort_word, p.timeout_ns))) break;
                        const uint64_t ad = desc0 + st.stage * (kStageBytes >> 4);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (h >= parts) continue;
                            if (!(ok = ok && mbar_wait_bounded_cluster(smem_u32(&ctl->tmem_empty[acc[h].acc]), acc[h].phase ^ 1u,
                                                               abort_word, p.timeout_ns)))
                                break;
                            tc_fence_after();
#pragma unroll
                            for (int kk = 0; kk < kBlockK / kUmmaK8; ++kk)
                                mma_e4m3_ss_pair(tmem_base + acc[h].acc * kAccCols, ad + kk * (kUmmaK8 >> 4),
                                                 ad + ((kHalfBytes + h * kPartBytes + kk * kUmmaK8) >> 4),
                                                 h == 0 ? idesc0 : idesc1, kk != 0 ? 1u : 0u);
                            mma_commit_pair_mc(smem_u32(&ctl->tmem_full[acc[h].acc]), 0x3);
                            acc[h].next();
                        }
                        if (!ok) break;
                        mma_commit_pair_mc(smem_u32(&ctl->empty[st.stage]), 0x3);
                        st.next();
                    }
                }
                if (!ok) {
                    raise_abort(ctl, peer);
                    report_error(p.status, MK_ERR_TIMEOUT, kSiteGemmMma);
                }
                // All MMAs issued complete before either CTA frees TMEM or shared memory.
                mma_commit_pair_mc(smem_u32(&ctl->drain), 0x1);
                if (!mbar_wait_bounded_cluster(smem_u32(&ctl->drain), 0u, never, p.timeout_ns))
                    report_error(p.status, MK_ERR_TIMEOUT, kSiteGemmDrain);
            }
            __syncwarp();
        } else if (warp == kScaleWarp) {
            // ---------------------------------------------------- scales (both CTAs)
            if (elect_one()) {
                StageCursor<kScaleSlots> sc;
                SlotCursor cur;
                bool ok = true;
                int issued = 0;
                for (;;) {
                    int4 info;
                    if (!(ok = take_slot_one(ctl, cur, info, abort_word, p))) break;
                    if (info.x < 0) break;
                    const int m_row = info.y + static_cast<int>(rank) * BM;
                    const int ws_row = info.x * p.n_blocks + info.w / kBlockN;
                    for (int kb = 0; kb < p.k_blocks; kb += kScaleSpan) {
                        if (!(ok = mbar_wait_bounded(smem_u32(&ctl->scale_empty[sc.stage]), sc.phase ^ 1u, abort_word,
                                                     p.timeout_ns)))
                            break;
                        const uint32_t bar = smem_u32(&ctl->scale_full[sc.stage]);
                        const uint32_t dst = smem_u32(scale_smem + sc.stage * kScaleSlotBytes);
                        const int groups = (min(kScaleSpan, p.k_blocks - kb) + kScaleGroup - 1) / kScaleGroup;
                        mbar_arrive_expect_tx(bar, groups * (kXScaleBytes + kWScaleBytes));
                        for (int g = 0; g < groups; ++g) {
                            tma_load_2d(dst + g * kScaleGroupBytes, &tm.xs, kb + g * kScaleGroup, m_row, bar);
                            tma_load_2d(dst + g * kScaleGroupBytes + kXScaleBytes, &tm.ws, kb + g * kScaleGroup, ws_row, bar);
                        }
                        sc.next();
                        issued = min(issued + 1, kScaleSlots);
                    }
                    if (!ok) break;
                }
                if (!ok) {
                    raise_abort(ctl, peer);
                    report_error(p.status, MK_ERR_TIMEOUT, kSiteGemmProducer);
                }
                // The copies issued last land before the CTA exits.
                for (int i = 0; i < issued; ++i) {
                    sc.prev();
                    mbar_wait_bounded(smem_u32(&ctl->scale_full[sc.stage]), sc.phase, never, p.timeout_ns);
                }
            }
            __syncwarp();
        } else if (warp == kSchedWarp) {
            const bool leader = elect_one();
            const int lead = __ffs(__ballot_sync(0xffffffffu, leader)) - 1;
            SlotCursor cur;
            bool ok = true;
            if (rank == 0) {
                // ------------------------------------------------ tile scheduler (CTA 0)
                const uint32_t peer_slot0 = mapa_shared(smem_u32(&ctl->slot[0]), peer);
                const uint32_t peer_slot_full0 = mapa_shared(smem_u32(&ctl->slot_full[0]), peer);
                for (;;) {
                    if (!__all_sync(0xffffffffu, mbar_wait_bounded_cluster(smem_u32(&ctl->slot_empty[cur.slot]),
                                                                          cur.phase ^ 1u, abort_word, p.timeout_ns))) {
                        ok = false;
                        break;
                    }
                    uint32_t tk = 0;
                    if (leader) tk = atomicAdd(p.ticket, 1u);
                    tk = __shfl_sync(0xffffffffu, tk, lead);
                    int4 nfo = make_int4(-1, 0, 0, 0);
                    if (tk < static_cast<uint32_t>(total_tiles)) nfo = decode_tile(static_cast<int>(tk), ctl, p);
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
        asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
        const int sub = warp & 3;                  // TMEM lanes [32 sub, 32 sub + 32) are this warp's
        const int part = (warp - kEpiWarp0) / kPartWarps;
        const uint32_t buf = smem_u32(store_smem + (warp - kEpiWarp0) * kStoreBytes);
        const uint32_t buf_row = lane * 128 + (lane & 7) * 16;
        constexpr int kPieceCols = 128 / sizeof(Out);  // columns of a 128-byte row of a store
        const uint32_t acc_empty0 = mapa_shared(smem_u32(&ctl->tmem_empty[0]), 0);
        const uint32_t tlane = tmem_base + (static_cast<uint32_t>(sub * 32) << 16);
        SlotCursor cur;
        StageCursor<kScaleSlots> sc;
        AccCursor acc(part);
        bool ok = true;
        float sum[kBlockN];
        bool ready = false;
        auto acc_wait = [&]() {
            const bool r = ready ||
                           warp_wait_cluster(smem_u32(&ctl->tmem_full[acc.acc]), acc.phase, abort_word, p.timeout_ns);
            tc_fence_after();
            return r;
        };
        auto acc_release = [&]() {
            tc_fence_before();
            __syncwarp();
            free_acc(lane == 0, acc_empty0 + acc.acc * 8u);
            acc.next();
        };
        // A block's scales multiplied, for blocks in order: a group's four are read, and its slot freed, at its start.
        const uint32_t x_at = (sub * 32 + lane) * 16, w_at = kXScaleBytes + part * 16;
        float4 scales;
        auto scale_of = [&](int kb, float& scale) {
            if (kb % kScaleGroup == 0) {
                if (kb % kScaleSpan == 0 && !warp_wait(smem_u32(&ctl->scale_full[sc.stage]), sc.phase, abort_word, p.timeout_ns))
                    return false;
                const uint32_t src = smem_u32(scale_smem) + sc.stage * kScaleSlotBytes + kb % kScaleSpan / kScaleGroup * kScaleGroupBytes;
                const float4 x = lds4(src + x_at), w = lds4(src + w_at);
                scales = make_float4(x.x * w.x, x.y * w.y, x.z * w.z, x.w * w.w);
                if (kb % kScaleSpan == kScaleSpan - kScaleGroup || kb + kScaleGroup >= p.k_blocks) {
                    __syncwarp();
                    mbar_arrive_if(lane == 0, smem_u32(&ctl->scale_empty[sc.stage]));
                    sc.next();
                }
            }
            scale = scales.x;
            scales = make_float4(scales.y, scales.z, scales.w, 0.0f);
            return true;
        };
        while (ok) {
            int4 info;
            if (!(ok = take_slot(ctl, cur, info, abort_word, p))) break;
            if (info.x < 0) break;
            const int cols = min(MMA_N, p.n - info.w);
            const int size = min(kBlockN, cols - part * kBlockN);  // of this half (<= 0: none)
#pragma unroll
            for (int i = 0; i < kBlockN; ++i) sum[i] = 0.0f;
            // this thread's row, the part's columns
            const int first = static_cast<int>(rank) * BM + sub * 32;  // of the warp's rows, in the tile
            const int group = min(32, info.z - first);                // of them, the expert's (<= 0: none)
            const int col0 = info.w + part * kBlockN;
            // loaded here, 600 cycles before its use (11 blocks per tile: 63 us, so 61)
            const float wr = p.row_weight != nullptr && lane < group ? __ldg(p.row_weight + info.y + first + lane) : 1.0f;
            if (size > 0 && group > 0) {
                for (int kb = 0; kb < p.k_blocks; ++kb) {
                    float scale;
                    if (!(ok = scale_of(kb, scale) && acc_wait())) break;
                    const uint32_t at = tlane + acc.acc * kAccCols;
                    uint64_t scale2;
                    asm("mov.b64 %0, {%1, %1};" : "=l"(scale2) : "f"(scale));
#pragma unroll
                    for (int c = 0; c < kBlockN; c += 32) {
                        uint32_t v[32];
                        tmem_ld_32x32b_x32(at + c, v);
                        tmem_ld_wait();
                        if (c + 32 == kBlockN) {
                            acc_release();
                            ready = __all_sync(0xffffffffu, mbar_test_cluster(smem_u32(&ctl->tmem_full[acc.acc]), acc.phase));
                        }
#pragma unroll
                        for (int q = 0; q < 32; q += 2) fma2(sum[c + q], sum[c + q + 1], v[q], v[q + 1], scale2);
                    }
                }
            } else {  // keeps step
                float scale;
                for (int kb = 0; kb < p.k_blocks && ok; ++kb) {
                    if (!(ok = scale_of(kb, scale))) break;
                    if (size <= 0) continue;
                    if (!(ok = acc_wait())) break;
                    acc_release();
                    ready = false;
                }
            }
            if (!ok) break;
            if (size <= 0 || group <= 0) continue;
#pragma unroll
            for (int c = 0; c < kBlockN; c += kPieceCols) {
                if (c >= size) break;  // a multiple of 64
                if (lane == 0) bulk_wait_read<0>();  // the last store has read the buffer
                __syncwarp();
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    uint4 o;
                    if (kF32Out)
                        o = make_uint4(__float_as_uint(sum[c + 4 * q] * wr), __float_as_uint(sum[c + 4 * q + 1] * wr),
                                       __float_as_uint(sum[c + 4 * q + 2] * wr), __float_as_uint(sum[c + 4 * q + 3] * wr));
                    else
                        o = make_uint4(pack_bf16x2(sum[c + 8 * q] * wr, sum[c + 8 * q + 1] * wr),
                                       pack_bf16x2(sum[c + 8 * q + 2] * wr, sum[c + 8 * q + 3] * wr),
                                       pack_bf16x2(sum[c + 8 * q + 4] * wr, sum[c + 8 * q + 5] * wr),
                                       pack_bf16x2(sum[c + 8 * q + 6] * wr, sum[c + 8 * q + 7] * wr));
                    st_shared_v4(buf + (buf_row ^ (q * 16)), o);
                }
                if (group == 32) {
                    fence_proxy_async_shared();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_2d(&tmOut, col0 + c, info.y + first, buf);
                        bulk_commit();
                    }
                } else {
                    __syncwarp();
                    // 8 lanes per row of 128 bytes
                    Out* o = static_cast<Out*>(p.out) + static_cast<int64_t>(info.y + first) * p.n + col0 + c;
                    for (int r = lane >> 3; r < group; r += 4) {
                        const float4 v = lds4(buf + r * 128 + (((lane & 7) * 16) ^ ((r & 7) * 16)));
                        reinterpret_cast<float4*>(o + static_cast<int64_t>(r) * p.n)[lane & 7] = v;
                    }
                    __syncwarp();
                }
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

// 2-D row-major codes [rows, inner], box {128, box_rows}, 128-byte swizzle.
bool make_map8(CUtensorMap* m, const void* base, uint64_t inner, uint64_t rows, uint32_t box_rows) {
    auto fn = encode_fn();
    if (fn == nullptr) return false;
    const cuuint64_t dims[2] = {inner, rows};
    const cuuint64_t strides[1] = {inner};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(kBlockK), box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Scales [rows, pitch(d)] fp32, box {4, box_rows}.
bool make_map_scales(CUtensorMap* m, const void* base, int d, uint64_t rows, uint32_t box_rows) {
    auto fn = encode_fn();
    if (fn == nullptr) return false;
    const cuuint64_t pitch = static_cast<cuuint64_t>(scale_pitch(d));
    const cuuint64_t dims[2] = {pitch, rows};
    const cuuint64_t strides[1] = {pitch * 4};
    const cuuint32_t box[2] = {kScaleGroup, box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool kF32Out>
cudaError_t launch8(const Maps8& m, const CUtensorMap& out, const Params8& p, int64_t S, cudaStream_t s) {
    static std::atomic<int> max_clusters[64];  // per device, 0 until configured
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    auto fn = grouped_gemm8_kernel<kF32Out>;
    LaunchCfg lc(dim3(2 * std::max(1, device_sm_count() / 2)), dim3(kThreads), kSmem8, s, true, 2);
    int n = dev < 64 ? max_clusters[dev].load(std::memory_order_acquire) : 0;
    if (n == 0) {
        err = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem8));
        if (err != cudaSuccess) return err;
        err = cudaOccupancyMaxActiveClusters(&n, fn, &lc.cfg);
        if (err != cudaSuccess) return err;
        if (n < 1) return cudaErrorInvalidConfiguration;
        if (dev < 64) max_clusters[dev].store(n, std::memory_order_release);
    }
    // Upper bound on the tiles: every expert adds at most one partial block.
    const int64_t tiles = ((S + PAIR_M - 1) / PAIR_M + p.E) * static_cast<int64_t>(p.n_tiles);
    lc.cfg.gridDim = dim3(2 * static_cast<unsigned>(std::min<int64_t>(n, tiles)));
    err = cudaLaunchKernelEx(&lc.cfg, fn, m, out, p);
    if (err != cudaSuccess) return err;
    return cudaGetLastError();
}

}  // namespace
}  // namespace mk

using namespace mk;

extern "C" int mk_moe_scale_pitch(int c) { return c > 0 ? scale_pitch(c) : 0; }

extern "C" mk_status mk_moe_grouped_gemm8(const uint8_t* codes, const float* scales, const int32_t* expert_offsets,
                                          const uint8_t* w_codes, const float* w_scales, const float* row_weight,
                                          int64_t S, int d, int E, int n, void* out, int out_type, void* ws,
                                          size_t ws_bytes, void* stream) {
    const mk_status st = check_sizes(0, d, E, 1, n);
    if (st != MK_OK) return st;
    if (S < 0) return MK_ERR_INVALID_ARG;
    // Rows and columns are 32-bit coordinates each, offsets in 64 bits: eight rows for each of four million tokens, of any length.
    if (S >= 1 << 25 || S * std::max(d, n) >= (int64_t(1) << 40)) return MK_ERR_UNSUPPORTED;
    // Columns are counted in 32 bits, a tile's past the end included; and a tile of 2^28 columns takes 1.2 s, a longer
    // one more than the bounded waits for its end allow.
    if (d >= 1 << 28 || n >= 1 << 30) return MK_ERR_UNSUPPORTED;
    if (out_type != MK_TYPE_BF16 && out_type != MK_TYPE_FP32) return MK_ERR_INVALID_ARG;
    if (S == 0) return MK_OK;
    if (!codes || !scales || !expert_offsets || !w_codes || !w_scales || !out) return MK_ERR_INVALID_ARG;
    if (!aligned16(codes) || !aligned16(scales) || !aligned16(w_codes) || !aligned16(w_scales) || !aligned16(out))
        return MK_ERR_INVALID_ARG;
    if (ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0 || ws_bytes < 256 + 4 * (size_t(E) + 1))
        return MK_ERR_WORKSPACE;
    const int64_t n_tiles = (n + MMA_N - 1) / MMA_N;
    if (((S + PAIR_M - 1) / PAIR_M + E) * n_tiles >= (int64_t(1) << 31)) return MK_ERR_UNSUPPORTED;
    if (!device_is_sm103()) return MK_ERR_UNSUPPORTED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool fp32 = out_type == MK_TYPE_FP32;
    Maps8 m;
    CUtensorMap o;
    const uint64_t w_rows = static_cast<uint64_t>(E) * n;
    if (!make_map8(&m.x128, codes, d, S, 128) || !make_map8(&m.x64, codes, d, S, 64) ||
        !make_map8(&m.x32, codes, d, S, 32) || !make_map8(&m.x16, codes, d, S, 16) ||
        !make_map8(&m.w, w_codes, d, w_rows, 64) || !make_map_scales(&m.xs, scales, d, S, BM) ||
        !make_map_scales(&m.ws, w_scales, d, static_cast<uint64_t>(E) * ((n + kBlockN - 1) / kBlockN), 2) ||
        !make_map_box(&o, out, fp32, n, S, 32))
        return MK_ERR_CUDA;
    Params8 p;
    p.offsets = expert_offsets;
    p.status = static_cast<uint32_t*>(ws);
    p.mtile_start = reinterpret_cast<const int32_t*>(static_cast<uint8_t*>(ws) + 256);
    p.row_weight = row_weight;
    p.out = out;
    p.E = E;
    p.n = n;
    p.n_tiles = static_cast<int>(n_tiles);
    p.n_blocks = (n + kBlockN - 1) / kBlockN;
    p.k_blocks = (d + kBlockK - 1) / kBlockK;
    p.slots = kSlots;
    p.ticket = p.status + 4;
    p.timeout_ns = kDefaultTimeoutNs;
    if (launch_mtile_table(expert_offsets, E, S, reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + 256), p.status, s,
                           true) != cudaSuccess)
        return MK_ERR_CUDA;
    const cudaError_t err = fp32 ? launch8<true>(m, o, p, S, s) : launch8<false>(m, o, p, S, s);
    return err == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}
