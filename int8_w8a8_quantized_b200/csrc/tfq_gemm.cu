// tfq_gemm.cu -- scaled FP8 GEMM with fused epilogue on 5th-generation
// tensor cores (tcgen05, sm_100a).
//
// Computes out[m,n] = bf16_rn(acc[m,n] * s_a[m] * s_w[n] + bias[n]) with
// acc[m,n] = sum_k e4m3(A[m,k]) * e4m3(W[n,k]) accumulated in fp32: the
// scaled GEMM of the TeleFuser "Quantization" page (sections "Scaled FP8
// checkpoints" and "tf-kernel FP8: online W8A8": per-token activation
// scales, per-output-channel weight scales, BF16 output).
//
// Two kernels: scaled_mm_pair_kernel (clusters of two CTAs computing 256 x
// 256 tiles with tcgen05.mma.cta_group::2; every problem of 512 rows or more)
// and scaled_mm_kernel (one CTA per 128 x 256 tile, smaller problems).  Both
// are templated on the operand kind: E4M3 with an fp32 or fp16 accumulator,
// or S8 with an s32 accumulator (the INT8 W8A8 path).
//
// One-CTA structure (one persistent CTA per SM, 192 threads; the pair kernel
// below follows it):
//   warp 0      TMA producer: streams 128x128 A tiles and 256x128 B tiles
//               (K-major, 128-byte swizzle) into a 4-stage shared-memory
//               ring, completion counted on "full" mbarriers.
//   warp 1      allocates 512 TMEM columns (two 128x256 fp32 accumulators)
//               and, from one thread, issues tcgen05.mma kind::f8f6f4
//               (M=128, N=256, K=32 per instruction, 4 per stage); each
//               stage is released to the producer by tcgen05.commit onto its
//               "empty" mbarrier, each finished tile by a commit onto the
//               accumulator's "tmem_full" mbarrier.
//   warps 2..5  epilogue: tcgen05.ld a 32-row quarter of the accumulator
//               (warp w may read TMEM lanes 32*(w%4)..+31), apply s_a, s_w
//               and bias in fp32, round to bf16, write 64-column chunks into
//               a 128-byte-swizzled staging buffer and TMA-store them; the
//               accumulator is handed back through "tmem_empty" so the MMA
//               of the next tile overlaps this epilogue.
// Tiles are visited in bands of N tiles holding ~40 MB of weight, each band
// sweeping every M tile, so that the CTAs running at the same time share the
// band's weight panels (kept in L2) and each activation panel; the pair
// kernel also keeps its clusters within one tile of each other (pacing,
// see tfq_gemm_common.cuh) and runs a last round of at most half as many
// tiles as clusters as half-width (256 x 128) tiles.  M and N tails are handled by
// TMA (zero fill on load, clipping on store); K tails by zero fill.
// Every wait is bounded (see tfq_ptx.cuh); a CTA that gives up records it in
// the error word, drains its own outstanding copies and MMAs, frees TMEM and
// returns.
#include <type_traits>

#include "tfq_gemm_common.cuh"
#include "tfq_quant_row.cuh"

namespace tfq {
namespace {

template <int kAcc>
__global__ void __launch_bounds__(THREADS, 1)
    scaled_mm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                           const __grid_constant__ CUtensorMap tmY, GemmArgs p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sA = smem;
    uint8_t* sB = sA + STAGES * A_STAGE_BYTES;
    uint8_t* sE = sB + STAGES * B_STAGE_BYTES;
    uint64_t* full = reinterpret_cast<uint64_t*>(sE + SMEM_EPI);
    uint64_t* empty = full + STAGES;
    uint64_t* tmem_full = empty + STAGES;
    uint64_t* tmem_empty = tmem_full + 2;
    uint64_t* drain = tmem_empty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int total_tiles = p.m_tiles * p.n_tiles;

    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tmem_full[i], 1);
            mbar_init(&tmem_empty[i], EPI_WARPS);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tensormap(&tmA);
        prefetch_tensormap(&tmB);
        prefetch_tensormap(&tmY);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    pdl_allow_next();
    pdl_wait();  // the set-up above may overlap the previous kernel; global memory only from here

    if (warp == 0) {
        // ---------------------------------------------------- TMA producer
        if (lane == 0) {
            uint64_t pol_a, pol_b;
            l2_policies(p, pol_a, pol_b);
            int it = 0;
            int issued_phase[STAGES];
            for (int i = 0; i < STAGES; ++i) issued_phase[i] = -1;
            bool ok = true;
            for (int t = blockIdx.x; t < total_tiles && ok; t += gridDim.x) {
                int tm, tn;
                tile_coords(t, p, tm, tn);
                for (int kb = 0; kb < p.k_blocks; ++kb, ++it) {
                    const int st = it % STAGES;
                    const uint32_t ph = static_cast<uint32_t>(it / STAGES) & 1u;
                    if (!mbar_wait(&empty[st], ph ^ 1u, abort_flag)) {
                        give_up(abort_flag, p.err, kErrGemmProducer);
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&full[st], A_STAGE_BYTES + B_STAGE_BYTES);
                    tma_load_2d_hint(sA + st * A_STAGE_BYTES, &tmA, kb * BK, tm * BM, &full[st], pol_a);
                    tma_load_2d_hint(sB + st * B_STAGE_BYTES, &tmB, kb * BK, tn * BN, &full[st], pol_b);
                    issued_phase[st] = static_cast<int>(ph);
                }
            }
            // Outstanding loads must land before the CTA may exit.
            for (int i = 0; i < STAGES; ++i)
                if (issued_phase[i] >= 0 && !mbar_wait(&full[i], static_cast<uint32_t>(issued_phase[i]), nullptr))
                    atomicOr(p.err, kErrGemmDrain);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------ MMA issuer
        if (lane == 0) {
            int it = 0, tcount = 0;
            bool ok = true;
            for (int t = blockIdx.x; t < total_tiles && ok; t += gridDim.x, ++tcount) {
                const int buf = tcount & 1;
                const uint32_t use = static_cast<uint32_t>(tcount >> 1);
                if (!mbar_wait(&tmem_empty[buf], (use & 1u) ^ 1u, abort_flag)) {
                    give_up(abort_flag, p.err, kErrGemmMma);
                    break;
                }
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(buf * BN);
                for (int kb = 0; kb < p.k_blocks; ++kb, ++it) {
                    const int st = it % STAGES;
                    const uint32_t ph = static_cast<uint32_t>(it / STAGES) & 1u;
                    if (!mbar_wait(&full[st], ph, abort_flag)) {
                        give_up(abort_flag, p.err, kErrGemmMma);
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t a_desc = sw128_kmajor_desc(sA + st * A_STAGE_BYTES);
                    const uint64_t b_desc = sw128_kmajor_desc(sB + st * B_STAGE_BYTES);
#pragma unroll
                    for (int k = 0; k < BK / UMMA_K; ++k) {
                        // advance the start address by k * 32 bytes inside the swizzle atom
                        const uint64_t koff = static_cast<uint64_t>((k * UMMA_K) >> 4);
                        mma_e4m3<kAcc == kAccS32>(d_tmem, a_desc + koff, b_desc + koff, make_idesc<kAcc>(BM, BN),
                                      (kb | k) != 0 ? 1u : 0u);
                    }
                    mma_commit(&empty[st]);
                }
                if (ok) mma_commit(&tmem_full[buf]);
            }
            // Every MMA issued above must finish before TMEM is freed.
            mma_commit(drain);
            if (!mbar_wait(drain, 0, nullptr)) atomicOr(p.err, kErrGemmDrain);
        }
    } else {
        // -------------------------------------------------------- epilogue
        const int ew = warp - 2;         // 0..3: staging buffers
        const int quarter = warp & 3;    // TMEM lanes this warp may read
        uint8_t* ebuf = sE + static_cast<size_t>(ew) * EPI_BUF_BYTES;
        float* colp = reinterpret_cast<float*>(sE + EPI_WARPS * EPI_BUF_BYTES + ew * COLP_BYTES);
        int tcount = 0;
        for (int t = blockIdx.x; t < total_tiles; t += gridDim.x, ++tcount) {
            int tm, tn;
            tile_coords(t, p, tm, tn);
            stage_col_params<BN>(p, colp, tn * BN, lane);
            const int buf = tcount & 1;
            const uint32_t use = static_cast<uint32_t>(tcount >> 1);
            if (!mbar_wait_warp(&tmem_full[buf], use & 1u, abort_flag)) {
                if (lane == 0) give_up(abort_flag, p.err, kErrGemmEpilogue);
                break;
            }
            tc_fence_after();
            const int row0 = tm * BM + quarter * 32;
            const int m = row0 + lane;
            const float sa = (m < p.M) ? __ldg(p.s_a + m) : 0.0f;
            const uint32_t t_row = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
                                   static_cast<uint32_t>(buf * BN);
            store_tile_rows<BN, kAcc>(p, tmY, t_row, ebuf, colp, tn * BN, row0, sa, lane);
            // All of this warp's TMEM reads of `buf` are complete: hand it back.
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tmem_empty[buf]);
        }
        if (lane == 0) bulk_wait<0>();
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem_base, TMEM_COLS);
    }
}

// ---------------------------------------------------------------------------
// CTA-pair kernel (cta_group::2): a cluster of two CTAs on two SMs computes a
// 256 x PBN tile.  CTA r of the pair loads rows [128 r, 128 r + 128) of the
// tile's A panel and rows [PBN/2 r, PBN/2 (r + 1)) of its B panel into its
// own shared memory; the even CTA's single MMA thread issues
// tcgen05.mma.cta_group::2 (M = 256, N = PBN, K = 32), which reads both
// CTAs' halves and leaves rows [128 r, 128 r + 128) of the accumulator in
// CTA r's TMEM.  Per CTA a stage is 16 KiB of A + PBN/2 x 128 B of B (32 KiB
// at PBN = 256 instead of 48 KiB), so six stages fit and each SM pulls a
// third less data from L2 per FLOP.  Both CTAs' loads complete on the even
// CTA's "full" barrier (which expects the bytes of both); the MMA thread
// releases each stage and each accumulator to both CTAs with a multicast
// commit; both CTAs' epilogue warps hand the accumulator back on the even
// CTA's "tmem_empty" barrier.  The epilogue is the same as above.
constexpr int PAIR_STAGES = 6;

template <int PBN>
struct PairCfg {
    static constexpr int kBHalf = PBN / 2;                      // B rows per CTA
    static constexpr int kAStage = 128 * BK;                    // 16 KiB
    static constexpr int kBStage = kBHalf * BK;
    static constexpr int kTmemCols = 512;                       // two PBN-column accumulators, power of 2
    static constexpr size_t kRing = static_cast<size_t>(PAIR_STAGES) * (kAStage + kBStage);
    static constexpr size_t kSmem = 1024 + kRing + SMEM_EPI + (2 * PAIR_STAGES + 4 + 1) * 8 + 16;
    static constexpr size_t kSmemLora = kSmem + 8 + 20 * PAIR_STAGES;  // a barrier; two and a word per stage
    static_assert(kSmemLora <= 232448, "shared memory budget exceeded");
    static_assert(2 * PBN <= kTmemCols, "two accumulators must fit in TMEM");
    static_assert(PBN % 64 == 0 && PBN >= 64 && PBN <= 256, "N tile");
};

// The CTA-pair kernel that quantizes its own activations (kQuant != 0) adds
// QUANT_WARPS quantizer warps to every CTA.  They take rows of the bf16
// activations in increasing order from a counter shared by the whole grid,
// quantize each (one warp per row: max |x|, the fp32 scale, the E4M3 codes,
// exactly as the row quantizer kernels do) into the A operand and the row
// scales, and publish each finished row on its 128-row share's counter.
// They wait for nothing, so they always finish; the producers and the
// epilogues wait (bounded) for the shares they need.  The tensor cores of an
// SM run the MMAs of the current tiles while its quantizer warps, with
// those of every other SM, stream the rows of the coming tiles.
// Measured on B200 this overlap does not pay: the GEMM slows down by about
// the quantizer's own time (the quantizer's loads and stores share the SM's
// memory path with the operand traffic of the MMAs, and under the power cap
// the same work costs the same energy), so the row quantizer followed by the
// plain GEMM stays the default path; this variant is kept, parity-tested,
// as the measured alternative.
// kQuant: 0 = operands given quantized; 1 = E4M3 rows, qmax an E4M3 value
// (no clamp needed); 2 = E4M3 rows with the clamp to +-qmax.
#ifndef TFQ_QUANT_WARPS
#define TFQ_QUANT_WARPS 8  // measured on B200: 8 beat 4 (the warps are latency bound, one row at a time)
#endif
constexpr int QUANT_WARPS = TFQ_QUANT_WARPS;
constexpr int QUANT_SEG = 20;  // 16-byte units per lane per segment: a K = 5120 row in one pass

constexpr int LORA_WARPS = 4;  // row warps of the kernel with low-rank adapters (below)

template <int kQuant, bool kLora = false>
constexpr int pair_threads() {
    return THREADS + (kQuant != 0 ? QUANT_WARPS * 32 : 0) + (kLora ? LORA_WARPS * 32 : 0);
}

// Rows of the 128-row share of A starting at row0 that must be quantized
// before they may be read (0 past the end of M).
__device__ __forceinline__ unsigned share_rows(const GemmArgs& p, int row0) {
    return row0 >= p.M ? 0u : static_cast<unsigned>(min(128, p.M - row0));
}

// Waits (bounded; one thread) until the share of A starting at row0 is
// quantized: an acquire load of its counter, so that this thread's later
// reads see the codes and scales written by the quantizer warps, then a
// proxy fence, so that its later TMA loads (the async proxy) see them too.
__device__ __forceinline__ bool wait_share_quantized(const GemmArgs& p, int row0, volatile int* abort) {
    const unsigned need = share_rows(p, row0);
    if (need == 0) return true;
    const unsigned* ctr = p.q_share_rows + row0 / 128;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t i = 0; i < TFQ_WAIT_LIMIT_POLLS; ++i) {
        unsigned v;
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(ctr) : "memory");
        if (v >= need) {
            asm volatile("fence.proxy.async.global;" ::: "memory");
            return true;
        }
        if ((i & 15u) == 15u) {
            if (abort != nullptr && *abort != 0) return false;
            if (globaltimer_ns() - t0 > TFQ_WAIT_LIMIT_NS) return false;
        }
        __nanosleep(256);
    }
    return false;
}

// The quantizer warps' loop (see above).
template <int kQuant>
__device__ __forceinline__ void quantize_rows_for_gemm(const GemmArgs& p, int lane) {
    const int units = p.K >> 3;
    const uint64_t keep = l2_policy_evict_last(), drop = l2_policy_evict_first();
    for (;;) {
        unsigned r = 0;
        if (lane == 0) r = atomicAdd(p.q_next_row, 1u);
        r = __shfl_sync(0xFFFFFFFFu, r, 0);
        if (r >= static_cast<unsigned>(p.M)) break;
        const size_t off = static_cast<size_t>(r) * static_cast<size_t>(units);
        quantize_row_warp<false, kQuant == 2, QUANT_SEG>(p.qx + off, units, p.qmax,
                                                        reinterpret_cast<uint2*>(p.qa + off * 8), p.qs + r, lane,
                                                        keep, drop);
        // Publish the row: each lane's stores are made visible to the async
        // proxy (the readers' TMA loads), the warp barrier orders them before
        // lane 0's release increment of the share counter (a release is
        // cumulative over the writes it has observed).  A full fence per
        // lane instead measured 10 % slower on the image-DiT Q projection.
        asm volatile("fence.proxy.async.global;" ::: "memory");
        __syncwarp();
        if (lane == 0)
            asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(p.q_share_rows + r / 128) : "memory");
    }
}

// Tensor maps of the CTA-pair kernel per Linear (see GemmArgs::n_lin): the
// weight with 128-row boxes (b) and 64-row boxes (bq, the half-width tiles of
// a split last round), and the output (y).
struct PairMaps {
    CUtensorMap b[kMaxLinears];
    CUtensorMap bq[kMaxLinears];
    CUtensorMap y[kMaxLinears];
};

// One Linear's operands on the host side: weight codes [N, K], column scales,
// bias (may be null), N, output [M, N].
struct LinearOperands {
    const void* W;
    const float* s_w;
    const void* bias;
    int64_t N;
    void* out;
};

// The CTA-pair kernel with low-rank adapters beside the Linear (kLora): row m
// adds sum_r t[m,r] Bs[a,n,r], a = idx[m], to its accumulator, with t and Bs in
// units of the row's and the column's scale (tfq_lora.cu), so the epilogue's
// s_a s_w covers both sums.  A tile's accumulator starts with the kind::f16
// stages of the adapters present in its 256 rows, then takes the kind::f8f6f4
// stages of the Linear.  Such a stage holds 64 columns: those of one adapter's
// rank, or the whole rank of two (R <= 32) or four (R <= 16) adapters side by
// side as operand tiles of their own.  Its B operands are the adapters' Bs
// tiles (TMA); the A operand is t with the rows of other
// adapters zero, which four more warps per CTA write: a thread keeps its
// row's t in registers and stores it to the stage of the row's own adapter,
// zeros to the others.  (Measured on B200 with 12 adapters of rank 24 in any
// order, 1777 x 13824 x 5120: a TMA gather of t's rows and a zero row instead
// took 195 us against 102 us without adapters, 660 us when all CTAs read the
// same zero row.  Now 126 us; rank 64 in runs on 32760 x 5120 x 5120 585 us
// against some 560 without, both bound by the tensor cores.)  The adapters of
// a tile are enumerated in increasing order from idx by the producers and the
// row warps alike, from values loaded a tile ahead.
//
// Only instructions of one shape and accumulator are ordered among themselves,
// so the adapters' instructions must be complete before the Linear's first one
// on the same accumulator.  To wait for that without idling the tensor cores,
// the adapters' stages of a tile come kLoraLead stages before the end of the
// tile before it (whose accumulator is the other one): they are long complete
// when their tile begins.  The even producer leaves each stage's kind in
// shared memory, and the MMA thread does what it says.
//
// kHalves: t has 16 bits, as an upper and a lower bf16 half, and every chunk of it
// is two stages, one for each half, with the same B.
struct LoraPairMaps : PairMaps {
    CUtensorMap bs;   // Bs [n_adapters * N, R], kLora x PBN / 2 boxes
    CUtensorMap bsq;  // ... kLora x PBN / 4 boxes (half-width tiles)
    const int32_t* idx;
    const uint4* t;  // [M, R] bf16; kHalves: [M, 2 R], upper and lower halves
    int n_adapters;
    int R;
};
constexpr int kLoraLead = 3;

// A stage's contents, for the MMA thread.
enum : uint32_t {
    kStageSteps = 7u,      // kind::f16 instructions of an adapter's stage
    kStageLora = 1u << 3,  // an adapter's stage
};

// idx[m] where it names an adapter, else 0xFFFFFFFF.
__device__ __forceinline__ uint32_t row_adapter(const int32_t* idx, int m, int M, int n_adapters) {
    if (m >= M) return 0xFFFFFFFFu;
    const uint32_t a = static_cast<uint32_t>(__ldg(idx + m));
    return a < static_cast<uint32_t>(n_adapters) ? a : 0xFFFFFFFFu;
}

// The adapters of the 256 rows of a tile, eight per lane.
struct TileAdapters {
    uint32_t v[8];
    uint32_t from = 0;
    __device__ __forceinline__ void load(const int32_t* idx, int tm, int M, int n_adapters, int lane) {
        from = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = row_adapter(idx, tm * 256 + lane * 8 + i, M, n_adapters);
    }
    // The next adapters in increasing order, at most `most` (up to 4) of them;
    // how many.  All lanes call it.
    __device__ __forceinline__ int next(uint32_t (&a)[4], int most) {
        int n = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            a[j] = 0xFFFFFFFFu;
            if (j < most && n == j) {
#pragma unroll
                for (int i = 0; i < 8; ++i) a[j] = min(a[j], v[i] >= from ? v[i] : 0xFFFFFFFFu);
                a[j] = __reduce_min_sync(0xFFFFFFFFu, a[j]);
                if (a[j] != 0xFFFFFFFFu) {
                    from = a[j] + 1;
                    ++n;
                }
            }
        }
        return n;
    }
};

// Work item w of the cluster: its tile coordinates and half; false past the last.
template <int PBN>
__device__ __forceinline__ bool lora_work_item(const GemmArgs& p, int w, int n_clusters, int& tm, int& tn, int& half) {
    const int m_tiles = (p.M + 255) / 256;
    int t;
    if (!pair_work_item(w, m_tiles * p.n_tiles, n_clusters, p.tail_halves, t, half)) return false;
    pair_tile_coords(t, m_tiles, p.n_tiles, p.group_m, p.band_n, tm, tn);
    return true;
}

// The producer warp: the whole warp enumerates adapters, lane 0 issues.
template <int PBN, int kWidth, bool kHalves>
struct LoraProducer {
    using C = PairCfg<PBN>;
    const CUtensorMap& tmA;
    const LoraPairMaps& maps;
    const GemmArgs& p;
    uint8_t *sA, *sB;
    uint64_t *full, *empty, *rows_go;
    uint32_t* stage_info;
    volatile int* abort_flag;
    int rank, lane;
    uint64_t pol_a, pol_b;
    int it = 0;
    bool ok = true;

    // Waits for the next stage (lane 0); its index, or -1 after giving up.
    __device__ __forceinline__ int stage() {
        const int st = it % PAIR_STAGES;
        ok = ok && mbar_wait(&empty[st], (static_cast<uint32_t>(it / PAIR_STAGES) & 1u) ^ 1u, abort_flag);
        return ok ? st : -1;
    }

    // The adapters' stages of a tile.  All lanes.
    __device__ __forceinline__ void adapters(TileAdapters& present, int tn, int half) {
        const int r_chunks = (maps.R + 63) / 64;
        const int b_rows = half < 0 ? C::kBHalf : C::kBHalf / 2;
        const int b_row = tn * PBN + (half > 0 ? PBN / 2 : 0) + rank * b_rows;
        const uint32_t tile_bytes = static_cast<uint32_t>(b_rows * kWidth * 2);
        const int steps = kWidth / 16;
        const CUtensorMap* map = half < 0 ? &maps.bs : &maps.bsq;
        uint32_t a[4];
        for (int n = present.next(a, 64 / kWidth); n > 0; n = present.next(a, 64 / kWidth)) {
            for (int i = 0; lane == 0 && i < (kHalves ? 2 : 1) * r_chunks; ++i) {
                const int c = kHalves ? i / 2 : i;
                const int st = stage();
                if (st < 0) break;
                mbar_arrive(&rows_go[st]);
                const uint32_t full_leader = mapa_shared(smem_u32(&full[st]), 0);
                if (rank == 0) {
                    stage_info[st] = kStageLora | static_cast<uint32_t>((n - 1) * steps + min(steps, (maps.R - c * 64 + 15) / 16));
                    mbar_arrive_expect_tx(&full[st], 2 * static_cast<uint32_t>(n) * tile_bytes);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j < n)
                        tma_load_2d_pair(sB + st * C::kBStage + j * tile_bytes, map, c * 64,
                                         static_cast<int>(a[j]) * p.N + b_row, full_leader, pol_b);
                ++it;
            }
        }
    }

    // Stages [kb0, kb1) of the Linear (lane 0).
    __device__ __forceinline__ void linear(int kb0, int kb1, int tm, int tn, int half) {
        const int b_rows = half < 0 ? C::kBHalf : C::kBHalf / 2;
        const int b_row = tn * PBN + (half > 0 ? PBN / 2 : 0) + rank * b_rows;
        const int a_row = tm * 256 + rank * 128;
        const CUtensorMap* map = half < 0 ? &maps.b[0] : &maps.bq[0];
        for (int kb = kb0; kb < kb1; ++kb) {
            const int st = stage();
            if (st < 0) return;
            const uint32_t full_leader = mapa_shared(smem_u32(&full[st]), 0);
            if (rank == 0) {
                stage_info[st] = 0u;
                mbar_arrive_expect_tx(&full[st], 2 * static_cast<uint32_t>(C::kAStage + b_rows * BK));
            }
            tma_load_2d_pair(sA + st * C::kAStage, &tmA, kb * BK, a_row, full_leader, pol_a);
            tma_load_2d_pair(sB + st * C::kBStage, map, kb * BK, b_row, full_leader, pol_b);
            ++it;
        }
    }

    __device__ __forceinline__ void run(int cluster, int n_clusters) {
        const int total_tiles = (p.M + 255) / 256 * p.n_tiles;
        // at least one stage of the tile (the one that waits for the tile's own
        // adapters) comes before the next tile's adapters
        const int lead = min(kLoraLead, p.k_blocks - 1);
        l2_policies(p, pol_a, pol_b);
        int tm, tn, half;
        bool more = lora_work_item<PBN>(p, cluster, n_clusters, tm, tn, half);
        TileAdapters present;
        if (more) {
            present.load(maps.idx, tm, p.M, maps.n_adapters, lane);
            adapters(present, tn, half);
        }
        for (int w = cluster, round = 0; more; w += n_clusters, ++round) {
            if (rank == 0 && lane == 0) pace_round(p.round_ctr, round, total_tiles, n_clusters);
            int tm2 = 0, tn2 = 0, half2 = 0;
            more = lora_work_item<PBN>(p, w + n_clusters, n_clusters, tm2, tn2, half2);
            if (more) present.load(maps.idx, tm2, p.M, maps.n_adapters, lane);
            if (lane == 0) linear(0, p.k_blocks - lead, tm, tn, half);
            __syncwarp();
            if (more) adapters(present, tn2, half2);
            if (lane == 0) {
                linear(p.k_blocks - lead, p.k_blocks, tm, tn, half);
                if (ok && rank == 0 && p.round_ctr != nullptr) atomicAdd(p.round_ctr, 1u);
            }
            ok = __shfl_sync(0xFFFFFFFFu, ok ? 1 : 0, 0) != 0;
            if (!ok) break;
            tm = tm2;
            tn = tn2;
            half = half2;
        }
        if (lane != 0) return;
        if (!ok) give_up(abort_flag, p.err, kErrGemmProducer);
        // As in the plain producer: the even CTA's waits out every load in flight.
        if (rank == 0) {
            for (int i = max(0, it - PAIR_STAGES); i < it; ++i)
                if (!mbar_wait(&full[i % PAIR_STAGES], static_cast<uint32_t>(i / PAIR_STAGES) & 1u, nullptr))
                    atomicOr(p.err, kErrGemmDrain);
            pacing_done(p.round_ctr, n_clusters);
        }
    }
};

// The warps that write the A operand of the adapters' stages: thread i of the
// 128 has row i of this CTA's half.  The CTA's producer tells them through
// rows_go when such a stage is free (they skip the Linear's stages, so they
// could not follow the phases of "empty" themselves).
template <int PBN, int kWidth, bool kHalves>
__device__ __forceinline__ void lora_pair_rows(const LoraPairMaps& maps, const GemmArgs& p, uint8_t* sA,
                                               uint64_t* rows_go, uint64_t* rows_full,
                                               volatile int* abort_flag, int rank, int cluster, int n_clusters,
                                               int row, int lane) {
    using C = PairCfg<PBN>;
    const int r_chunks = (maps.R + 63) / 64;
    const int units = maps.R / 8;  // 16-byte units of a row of t
    const int lead = min(kLoraLead, p.k_blocks - 1);  // as the producer
    constexpr int kUnits = kWidth / 8;
    int it = 0;
    uint32_t phase = 0;  // a bit per stage
    int tm, tn, half;
    for (int w = cluster; lora_work_item<PBN>(p, w, n_clusters, tm, tn, half); w += n_clusters) {
        if (w != cluster) it += p.k_blocks - lead;  // the tile before, up to its last stages
        const int m = tm * 256 + rank * 128 + row;
        const uint32_t mine = row_adapter(maps.idx, m, p.M, maps.n_adapters);
        TileAdapters present;
        present.load(maps.idx, tm, p.M, maps.n_adapters, lane);
        const uint4* t = maps.t + static_cast<int64_t>(m) * (kHalves ? 2 : 1) * units;
        uint4 v[kUnits], low[kHalves ? kUnits : 1];
        const auto fetch = [&](int c) {
#pragma unroll
            for (int u = 0; u < kUnits; ++u) {
                const bool in = mine != 0xFFFFFFFFu && c * 8 + u < units;
                v[u] = in ? __ldg(t + c * 8 + u) : make_uint4(0u, 0u, 0u, 0u);
                if constexpr (kHalves) low[u] = in ? __ldg(t + units + c * 8 + u) : make_uint4(0u, 0u, 0u, 0u);
            }
        };
        if (r_chunks == 1) fetch(0);
        uint32_t a[4];
        // Waits for the next stage and stores `from` to it, masked; the stage, -1 after giving up.
        const auto store = [&](const uint4* from, int n) {
            const int st = it % PAIR_STAGES;
            if (!mbar_wait_warp(&rows_go[st], (phase >> st) & 1u, abort_flag)) {
                if (lane == 0) give_up(abort_flag, p.err, kErrLora);
                return -1;
            }
            phase ^= 1u << st;
            ++it;
            uint8_t* dst = sA + st * C::kAStage;
            const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
            if constexpr (kWidth == 64) {  // 128-byte swizzle
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    *reinterpret_cast<uint4*>(dst + row * 128 + ((u ^ (row & 7)) << 4)) = mine == a[0] ? from[u] : zero;
            } else if constexpr (kWidth == 32) {  // 64-byte swizzle: unit u of row r at u ^ (r / 2 % 4)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        if (i < n)
                            *reinterpret_cast<uint4*>(dst + i * 8192 + row * 64 + ((u ^ ((row >> 1) & 3)) << 4)) =
                                mine == a[i] ? from[u] : zero;
            } else {  // 32-byte swizzle: u ^ (r / 4 % 2)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int u = 0; u < 2; ++u)
                        if (i < n)
                            *reinterpret_cast<uint4*>(dst + i * 4096 + row * 32 + ((u ^ ((row >> 2) & 1)) << 4)) =
                                mine == a[i] ? from[u] : zero;
            }
            return st;
        };
        for (int n = present.next(a, 64 / kWidth); n > 0; n = present.next(a, 64 / kWidth)) {
            for (int c = 0; c < r_chunks; ++c) {
                if (r_chunks > 1) fetch(c);
                const int st = store(v, n);
                if (st < 0) return;
                int st2 = 0;
                if constexpr (kHalves) {  // one fence for both halves
                    st2 = store(low, n);
                    if (st2 < 0) return;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive_cluster_local_data(mapa_shared(smem_u32(&rows_full[st]), 0));
                    if constexpr (kHalves) mbar_arrive_cluster_local_data(mapa_shared(smem_u32(&rows_full[st2]), 0));
                }
            }
        }
        if (w != cluster) it += lead;
    }
}

// The MMA warp of the even CTA.  It follows the producer's order: the first
// tile's adapters, then for every tile its stages up to the last few, the next
// tile's adapters, the rest.  How many stages the adapters take it reads from
// shared memory, stage by stage; everything an instruction of the Linear needs
// it knows per tile.  The whole warp runs the loops and one lane issues, so
// that addresses and descriptors live in uniform registers.  (Measured on B200:
// a loop that took accumulator and shape from each stage's word ran 1.4 times
// as long.)
template <int PBN, int kWidth>
struct LoraMma {
    using C = PairCfg<PBN>;
    const GemmArgs& p;
    uint8_t *sA, *sB;
    uint64_t *full, *empty, *order, *rows_full;
    const volatile uint32_t* stage_info;
    volatile int* abort_flag;
    bool leader;
    int st = 0;               // the next stage and its phase
    uint32_t phase = 0;
    uint32_t rows_phase = 0;  // a bit per stage
    bool ok = true;

    __device__ __forceinline__ bool wait_full() {
        ok = ok && mbar_wait(&full[st], phase, abort_flag);
        return ok;
    }
    __device__ __forceinline__ void advance() {
        if (++st == PAIR_STAGES) {
            st = 0;
            phase ^= 1u;
        }
    }

    // The adapters' stages, if the next stage is one; true if there were any.
    __device__ __forceinline__ bool adapters(uint64_t* tmem_empty_bar, uint32_t empty_parity, uint32_t d_tmem, int n) {
        const uint32_t idesc = make_idesc_bf16(256, n);
        // from one adapter's tile to the next, in 16-byte units
        constexpr uint32_t kATile = 128u * kWidth * 2 / 16;
        const uint32_t b_tile = static_cast<uint32_t>(n / 2) * (kWidth * 2 / 16);
        bool any = false;
        while (wait_full()) {
            const uint32_t info = __shfl_sync(0xFFFFFFFFu, stage_info[st], 0);
            if ((info & kStageLora) == 0) break;
            ok = any || mbar_wait(tmem_empty_bar, empty_parity, abort_flag);
            ok = ok && mbar_wait_cluster(&rows_full[st], (rows_phase >> st) & 1u, abort_flag);
            if (!ok) break;
            rows_phase ^= 1u << st;
            tc_fence_after();
            const uint64_t a_desc = swizzled_kmajor_desc<kWidth * 2>(sA + st * C::kAStage);
            const uint64_t b_desc = swizzled_kmajor_desc<kWidth * 2>(sB + st * C::kBStage);
            const uint32_t steps = info & kStageSteps;
            if (leader) {
#pragma unroll
                for (uint32_t k = 0; k < 4; ++k) {
                    constexpr uint32_t kPer = kWidth / 16;  // instructions per adapter's tile, 32 bytes of a row each
                    const uint64_t in_tile = 2 * (k % kPer);
                    if (k < steps)
                        mma_bf16_pair(d_tmem, a_desc + k / kPer * kATile + in_tile,
                                      b_desc + k / kPer * b_tile + in_tile, idesc, (any || k > 0) ? 1u : 0u);
                }
                mma_commit_pair(&empty[st], 0x3);
            }
            __syncwarp();
            any = true;
            advance();
        }
        if (any && leader) mma_commit_pair(order, 0x1);
        return any;
    }

    // `count` stages of the Linear; acc0: the accumulator already holds something.
    __device__ __forceinline__ void linear(int count, uint32_t d_tmem, uint32_t idesc, bool acc0) {
        for (int i = 0; i < count; ++i) {
            if (!wait_full()) return;
            tc_fence_after();
            const uint64_t a_desc = sw128_kmajor_desc(sA + st * C::kAStage);
            const uint64_t b_desc = sw128_kmajor_desc(sB + st * C::kBStage);
            if (leader) {
#pragma unroll
                for (int k = 0; k < BK / UMMA_K; ++k)
                    mma_e4m3_pair<false>(d_tmem, a_desc + 2 * k, b_desc + 2 * k, idesc, (i > 0 || k > 0 || acc0) ? 1u : 0u);
                mma_commit_pair(&empty[st], 0x3);
            }
            __syncwarp();
            advance();
        }
    }

    __device__ __forceinline__ void run(uint64_t* tmem_full, uint64_t* tmem_empty, uint32_t tmem_base, int cluster,
                                        int n_clusters) {
        const int total_tiles = (p.M + 255) / 256 * p.n_tiles;
        const int lead = min(kLoraLead, p.k_blocks - 1);  // as the producer
        uint32_t order_phase = 0;
        int t, half;
        bool more = pair_work_item(cluster, total_tiles, n_clusters, p.tail_halves, t, half);
        // tile number c uses accumulator c & 1, for the (c >> 1)-th time
        bool after_lora = more && adapters(&tmem_empty[0], 1u, tmem_base, half < 0 ? PBN : PBN / 2);
        for (int w = cluster, c = 0; more && ok; w += n_clusters, ++c) {
            const int buf = c & 1;
            const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(buf * PBN);
            const uint32_t idesc = make_idesc<kAccF32>(256, half < 0 ? PBN : PBN / 2);
            if (after_lora) {
                ok = mbar_wait(order, order_phase, abort_flag);
                order_phase ^= 1u;
            } else {
                ok = mbar_wait(&tmem_empty[buf], (static_cast<uint32_t>(c >> 1) & 1u) ^ 1u, abort_flag);
            }
            if (!ok) break;
            tc_fence_after();
            linear(p.k_blocks - lead, d_tmem, idesc, after_lora);
            int half2 = -1;
            more = pair_work_item(w + n_clusters, total_tiles, n_clusters, p.tail_halves, t, half2);
            const bool after2 =
                more && adapters(&tmem_empty[buf ^ 1], (static_cast<uint32_t>((c + 1) >> 1) & 1u) ^ 1u,
                                 tmem_base + static_cast<uint32_t>((buf ^ 1) * PBN), half2 < 0 ? PBN : PBN / 2);
            linear(lead, d_tmem, idesc, true);
            if (ok && leader) mma_commit_pair(&tmem_full[buf], 0x3);
            half = half2;
            after_lora = after2;
        }
    }
};

// kLora: 0, or the columns of an adapter's tile (16, 32 or 64).
template <int PBN, int kAcc, int kQuant = 0, int kLora = 0, bool kHalves = false>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(pair_threads<kQuant, kLora != 0>(), 1)
    scaled_mm_pair_kernel(const __grid_constant__ CUtensorMap tmA,
                          const __grid_constant__ std::conditional_t<kLora != 0, LoraPairMaps, PairMaps> maps,
                          GemmArgs p) {
    using C = PairCfg<PBN>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sA = smem;
    uint8_t* sB = sA + PAIR_STAGES * C::kAStage;
    uint8_t* sE = sB + PAIR_STAGES * C::kBStage;
    uint64_t* full = reinterpret_cast<uint64_t*>(sE + SMEM_EPI);
    uint64_t* empty = full + PAIR_STAGES;
    uint64_t* tmem_full = empty + PAIR_STAGES;
    uint64_t* tmem_empty = tmem_full + 2;
    uint64_t* drain = tmem_empty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    // kLora only (the last 16 bytes hold the two words above)
    uint64_t* order = drain + 3;
    uint64_t* rows_full = order + 1;
    uint64_t* rows_go = rows_full + PAIR_STAGES;
    uint32_t* stage_info = reinterpret_cast<uint32_t*>(rows_go + PAIR_STAGES);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int cluster = blockIdx.x >> 1;
    const int n_clusters = gridDim.x >> 1;
    const int m_tiles = (p.M + 255) / 256;
    const int total_tiles = m_tiles * p.n_tiles;

    if (threadIdx.x == 0) {
        for (int i = 0; i < PAIR_STAGES; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tmem_full[i], 1);
            mbar_init(&tmem_empty[i], 2 * EPI_WARPS);
        }
        mbar_init(drain, 1);
        if constexpr (kLora != 0) {
            mbar_init(order, 1);
            for (int i = 0; i < PAIR_STAGES; ++i) {
                mbar_init(&rows_full[i], 2 * LORA_WARPS);
                mbar_init(&rows_go[i], 1);
            }
        }
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tensormap(&tmA);
        for (int i = 0; i < p.n_lin; ++i) {
            prefetch_tensormap(&maps.b[i]);
            if (p.tail_halves) prefetch_tensormap(&maps.bq[i]);
            prefetch_tensormap(&maps.y[i]);
        }
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, C::kTmemCols);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync_all();  // barriers of both CTAs initialised, TMEM allocated
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    pdl_allow_next();
    pdl_wait();  // the set-up above may overlap the previous kernel; global memory only from here

    if (warp == 0) {
        // ---------------------------------------------------- TMA producer
        if constexpr (kLora != 0) {
            LoraProducer<PBN, kLora, kHalves> producer = {tmA,   maps,    p,          sA,         sB, full,
                                                          empty, rows_go, stage_info, abort_flag,
                                                          static_cast<int>(rank), lane};
            producer.run(cluster, n_clusters);
        } else if (lane == 0) {
            uint64_t pol_a, pol_b;
            l2_policies(p, pol_a, pol_b);
            int it = 0;
            int issued_phase[PAIR_STAGES];
            for (int i = 0; i < PAIR_STAGES; ++i) issued_phase[i] = -1;
            bool ok = true;
            int round = 0, t, half;
            for (int w = cluster; ok && pair_work_item(w, total_tiles, n_clusters, p.tail_halves, t, half);
                 w += n_clusters, ++round) {
                if (rank == 0) pace_round(p.round_ctr, round, total_tiles, n_clusters);
                int tm, tn_all, lin, tn;
                pair_tile_coords(t, m_tiles, p.n_tiles, p.group_m, p.band_n, tm, tn_all);
                split_linear_tile(p, tn_all, lin, tn);
                // a half tile: PBN / 2 columns, PBN / 4 B rows per CTA (bq's box)
                const int b_rows = half < 0 ? C::kBHalf : C::kBHalf / 2;
                const CUtensorMap* tmb = half < 0 ? &maps.b[lin] : &maps.bq[lin];
                const uint32_t stage_tx = 2 * static_cast<uint32_t>(C::kAStage + b_rows * BK);
                const int a_row = tm * 256 + static_cast<int>(rank) * 128;
                const int b_row = tn * PBN + (half > 0 ? PBN / 2 : 0) + static_cast<int>(rank) * b_rows;
                if constexpr (kQuant != 0) {
                    if (!wait_share_quantized(p, a_row, abort_flag)) {
                        give_up(abort_flag, p.err, kErrGemmProducer);
                        ok = false;
                        break;
                    }
                }
                for (int kb = 0; kb < p.k_blocks; ++kb, ++it) {
                    const int st = it % PAIR_STAGES;
                    const uint32_t ph = static_cast<uint32_t>(it / PAIR_STAGES) & 1u;
                    if (!mbar_wait(&empty[st], ph ^ 1u, abort_flag)) {
                        give_up(abort_flag, p.err, kErrGemmProducer);
                        ok = false;
                        break;
                    }
                    const uint32_t full_leader = mapa_shared(smem_u32(&full[st]), 0);
                    if (rank == 0) mbar_arrive_expect_tx(&full[st], stage_tx);
                    tma_load_2d_pair(sA + st * C::kAStage, &tmA, kb * BK, a_row, full_leader, pol_a);
                    tma_load_2d_pair(sB + st * C::kBStage, tmb, kb * BK, b_row, full_leader, pol_b);
                    issued_phase[st] = static_cast<int>(ph);
                }
                if (ok && rank == 0 && p.round_ctr != nullptr) atomicAdd(p.round_ctr, 1u);
            }
            // The even CTA's "full" barriers count both CTAs' loads: the even
            // producer waits for everything in flight before the final
            // cluster barrier lets either CTA exit.
            if (rank == 0) {
                for (int i = 0; i < PAIR_STAGES; ++i)
                    if (issued_phase[i] >= 0 &&
                        !mbar_wait(&full[i], static_cast<uint32_t>(issued_phase[i]), nullptr))
                        atomicOr(p.err, kErrGemmDrain);
                pacing_done(p.round_ctr, n_clusters);
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------- MMA issuer (even CTA)
        if constexpr (kLora != 0) {
            if (rank == 0) {
                const bool leader = elect_one();
                LoraMma<PBN, kLora> mma = {p,     sA,        sB,         full,       empty, order,
                                           rows_full, stage_info, abort_flag, leader};
                mma.run(tmem_full, tmem_empty, tmem_base, cluster, n_clusters);
                if (leader) {
                    if (!mma.ok) give_up(abort_flag, p.err, kErrGemmMma);
                    mma_commit_pair(drain, 0x1);
                    if (!mbar_wait(drain, 0, nullptr)) atomicOr(p.err, kErrGemmDrain);
                }
            }
        } else if (lane == 0 && rank == 0) {
            int it = 0, tcount = 0, t, half;
            bool ok = true;
            for (int w = cluster; ok && pair_work_item(w, total_tiles, n_clusters, p.tail_halves, t, half);
                 w += n_clusters, ++tcount) {
                const int buf = tcount & 1;
                const uint32_t use = static_cast<uint32_t>(tcount >> 1);
                if (!mbar_wait(&tmem_empty[buf], (use & 1u) ^ 1u, abort_flag)) {
                    give_up(abort_flag, p.err, kErrGemmMma);
                    break;
                }
                tc_fence_after();
                const uint32_t idesc = make_idesc<kAcc>(256, half < 0 ? PBN : PBN / 2);
                const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(buf * PBN);
                for (int kb = 0; kb < p.k_blocks; ++kb, ++it) {
                    const int st = it % PAIR_STAGES;
                    const uint32_t ph = static_cast<uint32_t>(it / PAIR_STAGES) & 1u;
                    if (!mbar_wait(&full[st], ph, abort_flag)) {
                        give_up(abort_flag, p.err, kErrGemmMma);
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t a_desc = sw128_kmajor_desc(sA + st * C::kAStage);
                    const uint64_t b_desc = sw128_kmajor_desc(sB + st * C::kBStage);
#pragma unroll
                    for (int k = 0; k < BK / UMMA_K; ++k) {
                        const uint64_t koff = static_cast<uint64_t>((k * UMMA_K) >> 4);
                        mma_e4m3_pair<kAcc == kAccS32>(d_tmem, a_desc + koff, b_desc + koff, idesc,
                                                       (kb | k) != 0 ? 1u : 0u);
                    }
                    mma_commit_pair(&empty[st], 0x3);
                }
                if (ok) mma_commit_pair(&tmem_full[buf], 0x3);
            }
            mma_commit_pair(drain, 0x1);
            if (!mbar_wait(drain, 0, nullptr)) atomicOr(p.err, kErrGemmDrain);
        }
    } else if (warp < 2 + EPI_WARPS) {
        // ------------------------------------------- epilogue (both CTAs)
        const int ew = warp - 2;
        const int quarter = warp & 3;
        uint8_t* ebuf = sE + static_cast<size_t>(ew) * EPI_BUF_BYTES;
        float* colp = reinterpret_cast<float*>(sE + EPI_WARPS * EPI_BUF_BYTES + ew * COLP_BYTES);
        const uint32_t tmem_empty_leader0 = mapa_shared(smem_u32(&tmem_empty[0]), 0);
        const uint32_t tmem_empty_leader1 = mapa_shared(smem_u32(&tmem_empty[1]), 0);
        int tcount = 0, t, half;
        for (int w = cluster; pair_work_item(w, total_tiles, n_clusters, p.tail_halves, t, half);
             w += n_clusters, ++tcount) {
            int tm, tn_all, lin, tn;
            pair_tile_coords(t, m_tiles, p.n_tiles, p.group_m, p.band_n, tm, tn_all);
            split_linear_tile(p, tn_all, lin, tn);
            const GemmArgs pl = linear_args(p, lin);
            const int n0 = tn * PBN + (half > 0 ? PBN / 2 : 0);
            stage_col_params<PBN>(pl, colp, n0, lane);
            const int row0 = tm * 256 + static_cast<int>(rank) * 128 + quarter * 32;
            const int m = row0 + lane;
            float sa;
            if constexpr (kQuant != 0) {
                // the row scales come from this launch's quantizer warps: wait
                // for the share (it is complete before the tile's MMAs run)
                int ok = 1;
                if (lane == 0) ok = wait_share_quantized(p, row0 - quarter * 32, abort_flag) ? 1 : 0;
                if (!__shfl_sync(0xFFFFFFFFu, ok, 0)) {
                    if (lane == 0) give_up(abort_flag, p.err, kErrGemmEpilogue);
                    break;
                }
                __syncwarp();
                sa = 0.0f;
                if (m < p.M) asm volatile("ld.relaxed.gpu.global.f32 %0, [%1];" : "=f"(sa) : "l"(p.qs + m) : "memory");
            } else {
                sa = (m < p.M) ? __ldg(p.s_a + m) : 0.0f;
            }
            const int buf = tcount & 1;
            const uint32_t use = static_cast<uint32_t>(tcount >> 1);
            if (!mbar_wait_warp(&tmem_full[buf], use & 1u, abort_flag)) {
                if (lane == 0) give_up(abort_flag, p.err, kErrGemmEpilogue);
                break;
            }
            tc_fence_after();
            const uint32_t t_row = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
                                   static_cast<uint32_t>(buf * PBN);
            store_tile_rows<PBN, kAcc>(pl, maps.y[lin], t_row, ebuf, colp, n0, row0, sa, lane,
                                       half < 0 ? PBN : PBN / 2);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(buf == 0 ? tmem_empty_leader0 : tmem_empty_leader1);
        }
        if (lane == 0) bulk_wait<0>();
        __syncwarp();
    } else if constexpr (kLora != 0) {
        // ------------------------------------ row warps of the adapters
        lora_pair_rows<PBN, kLora, kHalves>(maps, p, sA, rows_go, rows_full, abort_flag, static_cast<int>(rank), cluster,
                                            n_clusters, static_cast<int>(threadIdx.x) - THREADS, lane);
    } else {
        // ------------------------------------ quantizer warps (kQuant only)
        if constexpr (kQuant != 0) quantize_rows_for_gemm<kQuant>(p, lane);
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // neither CTA leaves while the pair may still touch its shared memory
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, C::kTmemCols);
    }
}

}  // namespace

namespace {

// A wait that can only end by running out: the barrier expects one arrival
// that nothing makes.  Exercises the bounded wait the GEMM roles use (same
// helper, a shorter limit) and the error word that reports it.
__global__ void wait_selftest_kernel(uint64_t limit_ns, uint32_t* err) {
    __shared__ uint64_t bar;
    __shared__ int abort_flag;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    __syncthreads();
    if (threadIdx.x == 0 && !mbar_wait(&bar, 0, &abort_flag, limit_ns)) atomicOr(err, kErrSelfTest);
}

// Opt-in shared memory of the scaled GEMM kernels of one accumulator kind (once per device).
template <int kAcc>
tfq_status set_gemm_attributes(DeviceState* ds) {
    return once_per_device(ds->gemm_attr_set[kAcc], [] {
        cudaError_t e = cudaFuncSetAttribute(scaled_mm_kernel<kAcc>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(SMEM_BYTES));
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(scaled_mm_pair_kernel<256, kAcc>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     static_cast<int>(PairCfg<256>::kSmem));
        return e;
    });
}

// The tensor maps and the Linear table of the CTA-pair kernel for n Linears
// that share A (their N tiles concatenated in order).
tfq_status pair_linear_setup(const LinearOperands* lins, int n, int64_t M, int64_t K, PairMaps& maps,
                             GemmArgs& a) {
    constexpr int kPBN = 256;
    using C = PairCfg<kPBN>;
    int tiles = 0;
    for (int i = 0; i < n; ++i) {
        const LinearOperands& l = lins[i];
        tfq_status st = encode_tensor_map_2d(&maps.b[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, l.W, K, l.N, K, BK,
                                             C::kBHalf, CU_TENSOR_MAP_SWIZZLE_128B);
        if (st == TFQ_OK)
            st = encode_tensor_map_2d(&maps.bq[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, l.W, K, l.N, K, BK, C::kBHalf / 2,
                                      CU_TENSOR_MAP_SWIZZLE_128B);
        if (st == TFQ_OK)
            st = encode_tensor_map_2d(&maps.y[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, l.out, l.N, M, l.N * 2, EPI_COLS,
                                      32, CU_TENSOR_MAP_SWIZZLE_128B);
        if (st != TFQ_OK) return st;
        a.lin_tile0[i] = tiles;
        a.lin_s_w[i] = l.s_w;
        a.lin_bias[i] = static_cast<const uint16_t*>(l.bias);
        a.lin_N[i] = static_cast<int>(l.N);
        tiles += static_cast<int>((l.N + kPBN - 1) / kPBN);
    }
    for (int i = n; i <= kMaxLinears; ++i) a.lin_tile0[i] = tiles;
    a.n_lin = n;
    a.n_tiles = tiles;
    a.s_w = lins[0].s_w;
    a.bias = static_cast<const uint16_t*>(lins[0].bias);
    a.N = static_cast<int>(lins[0].N);
    return TFQ_OK;
}

// n Linears that share A (n = 1: the plain GEMM) as one launch of the
// CTA-pair kernel (M >= TFQ_GEMM_PAIR_MIN_M).
template <int kAcc>
tfq_status launch_pair_linears(const void* A, const float* s_a, int64_t M, int64_t K, const LinearOperands* lins,
                               int n, cudaStream_t stream, DeviceState* ds) {
    tfq_status st = set_gemm_attributes<kAcc>(ds);
    if (st != TFQ_OK) return st;
    CUtensorMap tmA;
    st = encode_tensor_map_2d(&tmA, CU_TENSOR_MAP_DATA_TYPE_UINT8, A, K, M, K, BK, BM, CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != TFQ_OK) return st;
    PairMaps maps = {};
    GemmArgs a;
    st = pair_linear_setup(lins, n, M, K, maps, a);
    if (st != TFQ_OK) return st;
    a.s_a = s_a;
    a.M = static_cast<int>(M);
    a.K = static_cast<int>(K);
    a.m_tiles = static_cast<int>((M + BM - 1) / BM);
    a.k_blocks = static_cast<int>((K + BK - 1) / BK);
    choose_raster(K, 256, a.band_n, a.group_m);
    a.err = ds->err_word;
    const int64_t pair_tiles = ((M + 255) / 256) * static_cast<int64_t>(a.n_tiles);
    if (pair_tiles > INT32_MAX) return fail(TFQ_EUNSUPPORTED, "too many output tiles");
    const int clusters = static_cast<int>(std::min<int64_t>(pair_tiles, ds->sm_count / 2));
    a.tail_halves = choose_tail_halves(pair_tiles, clusters);
    a.round_ctr = take_round_counter(ds);
    const cudaError_t el = launch_kernel(scaled_mm_pair_kernel<256, kAcc>, dim3(2 * clusters), dim3(THREADS),
                                         PairCfg<256>::kSmem, stream, tmA, maps, a);
    if (el != cudaSuccess) return fail(TFQ_ECUDA, "GEMM launch: %s", cudaGetErrorString(el));
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? TFQ_OK : fail(TFQ_ECUDA, "GEMM launch: %s", cudaGetErrorString(e));
}

template <int kAcc>
tfq_status launch_scaled_mm(const void* A, const float* s_a, const void* W, const float* s_w, const void* bias,
                            int64_t M, int64_t N, int64_t K, void* out, cudaStream_t stream, DeviceState* ds) {
    if (M == 0 || N == 0) return TFQ_OK;
    if (use_pair_kernel(M, ds->sm_count)) {
        const LinearOperands lin = {W, s_w, bias, N, out};
        return launch_pair_linears<kAcc>(A, s_a, M, K, &lin, 1, stream, ds);
    }
    CUtensorMap tmA, tmY;
    tfq_status st = encode_tensor_map_2d(&tmA, CU_TENSOR_MAP_DATA_TYPE_UINT8, A, K, M, K, BK, BM,
                                         CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != TFQ_OK) return st;
    st = encode_tensor_map_2d(&tmY, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, out, N, M, N * 2, EPI_COLS, 32,
                              CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != TFQ_OK) return st;
    st = set_gemm_attributes<kAcc>(ds);
    if (st != TFQ_OK) return st;
    GemmArgs a;
    a.s_a = s_a;
    a.s_w = s_w;
    a.bias = static_cast<const uint16_t*>(bias);
    a.M = static_cast<int>(M);
    a.N = static_cast<int>(N);
    a.K = static_cast<int>(K);
    a.m_tiles = static_cast<int>((M + BM - 1) / BM);
    a.n_tiles = static_cast<int>((N + BN - 1) / BN);
    a.k_blocks = static_cast<int>((K + BK - 1) / BK);
    choose_raster(K, BN, a.band_n, a.group_m);
    a.err = ds->err_word;
    a.round_ctr = nullptr;
    const int64_t tiles = static_cast<int64_t>(a.m_tiles) * a.n_tiles;
    if (tiles > INT32_MAX) return fail(TFQ_EUNSUPPORTED, "too many output tiles");
    CUtensorMap tmB;
    st = encode_tensor_map_2d(&tmB, CU_TENSOR_MAP_DATA_TYPE_UINT8, W, K, N, K, BK, BN, CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != TFQ_OK) return st;
    const int grid = static_cast<int>(std::min<int64_t>(tiles, ds->sm_count));
    const cudaError_t el = launch_kernel(scaled_mm_kernel<kAcc>, dim3(grid), dim3(THREADS), SMEM_BYTES, stream, tmA,
                                         tmB, tmY, a);
    if (el != cudaSuccess) return fail(TFQ_ECUDA, "GEMM launch: %s", cudaGetErrorString(el));
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? TFQ_OK : fail(TFQ_ECUDA, "GEMM launch: %s", cudaGetErrorString(e));
}

}  // namespace

tfq_status launch_wait_selftest(uint64_t limit_ns, cudaStream_t stream, DeviceState* ds) {
    wait_selftest_kernel<<<1, 32, 0, stream>>>(limit_ns, ds->err_word);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? TFQ_OK : fail(TFQ_ECUDA, "self-test launch: %s", cudaGetErrorString(e));
}

size_t quant_gemm_workspace_bytes(int64_t M) {
    const size_t words = 32 + static_cast<size_t>((M + 127) / 128);
    return (words * sizeof(unsigned) + 255) / 256 * 256;
}

tfq_status launch_quant_scaled_fp8_gemm(const void* x, int64_t M, int64_t K, float qmax, bool clamp, const void* W,
                                        const float* s_w, const void* bias, int64_t N, void* A, float* s_a,
                                        void* out, void* workspace, cudaStream_t stream, DeviceState* ds) {
    if (M == 0) return TFQ_OK;
    if (!use_pair_kernel(M, ds->sm_count) || N == 0) {
        // Below the CTA-pair size: the row quantizer, then the GEMM.
        tfq_status st = launch_quant_rows(x, M, K, qmax, false, A, s_a, stream, ds);
        if (st != TFQ_OK || N == 0) return st;
        return launch_scaled_mm<kAccF32>(A, s_a, W, s_w, bias, M, N, K, out, stream, ds);
    }
    constexpr int kPBN = 256;
    using C = PairCfg<kPBN>;
    // The row counter (word 0) and the per-share counters (from word 32)
    // start at zero.
    cudaError_t e = cudaMemsetAsync(workspace, 0, quant_gemm_workspace_bytes(M), stream);
    if (e != cudaSuccess) return fail(TFQ_ECUDA, "clearing the workspace: %s", cudaGetErrorString(e));
    CUtensorMap tmA;
    tfq_status st = encode_tensor_map_2d(&tmA, CU_TENSOR_MAP_DATA_TYPE_UINT8, A, K, M, K, BK, BM,
                                         CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != TFQ_OK) return st;
    PairMaps maps = {};
    GemmArgs a;
    const LinearOperands lin = {W, s_w, bias, N, out};
    st = pair_linear_setup(&lin, 1, M, K, maps, a);
    if (st != TFQ_OK) return st;
    auto kernel = clamp ? scaled_mm_pair_kernel<kPBN, kAccF32, 2> : scaled_mm_pair_kernel<kPBN, kAccF32, 1>;
    st = once_per_device(ds->gemm_attr_set[5], [] {
        cudaError_t e = cudaFuncSetAttribute(scaled_mm_pair_kernel<kPBN, kAccF32, 1>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(C::kSmem));
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(scaled_mm_pair_kernel<kPBN, kAccF32, 2>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(C::kSmem));
        return e;
    });
    if (st != TFQ_OK) return st;
    a.s_a = s_a;
    a.M = static_cast<int>(M);
    a.K = static_cast<int>(K);
    a.m_tiles = static_cast<int>((M + BM - 1) / BM);
    a.k_blocks = static_cast<int>((K + BK - 1) / BK);
    choose_raster(K, kPBN, a.band_n, a.group_m);
    a.err = ds->err_word;
    const int64_t pair_tiles = ((M + 255) / 256) * static_cast<int64_t>(a.n_tiles);
    if (pair_tiles > INT32_MAX) return fail(TFQ_EUNSUPPORTED, "too many output tiles");
    const int clusters = static_cast<int>(std::min<int64_t>(pair_tiles, ds->sm_count / 2));
    a.tail_halves = choose_tail_halves(pair_tiles, clusters);
    a.round_ctr = take_round_counter(ds);
    unsigned* ws = static_cast<unsigned*>(workspace);
    a.qx = static_cast<const uint4*>(x);
    a.qa = static_cast<uint8_t*>(A);
    a.qs = s_a;
    a.q_next_row = ws;
    a.q_share_rows = ws + 32;
    a.qmax = qmax;
    e = launch_kernel(kernel, dim3(2 * clusters), dim3(pair_threads<1>()), C::kSmem, stream, tmA, maps, a);
    if (e != cudaSuccess) return fail(TFQ_ECUDA, "GEMM launch: %s", cudaGetErrorString(e));
    e = cudaGetLastError();
    return e == cudaSuccess ? TFQ_OK : fail(TFQ_ECUDA, "GEMM launch: %s", cudaGetErrorString(e));
}

tfq_status launch_scaled_fp8_gemm(const void* A, const float* s_a, const void* W, const float* s_w,
                                  const void* bias, int64_t M, int64_t N, int64_t K, void* out,
                                  cudaStream_t stream, DeviceState* ds) {
    return launch_scaled_mm<kAccF32>(A, s_a, W, s_w, bias, M, N, K, out, stream, ds);
}

namespace {

template <int kAcc>
tfq_status launch_gemm_multi(const void* A, const float* s_a, int64_t M, int64_t K, int n, const void* const* W,
                             const float* const* s_w, const void* const* bias, const int64_t* N, void* const* out,
                             cudaStream_t stream, DeviceState* ds) {
    if (M == 0) return TFQ_OK;
    LinearOperands lins[kMaxLinears];
    int m = 0;
    for (int i = 0; i < n; ++i)
        if (N[i] > 0) lins[m++] = {W[i], s_w[i], bias != nullptr ? bias[i] : nullptr, N[i], out[i]};
    if (m == 0) return TFQ_OK;
    if (!use_pair_kernel(M, ds->sm_count)) {  // one-CTA kernel, one launch per Linear
        for (int i = 0; i < m; ++i) {
            const tfq_status st = launch_scaled_mm<kAcc>(A, s_a, lins[i].W, lins[i].s_w, lins[i].bias, M, lins[i].N,
                                                         K, lins[i].out, stream, ds);
            if (st != TFQ_OK) return st;
        }
        return TFQ_OK;
    }
    return launch_pair_linears<kAcc>(A, s_a, M, K, lins, m, stream, ds);
}

}  // namespace

// The Linear with the adapters' first product t [M, R], with `halves` [M, 2 R], beside it.
tfq_status launch_lora_pair_gemm(const void* A, const float* s_a, const void* W, const float* s_w, const void* bias,
                                 int64_t M, int64_t N, int64_t K, const LoraCall& l, const void* t, bool halves,
                                 void* out, cudaStream_t stream, DeviceState* ds) {
    constexpr int kPBN = 256;
    using C = PairCfg<kPBN>;
    const int width = l.R <= 16 ? 16 : l.R <= 32 ? 32 : 64;
    auto kernel = width == 64   ? scaled_mm_pair_kernel<kPBN, kAccF32, 0, 64>
                  : width == 32 ? scaled_mm_pair_kernel<kPBN, kAccF32, 0, 32>
                                : scaled_mm_pair_kernel<kPBN, kAccF32, 0, 16>;
    if (halves)
        kernel = width == 64   ? scaled_mm_pair_kernel<kPBN, kAccF32, 0, 64, true>
                 : width == 32 ? scaled_mm_pair_kernel<kPBN, kAccF32, 0, 32, true>
                               : scaled_mm_pair_kernel<kPBN, kAccF32, 0, 16, true>;
    tfq_status st = once_per_device(ds->lora_attr_set, [] {
        cudaError_t e = cudaSuccess;
        for (auto k : {scaled_mm_pair_kernel<kPBN, kAccF32, 0, 16>, scaled_mm_pair_kernel<kPBN, kAccF32, 0, 32>,
                       scaled_mm_pair_kernel<kPBN, kAccF32, 0, 64>, scaled_mm_pair_kernel<kPBN, kAccF32, 0, 16, true>,
                       scaled_mm_pair_kernel<kPBN, kAccF32, 0, 32, true>,
                       scaled_mm_pair_kernel<kPBN, kAccF32, 0, 64, true>})
            if (e == cudaSuccess)
                e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(C::kSmemLora));
        return e;
    });
    if (st != TFQ_OK) return st;
    CUtensorMap tmA;
    st = encode_tensor_map_2d(&tmA, CU_TENSOR_MAP_DATA_TYPE_UINT8, A, K, M, K, BK, BM, CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != TFQ_OK) return st;
    LoraPairMaps maps = {};
    GemmArgs a;
    const LinearOperands lin = {W, s_w, bias, N, out};
    st = pair_linear_setup(&lin, 1, M, K, maps, a);
    const auto bf16_map = [&](CUtensorMap* m, const void* base, int64_t rows, uint32_t box_rows) {
        if (st == TFQ_OK)
            st = encode_tensor_map_2d(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, l.R, rows, l.R * 2,
                                      static_cast<uint32_t>(width), box_rows,
                                      width == 64   ? CU_TENSOR_MAP_SWIZZLE_128B
                                      : width == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                    : CU_TENSOR_MAP_SWIZZLE_32B);
    };
    bf16_map(&maps.bs, l.Bs, l.n_adapters * N, C::kBHalf);
    bf16_map(&maps.bsq, l.Bs, l.n_adapters * N, C::kBHalf / 2);
    if (st != TFQ_OK) return st;
    maps.idx = l.idx;
    maps.t = static_cast<const uint4*>(t);
    maps.n_adapters = l.n_adapters;
    maps.R = l.R;
    a.s_a = s_a;
    a.M = static_cast<int>(M);
    a.K = static_cast<int>(K);
    a.m_tiles = static_cast<int>((M + BM - 1) / BM);
    a.k_blocks = static_cast<int>((K + BK - 1) / BK);
    choose_raster(K, kPBN, a.band_n, a.group_m);
    a.err = ds->err_word;
    const int64_t pair_tiles = ((M + 255) / 256) * static_cast<int64_t>(a.n_tiles);
    if (pair_tiles > INT32_MAX) return fail(TFQ_EUNSUPPORTED, "too many output tiles");
    const int clusters = static_cast<int>(std::min<int64_t>(pair_tiles, ds->sm_count / 2));
    a.tail_halves = choose_tail_halves(pair_tiles, clusters);
    a.round_ctr = take_round_counter(ds);
    cudaError_t e = launch_kernel(kernel, dim3(2 * clusters), dim3(pair_threads<0, true>()), C::kSmemLora, stream, tmA, maps, a);
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? TFQ_OK : fail(TFQ_ECUDA, "GEMM launch: %s", cudaGetErrorString(e));
}

tfq_status launch_scaled_fp8_gemm_multi(const void* A, const float* s_a, int64_t M, int64_t K, int n,
                                        const void* const* W, const float* const* s_w, const void* const* bias,
                                        const int64_t* N, void* const* out, cudaStream_t stream, DeviceState* ds) {
    return launch_gemm_multi<kAccF32>(A, s_a, M, K, n, W, s_w, bias, N, out, stream, ds);
}

tfq_status launch_scaled_int8_gemm_multi(const void* A, const float* s_a, int64_t M, int64_t K, int n,
                                         const void* const* W, const float* const* s_w, const void* const* bias,
                                         const int64_t* N, void* const* out, cudaStream_t stream, DeviceState* ds) {
    return launch_gemm_multi<kAccS32>(A, s_a, M, K, n, W, s_w, bias, N, out, stream, ds);
}

tfq_status launch_scaled_fp8_gemm_f16acc(const void* A, const float* s_a, const void* W, const float* s_w,
                                         const void* bias, int64_t M, int64_t N, int64_t K, void* out,
                                         cudaStream_t stream, DeviceState* ds) {
    return launch_scaled_mm<kAccF16>(A, s_a, W, s_w, bias, M, N, K, out, stream, ds);
}

tfq_status launch_scaled_int8_gemm(const void* A, const float* s_a, const void* W, const float* s_w,
                                   const void* bias, int64_t M, int64_t N, int64_t K, void* out,
                                   cudaStream_t stream, DeviceState* ds) {
    return launch_scaled_mm<kAccS32>(A, s_a, W, s_w, bias, M, N, K, out, stream, ds);
}

}  // namespace tfq
