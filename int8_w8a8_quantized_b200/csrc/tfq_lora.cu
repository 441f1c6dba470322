// tfq_lora.cu -- the scaled FP8 Linear with low-rank adapters of many
// requests beside it:
//   out[m,n] = s_a[m] s_w[n] sum_k A_q[m,k] W_q[n,k] + bias[n]
//              + scaling[a] sum_r (sum_k x[m,k] A[a,r,k]) B[a,n,r],   a = idx[m].
// The second factor is kept in units of the weight's scale, Bs = scaling B /
// s_w, and the first product in units of the row's, t[m,r] = sum_k x A / s_a,
// so that both sums share the factor s_a[m] s_w[n].
#include <cuda_bf16.h>

#include <algorithm>

#include "tfq_gemm_common.cuh"
#include "tfq_internal.h"
#include "tfq_ptx.cuh"
#include "tfq_quant_common.cuh"

namespace tfq {
namespace {

// Once per adapter and weight, one warp per row of R values: four adapters of rank
// 64 on 5120 channels 7 us, 64 of rank 16 40 us (half the lanes idle), 64 of rank 64
// on 13824 138 us, 1.6 TB/s.
__global__ void __launch_bounds__(256) lora_fold_kernel(const __nv_bfloat16* B, const float* scaling,
                                                        const float* s_w, int64_t n, int64_t N, int64_t R,
                                                        __nv_bfloat16* out) {
    pdl_allow_next();
    pdl_wait();
    const int64_t rows = n * N;
    // one warp per row: R consecutive values with one scale
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
    for (int64_t row = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5; row < rows; row += warps) {
        const int64_t a = row / N;
        const float f = scaling != nullptr ? scaling[a] : 1.0f;
        const float sw = s_w[row - a * N];
        for (int64_t r = threadIdx.x & 31; r < R; r += 32) {
            // Never inf or NaN: a tile of the second product multiplies the
            // rows of other adapters by zero, which must stay zero.
            const float v = __fdiv_rn(f * __bfloat162float(B[row * R + r]), sw);
            constexpr float kMax = 0x1.fep127f;  // the largest finite bf16
            out[row * R + r] = __float2bfloat16_rn(v == v ? fminf(fmaxf(v, -kMax), kMax) : kMax);
        }
    }
}

// ---------------------------------------------------------------------------
// First product, many rows (lora_shrink_kernel):
//   t[m, r] = sum_k x[m,k] A[idx[m],r,k] / s_a[m],
// rounded to bf16, an operand of the tensor cores, or up to K = kHalvesK left as
// two of them, hi = bf16(t) and lo = bf16(t - hi).  (One bf16 puts an error of half
// a step, at random, on the adapters' share of a result that is itself rounded to
// bf16, and lora_Bs' own rounding as much again.  The Linear's sum grows with
// sqrt(K), the adapters' does not: with weights of 0.02 and adapters whose factors
// are 1 / sqrt(K) and 0.3 / sqrt(R), the rms error against 64 bits was 1.60 times
// that of a 32-bit form at K = 64, 1.40 at 256, 1.28 at 512, 1.18 at 1024 and 1.04 at
// 5120; with halves it is 1.34 at 64 and less above, all of it lora_Bs' rounding.
// They cost the second product twice its stages: 20000 x 4000 x 256, five adapters
// of rank 16 in runs, 126 us against 122; K = 64, rank 8, any order 142 against 123;
// at 32760 x 5120 x 5120 four adapters of rank 64 in runs 3.5 %, 64 in any order 36 %.)
// Rows are taken in blocks of kShrinkRows.  A CTA puts its block's rows in the
// order of their adapters and cuts that into items of up to 128 rows of one
// adapter, which the block's `item_ctas` CTAs share out.  An item is a
// [128, K] x [K, Rn] product on the tensor cores (Rn = R rounded up to 16):
// its x rows come as one TMA box where they are consecutive, else row by row
// as asynchronous copies that the epilogue's warps, idle then, issue; either
// way every row of x is used once, and A read once per item (from L2).  A box is
// 128 rows, so a short item's brings along the rows behind it, from L2 mostly: items
// of under 16 rows by copies instead took 144 us for 171 (64 adapters of rank 16 in any
// order, 1777 x 5120 to 1024), but 1748 for 1583 (1000 of rank 64, 9472 rows).  (Measured
// on B200, 12 adapters of rank 64 in any order, 9472 x 5120: streaming a
// tile's x once for two adapters at a time and keeping each row's own product
// 242 us, TMA gathers of four rows 116 us (some 56 cycles each), rows through
// the warps' registers 85 us, asynchronous copies 64 us; with the fence between
// copies and tensor cores behind each step's copies, where it waits for all of
// them, instead of in front of the step's MMAs 163 us.)  Bound
// by HBM: 2 R flops per value of x are far below the tensor cores' ratio; they
// are used because plain FMAs would not keep up.
// (One adapter per run of rows, rank 64: 32760 x 5120 43 us, 7.7 TB/s; 9472 x
// 5120 29 us, of which the start, the ordering and the joins take some 8.)
// Few rows split K over a cluster of S CTAs, whose partial sums meet in
// shared memory and are added in rank order (the same bits every time).
// Roles as in the GEMM: warp 0 TMA producer, warp 1 MMA, warps 2..5 epilogue.
constexpr int kShrinkThreads = 192;
constexpr int kShrinkMaxStages = 8;
constexpr int kShrinkXStage = 128 * 128;  // 128 rows x 64 bf16
constexpr int kShrinkRows = 512;
constexpr int kShrinkTable = 1024;  // up to so many adapters the rows are counted, more are ranked by comparison
constexpr uint32_t kNoAdapter = 0xFFFFFFFFu / kShrinkRows;  // a key's adapter where the row has none

struct ShrinkArgs {
    int M, R, Rn, n_adapters;
    int stages, k_blocks, splits, item_ctas;
    int K;
    const __nv_bfloat16* x;
    const int32_t* idx;
    const float* s_a;
    __nv_bfloat16* t;  // [M, R]; kHalves: [M, 2 R]
    uint32_t* err;
};

// Shared memory behind the stages and, with splits > 1, the partial sums.
struct ShrinkTail {
    uint64_t full[kShrinkMaxStages], empty[kShrinkMaxStages];
    uint64_t x_full[kShrinkMaxStages];  // x rows copied one by one
    uint64_t tmem_full, tmem_empty, drain;
    uint32_t tmem_slot;
    int abort_flag;
    int segments;
    alignas(16) uint32_t key[kShrinkRows];  // adapter * kShrinkRows + row in the block
    uint32_t order[kShrinkRows];            // the keys of rows with an adapter, in increasing order
    int16_t segment[kShrinkRows + 1];       // where each adapter's rows begin in that order, and the end
    int16_t count[kShrinkTable];            // rows per adapter, then where they begin
};

__host__ __device__ constexpr int shrink_stage_bytes(int rn) { return kShrinkXStage + rn * 128; }

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// Stores N (4 or 8) bf16 values as one access.
template <int N>
__device__ __forceinline__ void store_bf16(__nv_bfloat16* to, const float (&f)[N]) {
    if constexpr (N == 8)
        *reinterpret_cast<uint4*>(to) =
            make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
    else
        *reinterpret_cast<uint2*>(to) = make_uint2(pack2(f[0], f[1]), pack2(f[2], f[3]));
}

// t of N columns from `col` on of row m: the sums f over s_a.
template <bool kHalves, int N>
__device__ __forceinline__ void store_t(const ShrinkArgs& p, int m, int col, float (&f)[N], float sa) {
#pragma unroll
    for (int j = 0; j < N; ++j) f[j] = __fdiv_rn(f[j], sa);
    __nv_bfloat16* t = p.t + static_cast<int64_t>(m) * (kHalves ? 2 * p.R : p.R) + col;
    store_bf16(t, f);
    if constexpr (kHalves) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            f[j] -= __bfloat162float(__float2bfloat16_rn(f[j]));
            if (!isfinite(f[j])) f[j] = 0.0f;  // of an infinity or NaN the lower half is 0
        }
        store_bf16(t + p.R, f);
    }
}

// The items of a block that are this CTA's: next() is false past the last.
struct ShrinkItems {
    const ShrinkTail& s;
    int first, step;       // this CTA's items: first, first + step, ...
    int segment = 0, at = 0, item = 0;
    int start = 0, len = 0;  // of the present item, in the order

    __device__ __forceinline__ bool next() {
        for (; segment < s.segments; ++segment, at = 0) {
            const int begin = s.segment[segment], end = s.segment[segment + 1];
            for (; begin + at < end; ++item) {
                start = begin + at;
                len = min(128, end - start);
                at += 128;
                if (item % step == first) {
                    ++item;
                    return true;
                }
            }
        }
        return false;
    }
    __device__ __forceinline__ uint32_t adapter() const { return s.order[start] / kShrinkRows; }
    __device__ __forceinline__ int row(int i) const { return static_cast<int>(s.order[start + i] % kShrinkRows); }
    __device__ __forceinline__ bool box() const { return row(len - 1) - row(0) == len - 1; }  // consecutive rows
};

// Fills order, segment and segments from key (all threads; count zeroed).
// in_order: every key is below the next one or its row has no adapter, which
// all batches in the adapters' order meet (requests one after the other, the
// usual case).  Warp 0 then compares each row with the last one before it that
// has an adapter, so that rows without one in between, wherever they stand, do
// not cut an adapter's rows apart; if the adapters turn out to decrease
// somewhere, the rows are counted or ranked as any others.
__device__ __forceinline__ void order_rows(ShrinkTail& s, int n_adapters, bool in_order) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t before = (1u << lane) - 1u;
    if (in_order) {
        bool decreases = false;
        if (warp == 0) {
            int begin = 0, n = 0;
            uint32_t last = kNoAdapter;  // the adapter of the last row that has one
#pragma unroll
            for (int c = 0; c < kShrinkRows / 32; ++c) {
                const uint32_t key = s.key[c * 32 + lane], a = key / kShrinkRows;
                const uint32_t has = __ballot_sync(0xFFFFFFFFu, a != kNoAdapter);
                const uint32_t earlier = __shfl_sync(0xFFFFFFFFu, a, 31 - __clz(static_cast<int>(has & before | 1u)));
                const uint32_t prev = (has & before) != 0 ? earlier : last;
                const uint32_t begins = __ballot_sync(0xFFFFFFFFu, a != kNoAdapter && a != prev);
                decreases = decreases || (a != kNoAdapter && prev != kNoAdapter && a < prev);
                const int at = begin + __popc(has & before);
                if (a != kNoAdapter) s.order[at] = key;
                if ((begins >> lane & 1u) != 0) s.segment[n + __popc(begins & before)] = static_cast<int16_t>(at);
                begin += __popc(has);
                n += __popc(begins);
                const uint32_t final = __shfl_sync(0xFFFFFFFFu, a, 31 - __clz(static_cast<int>(has | 1u)));
                if (has != 0) last = final;
            }
            if (lane == 0) {
                s.segment[n] = static_cast<int16_t>(begin);
                s.segments = n;
            }
        }
        if (!__syncthreads_or(decreases)) return;
    }
    if (n_adapters <= kShrinkTable) {
        if (warp != 0) return;
        uint32_t key[kShrinkRows / 32];
        int place[kShrinkRows / 32];  // among the rows of its adapter
#pragma unroll
        for (int c = 0; c < kShrinkRows / 32; ++c) {
            key[c] = s.key[c * 32 + lane];
            const uint32_t a = key[c] / kShrinkRows;
            const uint32_t same = __match_any_sync(0xFFFFFFFFu, a);
            const int done = a != kNoAdapter ? s.count[a] : 0;
            place[c] = done + __popc(same & before);
            __syncwarp();
            if (a != kNoAdapter && (same & before) == 0) s.count[a] = static_cast<int16_t>(done + __popc(same));
            __syncwarp();
        }
        int begin = 0, n = 0;  // rows and segments so far
        for (int e0 = 0; e0 < n_adapters; e0 += 32) {
            const int mine = s.count[e0 + lane];
            int sum = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
                if (lane >= o) sum += v;
            }
            const uint32_t used = __ballot_sync(0xFFFFFFFFu, mine > 0);
            s.count[e0 + lane] = static_cast<int16_t>(begin + sum - mine);
            if (mine > 0) s.segment[n + __popc(used & before)] = static_cast<int16_t>(begin + sum - mine);
            n += __popc(used);
            begin += __shfl_sync(0xFFFFFFFFu, sum, 31);
        }
        if (lane == 0) {
            s.segment[n] = static_cast<int16_t>(begin);
            s.segments = n;
        }
        __syncwarp();
#pragma unroll
        for (int c = 0; c < kShrinkRows / 32; ++c) {
            const uint32_t a = key[c] / kShrinkRows;
            if (a != kNoAdapter) s.order[s.count[a] + place[c]] = key[c];
        }
        return;
    }
    for (int i = threadIdx.x; i < kShrinkRows; i += kShrinkThreads) {
        const uint32_t key = s.key[i];
        int rank = 0;
#pragma unroll 4
        for (int j = 0; j < kShrinkRows / 4; ++j) {
            const uint4 k = reinterpret_cast<const uint4*>(s.key)[j];
            rank += (k.x < key) + (k.y < key) + (k.z < key) + (k.w < key);
        }
        s.order[rank] = key;
    }
    __syncthreads();
    if (warp != 0) return;
    int n = 0;
    for (int i0 = 0; i0 < kShrinkRows; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t a = s.order[i] / kShrinkRows;
        const bool begins = i == 0 || s.order[i - 1] / kShrinkRows != a;
        const uint32_t mask = __ballot_sync(0xFFFFFFFFu, begins);
        if (begins) s.segment[n + __popc(mask & before)] = static_cast<int16_t>(i);
        n += __popc(mask);
    }
    if (lane == 0) {
        s.segment[n] = kShrinkRows;
        // the last segment may be the rows without an adapter
        s.segments = s.order[kShrinkRows - 1] / kShrinkRows == kNoAdapter ? n - 1 : n;
    }
}

// The x rows of an item that are not consecutive, by the epilogue's 128 threads:
// eight threads a row, 16 rows at a time, as asynchronous copies on whose
// completion the stage's x_full counts.  The threads only issue: nothing waits
// for the data but the MMA thread, which also makes it visible to the tensor
// cores.  False after giving up.
__device__ __forceinline__ bool x_rows(ShrinkTail& s, const ShrinkArgs& p, uint8_t* smem, const ShrinkItems& item,
                                       int row0, int kb0, int kb1, int& it) {
    const int chunk = threadIdx.x & 7, sub = (threadIdx.x - 64) >> 3;
    const int stage_bytes = shrink_stage_bytes(p.Rn);
    const __nv_bfloat16* src[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int r = sub + 16 * j;
        src[j] = r < item.len ? p.x + static_cast<int64_t>(row0 + item.row(r)) * p.K + chunk * 8 : nullptr;
    }
    // 128-byte swizzle; rows 16 apart have the same unit
    const uint32_t dst0 = smem_u32(smem) + static_cast<uint32_t>(sub * 128 + ((chunk ^ (sub & 7)) << 4));
    for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const int st = it % p.stages;
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(&s.empty[st], (static_cast<uint32_t>(it / p.stages) & 1u) ^ 1u, &s.abort_flag)))
            return false;
        const bool in = kb * 64 + chunk * 8 < p.K;  // zeros past the row's end
        const uint32_t dst = dst0 + static_cast<uint32_t>(st * stage_bytes);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (src[j] != nullptr) cp_async_16(dst + j * 2048, in ? src[j] + kb * 64 : src[j], in ? 16u : 0u);
        cp_async_arrive(&s.x_full[st]);
    }
    return true;
}

// Adds the S CTAs' partial sums of this CTA's share of the item's rows, in rank
// order, and writes them to t (the epilogue's 128 threads; several remote loads
// of each in flight).
template <int S, bool kHalves>
__device__ __forceinline__ void join_parts(const ShrinkArgs& p, const float* part, const ShrinkItems& item, int row0,
                                           int rank) {
    constexpr int kShare = 128 / S, kBatch = S == 2 ? 4 : 1;
    const int units = p.R / 4;
    const int rows = min(kShare, item.len - rank * kShare);
    const int n = rows * units;  // 16-byte units of this share, negative or 0: none
    uint32_t base[S];
#pragma unroll
    for (int q = 0; q < S; ++q) base[q] = mapa_shared(smem_u32(part), q);
    for (int e0 = threadIdx.x - 64; e0 < n; e0 += 128 * kBatch) {
        float4 v[kBatch][S];
        float sa[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int e = e0 + 128 * b, i = rank * kShare + e / units, u = e % units;
            if (e >= n) break;
            sa[b] = __ldg(p.s_a + row0 + item.row(i));
#pragma unroll
            for (int q = 0; q < S; ++q) v[b][q] = ld_cluster_v4(base[q] + (i * (p.R + 4) + 4 * u) * 4);
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int e = e0 + 128 * b, i = rank * kShare + e / units, u = e % units;
            if (e >= n) break;
            float4 s = v[b][0];
#pragma unroll
            for (int q = 1; q < S; ++q) s = make_float4(s.x + v[b][q].x, s.y + v[b][q].y, s.z + v[b][q].z, s.w + v[b][q].w);
            float f[4] = {s.x, s.y, s.z, s.w};
            store_t<kHalves>(p, row0 + item.row(i), 4 * u, f, sa[b]);
        }
    }
}

template <bool kHalves>
__global__ void __launch_bounds__(kShrinkThreads, 3)
    lora_shrink_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmA,
                       const ShrinkArgs p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int stage_bytes = shrink_stage_bytes(p.Rn);
    // splits > 1: an item's partial sums [128][R + 4] (padded so that a warp's
    // rows spread over the banks), in the stages' memory once they are consumed
    float* part = reinterpret_cast<float*>(smem);
    ShrinkTail* s = reinterpret_cast<ShrinkTail*>(smem + p.stages * stage_bytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = p.splits > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int unit = blockIdx.x / p.splits;
    const int block = unit / p.item_ctas;
    const int row0 = block * kShrinkRows;
    const int rows = min(kShrinkRows, p.M - row0);
    uint32_t tmem_cols = 32;
    while (static_cast<int>(tmem_cols) < p.Rn) tmem_cols *= 2;

    if (threadIdx.x == 0) {
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(&s->full[i], 1);
            mbar_init(&s->empty[i], 1);
            mbar_init(&s->x_full[i], 128);
        }
        mbar_init(&s->tmem_full, 1);
        mbar_init(&s->tmem_empty, 4);
        mbar_init(&s->drain, 1);
        s->abort_flag = 0;
        fence_mbar_init();
        prefetch_tensormap(&tmX);
        prefetch_tensormap(&tmA);
    }
    if (warp == 1) {
        tmem_alloc(&s->tmem_slot, tmem_cols);
        tmem_relinquish();
    }
    pdl_allow_next();
    pdl_wait();
    // Keys; rows past the end and rows without an adapter sort behind all others.
    for (int i = threadIdx.x; i < kShrinkRows; i += kShrinkThreads) {
        const uint32_t a = i < rows ? static_cast<uint32_t>(__ldg(p.idx + row0 + i)) : 0xFFFFFFFFu;
        s->key[i] = (a < static_cast<uint32_t>(p.n_adapters) ? a : kNoAdapter) * kShrinkRows + i;
    }
    for (int i = threadIdx.x; i < kShrinkTable; i += kShrinkThreads) s->count[i] = 0;
    __syncthreads();
    bool in_order = true;  // a row without an adapter may stand anywhere between two runs
    for (int i = threadIdx.x; i < kShrinkRows - 1; i += kShrinkThreads)
        in_order = in_order && (s->key[i] < s->key[i + 1] || s->key[i] / kShrinkRows == kNoAdapter);
    in_order = __syncthreads_and(in_order);
    order_rows(*s, p.n_adapters, in_order);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = s->tmem_slot;
    volatile int* abort_flag = &s->abort_flag;
    const int kb0 = static_cast<int>(static_cast<int64_t>(p.k_blocks) * rank / p.splits);
    const int kb1 = static_cast<int>(static_cast<int64_t>(p.k_blocks) * (rank + 1) / p.splits);

    int it = 0;
    bool ok = true;
    uint32_t turn = 0;  // items done by this CTA
    uint32_t x_phase = 0;  // a bit per stage
    ShrinkItems item = {*s, unit - block * p.item_ctas, p.item_ctas};
    for (; item.next(); ++turn) {
        if (warp == 0) {
            if (lane == 0) {
                const int a_row = static_cast<int>(item.adapter()) * p.R;
                const int first = row0 + item.row(0);
                const bool box = item.box();
                const uint32_t tx = static_cast<uint32_t>((box ? kShrinkXStage : 0) + p.Rn * 128);
                for (int kb = kb0; ok && kb < kb1; ++kb, ++it) {
                    const int st = it % p.stages;
                    ok = mbar_wait(&s->empty[st], (static_cast<uint32_t>(it / p.stages) & 1u) ^ 1u, abort_flag);
                    if (!ok) break;
                    uint8_t* sx = smem + st * stage_bytes;
                    mbar_arrive_expect_tx(&s->full[st], tx);
                    if (box) tma_load_2d(sx, &tmX, kb * 64, first, &s->full[st]);
                    tma_load_2d(sx + kShrinkXStage, &tmA, kb * 64, a_row, &s->full[st]);
                }
            }
            if (!ok && lane == 0) {
                *abort_flag = 1;
                atomicOr(p.err, kErrLora);
            }
        } else if (warp == 1) {
            if (lane == 0) {
                if (ok) ok = mbar_wait(&s->tmem_empty, (turn & 1u) ^ 1u, abort_flag);
                tc_fence_after();
                const uint32_t idesc = make_idesc_bf16(128, p.Rn);
                const bool box = item.box();
                for (int kb = kb0; ok && kb < kb1; ++kb, ++it) {
                    const int st = it % p.stages;
                    ok = mbar_wait(&s->full[st], static_cast<uint32_t>(it / p.stages) & 1u, abort_flag);
                    if (ok && !box) {
                        ok = mbar_wait(&s->x_full[st], (x_phase >> st) & 1u, abort_flag);
                        x_phase ^= 1u << st;
                        fence_proxy_async_smem();
                    }
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t a_desc = sw128_kmajor_desc(smem + st * stage_bytes);
                    const uint64_t b_desc = sw128_kmajor_desc(smem + st * stage_bytes + kShrinkXStage);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_bf16(tmem_base, a_desc + 2 * k, b_desc + 2 * k, idesc, (kb > kb0 || k > 0) ? 1u : 0u);
                    mma_commit(&s->empty[st]);
                }
                if (ok) {
                    mma_commit(&s->tmem_full);
                } else {
                    *abort_flag = 1;
                    atomicOr(p.err, kErrLora);
                }
            }
        } else {
            const int quarter = warp & 3;
            const int i = quarter * 32 + lane;
            const bool mine = i < item.len;
            const int m = row0 + (mine ? item.row(i) : 0);
            if (item.box() || !ok) {
                it += kb1 - kb0;
            } else {
                ok = x_rows(*s, p, smem, item, row0, kb0, kb1, it);
            }
            if (ok) ok = mbar_wait_warp(&s->tmem_full, turn & 1u, abort_flag);
            if (ok) {
                tc_fence_after();
                const float sa = mine ? __ldg(p.s_a + m) : 1.0f;
                for (int c = 0; quarter * 32 < item.len && c < p.R; c += 16) {
                    uint32_t acc[16];
                    __syncwarp();
                    tmem_ld_32x32b_x16(tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(c), acc);
                    tmem_ld_wait();
                    if (!mine) continue;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {  // R % 8 == 0
                        if (c + 8 * h >= p.R) continue;
                        float f[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(acc[8 * h + j]);
                        if (p.splits > 1) {
                            float4* dst = reinterpret_cast<float4*>(part + i * (p.R + 4) + c + 8 * h);
                            dst[0] = make_float4(f[0], f[1], f[2], f[3]);
                            dst[1] = make_float4(f[4], f[5], f[6], f[7]);
                        } else {
                            store_t<kHalves>(p, m, c + 8 * h, f, sa);
                        }
                    }
                }
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&s->tmem_empty);
        }
        if (p.splits > 1) {
            // every CTA's partial sums are in its shared memory: CTA `rank` adds up its share of the rows
            fence_proxy_async_smem();  // the next item's copies write there
            __syncwarp();
            cluster_sync_all();
            if (warp >= 2) {
                if (p.splits == 2) join_parts<2, kHalves>(p, part, item, row0, rank);
                else if (p.splits == 4) join_parts<4, kHalves>(p, part, item, row0, rank);
                else join_parts<8, kHalves>(p, part, item, row0, rank);
            }
            __syncwarp();
            cluster_sync_after_reads();  // nobody overwrites or leaves what another still reads
        }
    }
    if (warp == 0 && lane == 0) {  // loads in flight must land before the CTA leaves
        for (int i = max(0, it - p.stages); i < it; ++i)
            if (!mbar_wait(&s->full[i % p.stages], static_cast<uint32_t>(i / p.stages) & 1u, nullptr))
                atomicOr(p.err, kErrGemmDrain);
    } else if (warp == 1 && lane == 0) {
        mma_commit(&s->drain);
        if (!mbar_wait(&s->drain, 0, nullptr)) atomicOr(p.err, kErrGemmDrain);
    } else if (warp >= 2) {
        cp_async_wait_all();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem_base, tmem_cols);
    }
}

// ---------------------------------------------------------------------------
// Few rows (M <= kSmallM: a decoding step).  Everything is read once and
// little is computed, so both kernels are built to have many loads in flight:
//
// lora_rows_kernel: t[m, r] = sum_k x[m,k] A[idx[m],r,k] / s_a[m] (fp32), four
// rows' dot products with their r-th factors per `dot_warps` warps.
//
// small_lora_kernel: the Linear with the weight as the tensor cores' M operand
// (128 output channels per CTA) and the rows as N (rounded up to 16), so that a
// tile is 128 channels wide however few rows there are, and K split over a
// cluster: N / 128 tiles times the split reach all SMs.  While the weight
// streams, the epilogue's eight warps add up the adapters' second product on
// plain FMAs: a warp has 32 channels and reads their Bs[a, n, :] once per
// row.  The partial sums of the cluster meet in shared memory; CTA
// `rank` finishes its share of the rows.  Bound by latency: launch, first
// loads and joins (measured on B200, 5120 x 5120: both kernels 17.5 us for 64
// rows of 64 adapters of rank 16, 49 MB or 2.8 TB/s, and 11 us for one row of
// rank 32; the plain Linear takes 16.6 us).
constexpr int kSmallM = 128;
constexpr int kSmallThreads = 64 + 256;
constexpr int kSmallMaxStages = 6;

// fp32 += the products of two 16-byte units of bf16.
__device__ __forceinline__ float dot8(uint4 a, uint4 b, float s) {
    const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        s = fmaf(bf16_lo(x[i]), bf16_lo(y[i]), s);
        s = fmaf(bf16_hi(x[i]), bf16_hi(y[i]), s);
    }
    return s;
}

__global__ void __launch_bounds__(256) lora_rows_kernel(const uint4* x, const uint4* A, const int32_t* idx,
                                                        const float* s_a, int M, int n_adapters, int R, int units,
                                                        int dot_warps, float* t) {
    constexpr int kRows = 4;
    __shared__ float sums[8][kRows];
    // The wait comes first: a kernel that starts after every CTA here has allowed
    // it knows that all earlier kernels of the stream are complete.
    pdl_wait();
    pdl_allow_next();
    const int dots = 8 / dot_warps;  // per CTA; divides R
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per_rows = R / dots;
    const int m0 = static_cast<int>(blockIdx.x) / per_rows * kRows;
    const int r = static_cast<int>(blockIdx.x) % per_rows * dots + warp / dot_warps;
    const uint4* xr[kRows];
    const uint4* ar[kRows];  // null: no row, or none with an adapter
    bool same = true;
    uint32_t first = 0xFFFFFFFFu;
#pragma unroll
    for (int q = 0; q < kRows; ++q) {
        const int m = m0 + q;
        const uint32_t a = m < M ? static_cast<uint32_t>(__ldg(idx + m)) : 0xFFFFFFFFu;
        const bool has = a < static_cast<uint32_t>(n_adapters);
        xr[q] = x + static_cast<int64_t>(m) * units;
        ar[q] = has ? A + (static_cast<int64_t>(a) * R + r) * units : nullptr;
        if (has) {
            if (first == 0xFFFFFFFFu) first = a;
            same = same && a == first;
        }
    }
    if (first == 0xFFFFFFFFu) return;  // the whole CTA has these rows
    const int step = 32 * dot_warps;
    const int begin = (warp % dot_warps) * 32 + lane;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    float s[kRows] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (same) {  // the factor is read once for all rows
        const uint4* shared_a = A + (static_cast<int64_t>(first) * R + r) * units;
#pragma unroll 1
        for (int base = begin; base < units; base += 3 * step) {
            uint4 av[3], xv[kRows][3];
#pragma unroll
            for (int j = 0; j < 3; ++j) {
                const int u = base + j * step;
                av[j] = u < units ? ldg_nc_v4(shared_a + u) : zero;
#pragma unroll
                for (int q = 0; q < kRows; ++q) xv[q][j] = u < units && ar[q] != nullptr ? __ldg(xr[q] + u) : zero;
            }
#pragma unroll
            for (int j = 0; j < 3; ++j)
#pragma unroll
                for (int q = 0; q < kRows; ++q) s[q] = dot8(xv[q][j], av[j], s[q]);
        }
    } else {
#pragma unroll 1
        for (int base = begin; base < units; base += 2 * step) {
            uint4 av[kRows][2], xv[kRows][2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int u = base + j * step;
#pragma unroll
                for (int q = 0; q < kRows; ++q) {
                    const bool in = u < units && ar[q] != nullptr;
                    av[q][j] = in ? ldg_nc_v4(ar[q] + u) : zero;
                    xv[q][j] = in ? __ldg(xr[q] + u) : zero;
                }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int q = 0; q < kRows; ++q) s[q] = dot8(xv[q][j], av[q][j], s[q]);
        }
    }
#pragma unroll
    for (int q = 0; q < kRows; ++q)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s[q] += __shfl_xor_sync(0xFFFFFFFFu, s[q], o);
    if (dot_warps > 1) {
        if (lane == 0)
#pragma unroll
            for (int q = 0; q < kRows; ++q) sums[warp][q] = s[q];
        __syncthreads();
        if (warp % dot_warps != 0) return;
        for (int i = 1; i < dot_warps; ++i)
#pragma unroll
            for (int q = 0; q < kRows; ++q) s[q] += sums[warp + i][q];
    }
    if (lane == 0) {
#pragma unroll
        for (int q = 0; q < kRows; ++q)
            if (ar[q] != nullptr) t[static_cast<int64_t>(m0 + q) * R + r] = __fdiv_rn(s[q], __ldg(s_a + m0 + q));
    }
}

struct SmallArgs {
    int M, Mn, N, k_blocks, splits, stages, share;  // share: rows per CTA of a cluster
    int n_adapters, R;
    const int32_t* idx;
    const float* t;  // [M, R]
    const uint4* Bs;
    const float* s_a;
    const float* s_w;
    const __nv_bfloat16* bias;
    __nv_bfloat16* out;
    uint32_t* err;
};

struct SmallTail {
    uint64_t full[kSmallMaxStages], empty[kSmallMaxStages];
    uint64_t tmem_full;
    uint32_t tmem_slot;
    int abort_flag;
    alignas(16) float t[2][4][TFQ_LORA_MAX_RANK];  // four rows' first product, for each half of the epilogue
};

// The adapters' second product of up to four rows mb .. and a warp's 32 channels
// from n_base: out[row * 128 + channel] = sum_r t[row][r] Bs[idx[mb + row], channel, r].
// L neighbouring lanes share a channel's row of Bs, a 16-byte unit each, so that
// the loads are consecutive (with a channel per lane they touched a line each,
// and rank 64 took 7 us more than rank 16 on 16 x 5120 x 5120); a lane meets 32
// channels in L passes, and the lanes' sums are joined by exchanging halves,
// after which lane l holds one channel.
template <int L>
__device__ __forceinline__ void small_expand(const SmallArgs& p, const float (*t)[TFQ_LORA_MAX_RANK], int mb, int m1,
                                             int n_base, int units, float* out) {
    constexpr int kAtOnce = L == 1 ? 4 : 8 / L;  // rows in flight: up to 8 loads
    const int lane = threadIdx.x & 31, c = lane % L, group = lane / L;
#pragma unroll
    for (int j0 = 0; j0 < 4; j0 += kAtOnce) {
        if (mb + j0 >= m1) break;
        int64_t row[kAtOnce];  // the adapter's first row of Bs, -1: none
        float acc[kAtOnce][L];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const uint32_t a = mb + j0 + j < m1 ? static_cast<uint32_t>(__ldg(p.idx + mb + j0 + j)) : 0xFFFFFFFFu;
            row[j] = a < static_cast<uint32_t>(p.n_adapters) ? static_cast<int64_t>(a) * p.N : -1;
#pragma unroll
            for (int i = 0; i < L; ++i) acc[j][i] = 0.0f;
        }
        for (int u = c; u < (units + L - 1) / L * L; u += L) {
            uint4 v[kAtOnce][L];
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j)
#pragma unroll
                for (int i = 0; i < L; ++i) {
                    const int n = n_base + i * (32 / L) + group;
                    v[j][i] = row[j] >= 0 && u < units && n < p.N ? __ldg(p.Bs + (row[j] + n) * units + u)
                                                                  : make_uint4(0u, 0u, 0u, 0u);
                }
            if (u >= units) continue;
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                if (row[j] < 0) continue;  // t was not written
                const float4 lo = reinterpret_cast<const float4*>(t[j0 + j])[2 * u];
                const float4 hi = reinterpret_cast<const float4*>(t[j0 + j])[2 * u + 1];
#pragma unroll
                for (int i = 0; i < L; ++i) {
                    acc[j][i] = fmaf(bf16_lo(v[j][i].x), lo.x, acc[j][i]);
                    acc[j][i] = fmaf(bf16_hi(v[j][i].x), lo.y, acc[j][i]);
                    acc[j][i] = fmaf(bf16_lo(v[j][i].y), lo.z, acc[j][i]);
                    acc[j][i] = fmaf(bf16_hi(v[j][i].y), lo.w, acc[j][i]);
                    acc[j][i] = fmaf(bf16_lo(v[j][i].z), hi.x, acc[j][i]);
                    acc[j][i] = fmaf(bf16_hi(v[j][i].z), hi.y, acc[j][i]);
                    acc[j][i] = fmaf(bf16_lo(v[j][i].w), hi.z, acc[j][i]);
                    acc[j][i] = fmaf(bf16_hi(v[j][i].w), hi.w, acc[j][i]);
                }
            }
        }
        __syncwarp();
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
#pragma unroll
            for (int o = L / 2; o > 0; o >>= 1) {  // keep the passes with bit o as in c, give the others away
#pragma unroll
                for (int i = 0; i < o; ++i) {
                    const float keep = (c & o) != 0 ? acc[j][i + o] : acc[j][i];
                    const float give = (c & o) != 0 ? acc[j][i] : acc[j][i + o];
                    acc[j][i] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, o);
                }
            }
            if (mb + j0 + j < m1) out[(j0 + j) * 128 + c * (32 / L) + group] = acc[j][0];
        }
    }
}

__host__ __device__ constexpr int small_stage_bytes(int mn) { return (128 + mn) * BK; }

__global__ void __launch_bounds__(kSmallThreads, 2)  // all CTAs of a small grid resident
    small_lora_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                      const SmallArgs p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int stage_bytes = small_stage_bytes(p.Mn);
    float* part = reinterpret_cast<float*>(smem);  // [Mn][128]: the ring's memory, once every stage is consumed
    float* lora = reinterpret_cast<float*>(smem + p.stages * stage_bytes);  // [share][128]
    SmallTail* s = reinterpret_cast<SmallTail*>(lora + p.share * 128);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = p.splits > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int n0 = static_cast<int>(blockIdx.x) / p.splits * 128;
    const uint32_t tmem_cols = p.Mn <= 32 ? 32 : p.Mn <= 64 ? 64 : 128;
    if (threadIdx.x == 0) {
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(&s->full[i], 1);
            mbar_init(&s->empty[i], 1);
        }
        mbar_init(&s->tmem_full, 1);
        s->abort_flag = 0;
        fence_mbar_init();
        prefetch_tensormap(&tmW);
        prefetch_tensormap(&tmX);
    }
    if (warp == 1) {
        tmem_alloc(&s->tmem_slot, tmem_cols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = s->tmem_slot;
    volatile int* abort_flag = &s->abort_flag;
    const int kb0 = static_cast<int>(static_cast<int64_t>(p.k_blocks) * rank / p.splits);
    const int kb1 = static_cast<int>(static_cast<int64_t>(p.k_blocks) * (rank + 1) / p.splits);
    bool ok = true;
    pdl_allow_next();
    if (warp == 0) {
        // The codes and scales are complete before this kernel can start (the
        // kernel in front of it, lora_rows_kernel, waits for its predecessors
        // and only then lets this one start): the loads need no wait, and the
        // weight streams while that kernel still runs.
        if (lane == 0) {
            int issued = 0;
            for (int kb = kb0; ok && kb < kb1; ++kb, ++issued) {
                const int it = kb - kb0, st = it % p.stages;
                ok = mbar_wait(&s->empty[st], (static_cast<uint32_t>(it / p.stages) & 1u) ^ 1u, abort_flag);
                if (!ok) break;
                mbar_arrive_expect_tx(&s->full[st], stage_bytes);
                tma_load_2d(smem + st * stage_bytes, &tmW, kb * BK, n0, &s->full[st]);
                tma_load_2d(smem + st * stage_bytes + 128 * BK, &tmX, kb * BK, 0, &s->full[st]);
            }
            if (!ok) {
                *abort_flag = 1;
                atomicOr(p.err, kErrLora);
            }
            // loads in flight must land before the CTA may leave
            for (int i = max(0, issued - p.stages); i < issued; ++i)
                if (!mbar_wait(&s->full[i % p.stages], static_cast<uint32_t>(i / p.stages) & 1u, nullptr))
                    atomicOr(p.err, kErrGemmDrain);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = make_idesc<kAccF32>(128, p.Mn);
            for (int kb = kb0; ok && kb < kb1; ++kb) {
                const int it = kb - kb0, st = it % p.stages;
                ok = mbar_wait(&s->full[st], static_cast<uint32_t>(it / p.stages) & 1u, abort_flag);
                if (!ok) break;
                tc_fence_after();
                const uint64_t w_desc = sw128_kmajor_desc(smem + st * stage_bytes);
                const uint64_t x_desc = sw128_kmajor_desc(smem + st * stage_bytes + 128 * BK);
#pragma unroll
                for (int k = 0; k < BK / UMMA_K; ++k)
                    mma_e4m3<false>(tmem_base, w_desc + 2 * k, x_desc + 2 * k, idesc, (kb > kb0 || k > 0) ? 1u : 0u);
                mma_commit(&s->empty[st]);
            }
            // Also with a failed wait: every MMA issued must end before TMEM is freed.
            mma_commit(&s->tmem_full);
            if (!ok) {
                *abort_flag = 1;
                atomicOr(p.err, kErrLora);
            }
            if (!mbar_wait(&s->tmem_full, 0, nullptr)) atomicOr(p.err, kErrGemmDrain);
        }
    } else {
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        const int nl = quarter * 32 + lane;
        const int m0 = rank * p.share, m1 = min(p.M, m0 + p.share);
        pdl_wait();  // t
        const int units = p.R / 8;
        const int in_half = static_cast<int>(threadIdx.x) - 64 - 128 * half;
        for (int mb = m0 + 4 * half; mb < m1; mb += 8) {
            for (int e = in_half; e < p.R; e += 128)  // 4 R floats, 16 bytes at a time
                if (mb + e / (p.R / 4) < m1)
                    reinterpret_cast<float4*>(s->t[half][e / (p.R / 4)])[e % (p.R / 4)] =
                        __ldg(reinterpret_cast<const float4*>(p.t + static_cast<int64_t>(mb) * p.R) + e);
            named_bar_sync(1 + half, 128);
            float* to = lora + (mb - m0) * 128 + quarter * 32;
            if (units >= 8) small_expand<8>(p, s->t[half], mb, m1, n0 + quarter * 32, units, to);
            else if (units >= 4) small_expand<4>(p, s->t[half], mb, m1, n0 + quarter * 32, units, to);
            else if (units >= 2) small_expand<2>(p, s->t[half], mb, m1, n0 + quarter * 32, units, to);
            else small_expand<1>(p, s->t[half], mb, m1, n0 + quarter * 32, units, to);
            named_bar_sync(1 + half, 128);  // t is read
        }
        ok = mbar_wait_warp(&s->tmem_full, 0, abort_flag);
        if (ok) {
            tc_fence_after();
            for (int c = 16 * half; c < p.Mn; c += 32) {
                uint32_t acc[16];
                tmem_ld_32x32b_x16(tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(c), acc);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j) part[(c + j) * 128 + nl] = __uint_as_float(acc[j]);
            }
            tc_fence_before();
        } else if (lane == 0) {
            *abort_flag = 1;
            atomicOr(p.err, kErrLora);
        }
        if (p.splits == 1) named_bar_sync(3, 256);  // the halves read each other's sums
    }
    __syncwarp();
    if (p.splits > 1) cluster_sync_all();  // every CTA's partial sums are written
    if (warp >= 2) {
        const int nl = (warp & 3) * 32 + lane, n = n0 + nl, half = (warp - 2) >> 2;
        const int m0 = rank * p.share, m1 = min(p.M, m0 + p.share);
        if (n < p.N) {
            const float sw = __ldg(p.s_w + n);
            const float bias = p.bias != nullptr ? __bfloat162float(p.bias[n]) : 0.0f;
            for (int m = m0 + half; m < m1; m += 2) {
                // rows 4 .. 7 of every eight are the other half's: the barriers behind that are passed
                float v = lora[(m - m0) * 128 + nl];
                const uint32_t at = smem_u32(part + m * 128 + nl);
                if (p.splits > 1) {
                    float w[8];
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        if (q < p.splits) w[q] = ld_cluster_f32(mapa_shared(at, q));
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        if (q < p.splits) v += w[q];
                } else {
                    v += part[m * 128 + nl];
                }
                p.out[static_cast<int64_t>(m) * p.N + n] = __float2bfloat16_rn(fmaf(v * __ldg(p.s_a + m), sw, bias));
            }
        }
    }
    __syncwarp();
    if (p.splits > 1) cluster_sync_after_reads();  // nobody leaves while its partial sums are read
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem_base, tmem_cols);
    }
}

tfq_status lora_launch_error(cudaError_t e) {
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? TFQ_OK : fail(TFQ_ECUDA, "adapter launch: %s", cudaGetErrorString(e));
}

}  // namespace

tfq_status launch_lora_fold(const void* B, const float* scaling, const float* s_w, int64_t n, int64_t N, int64_t R,
                            void* Bs, cudaStream_t stream) {
    const int64_t blocks = std::min<int64_t>((n * N + 7) / 8, 148 * 16);
    return lora_launch_error(launch_kernel(lora_fold_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream,
                                           static_cast<const __nv_bfloat16*>(B), scaling, s_w, n, N, R,
                                           static_cast<__nv_bfloat16*>(Bs)));
}

namespace {

// A kernel launch with programmatic stream serialization and, from two CTAs up, a cluster.
template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kernel)(KArgs...), unsigned grid, unsigned block, size_t smem, int cluster,
                           cudaStream_t stream, Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = TFQ_PDL;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

tfq_status launch_shrink(const LoraCall& l, const float* s_a, int64_t M, int64_t K, __nv_bfloat16* t, bool halves,
                         cudaStream_t stream, DeviceState* ds) {
    ShrinkArgs a = {};
    a.M = static_cast<int>(M);
    a.R = l.R;
    a.Rn = (l.R + 15) / 16 * 16;
    a.n_adapters = l.n_adapters;
    a.k_blocks = static_cast<int>((K + 63) / 64);
    a.K = static_cast<int>(K);
    a.x = static_cast<const __nv_bfloat16*>(l.x);
    a.idx = l.idx;
    a.s_a = s_a;
    a.t = t;
    a.err = ds->err_word;
    const int blocks = static_cast<int>((M + kShrinkRows - 1) / kShrinkRows);
    // A CTA per 128 rows and one more, further ones where rows of many adapters
    // make more items and the grid is small; K over a cluster while every CTA
    // keeps four steps.  Those with work are resident at once.
    const int block_rows = static_cast<int>(std::min<int64_t>(M, kShrinkRows));
    const int least = (block_rows + 127) / 128 + (l.n_adapters > 1 ? 1 : 0);  // a run's end makes one item more
    const int items = std::min(block_rows, (block_rows + 127) / 128 + l.n_adapters - 1);
    // Three CTAs per SM where that leaves three stages each: more of them share a
    // block's items (12 adapters of rank 24 in any order, 1777 x 5120: 29 us
    // against 36 with two).  Higher ranks would be left with two stages (rank 64,
    // the whole call on 9472 x 5120 x 5120, two against three CTAs: one adapter
    // 233 / 243 us, four in any order 251 / 265, 64 of them 757 / 725).
    const int per_sm = a.Rn <= 32 ? 3 : 2;
    a.splits = 1;
    while (a.splits < 8 && blocks * ((block_rows + 127) / 128) * a.splits * 2 <= 2 * ds->sm_count &&
           a.k_blocks >= a.splits * 8)
        a.splits *= 2;
    a.item_ctas = std::max(least, std::min(items, per_sm * ds->sm_count / (a.splits * blocks)));
    const int stage = shrink_stage_bytes(a.Rn);
    const int rest = 1024 + static_cast<int>(sizeof(ShrinkTail));
    // as many stages as leave room for them, but two, and enough to hold an
    // item's partial sums afterwards (the largest ranks: one CTA per SM)
    const int least_stages = std::max(2, a.splits > 1 ? (128 * (a.R + 4) * 4 + stage - 1) / stage : 0);
    a.stages = std::max(least_stages, std::min(kShrinkMaxStages, ((per_sm == 3 ? 75 : 112) * 1024 - rest) / stage));
    const size_t smem = static_cast<size_t>(rest) + static_cast<size_t>(a.stages) * stage;
    tfq_status st = once_per_device(ds->shrink_attr_set, [] {
        cudaError_t e = cudaSuccess;
        for (auto k : {lora_shrink_kernel<false>, lora_shrink_kernel<true>})
            if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
        return e;
    });
    if (st != TFQ_OK) return st;
    CUtensorMap tmX, tmA;
    st = encode_tensor_map_2d(&tmX, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, l.x, K, M, K * 2, 64, 128,
                                         CU_TENSOR_MAP_SWIZZLE_128B);
    if (st == TFQ_OK)
        st = encode_tensor_map_2d(&tmA, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, l.A, K,
                                  static_cast<uint64_t>(l.n_adapters) * l.R, K * 2, 64, a.Rn,
                                  CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != TFQ_OK) return st;
    return lora_launch_error(launch_cluster(halves ? lora_shrink_kernel<true> : lora_shrink_kernel<false>,
                                            static_cast<unsigned>(blocks * a.item_ctas * a.splits), kShrinkThreads,
                                            smem, a.splits, stream, tmX, tmA, a));
}

}  // namespace

namespace {

tfq_status launch_small_lora(const void* A_q, const float* s_a, const void* W_q, const float* s_w, const void* bias,
                             int64_t M, int64_t N, int64_t K, const LoraCall& l, void* out, cudaStream_t stream,
                             DeviceState* ds) {
    float* t = static_cast<float*>(l.workspace);
    const int units = static_cast<int>(K / 8);
    // warps per dot product: enough warps to keep the GPU's loads in flight, at least two loads a lane
    int dot_warps = 1;
    while (dot_warps < 8 && (M + 3) / 4 * l.R * dot_warps * 2 <= 32 * ds->sm_count && units >= 64 * dot_warps)
        dot_warps *= 2;
    const int64_t ctas = (M + 3) / 4 * l.R * dot_warps / 8;
    tfq_status st = lora_launch_error(launch_cluster(lora_rows_kernel, static_cast<unsigned>(ctas), 256, 0, 1, stream,
                                                     static_cast<const uint4*>(l.x), static_cast<const uint4*>(l.A),
                                                     l.idx, s_a, static_cast<int>(M), l.n_adapters, l.R,
                                                     units, dot_warps, t));
    if (st != TFQ_OK) return st;
    SmallArgs a = {};
    a.M = static_cast<int>(M);
    a.Mn = static_cast<int>((M + 15) / 16 * 16);
    a.N = static_cast<int>(N);
    a.k_blocks = static_cast<int>((K + BK - 1) / BK);
    a.n_adapters = l.n_adapters;
    a.R = l.R;
    a.idx = l.idx;
    a.t = t;
    a.Bs = static_cast<const uint4*>(l.Bs);
    a.s_a = s_a;
    a.s_w = s_w;
    a.bias = static_cast<const __nv_bfloat16*>(bias);
    a.out = static_cast<__nv_bfloat16*>(out);
    a.err = ds->err_word;
    const int64_t tiles = (N + 127) / 128;
    // K over a cluster while the grid stays within two CTAs per SM and every CTA has four steps
    a.splits = 1;
    while (a.splits < 8 && tiles * a.splits * 2 <= 2 * ds->sm_count && a.k_blocks >= a.splits * 8) a.splits *= 2;
    a.share = static_cast<int>((M + a.splits - 1) / a.splits);
    const int rest = 1024 + a.share * 512 + static_cast<int>(sizeof(SmallTail));
    const int stage = small_stage_bytes(a.Mn);
    // as many stages as leave room for two CTAs per SM, but two, and enough to
    // hold the partial sums afterwards (a short K is not split, and one CTA then
    // has all rows' second product: that may take more than half an SM)
    const int least = std::max(2, (a.Mn * 512 + stage - 1) / stage);
    a.stages = std::max(least, std::min(kSmallMaxStages, (112 * 1024 - rest) / stage));
    const size_t smem = static_cast<size_t>(rest) + static_cast<size_t>(a.stages) * stage;
    st = once_per_device(ds->small_attr_set, [] {
        return cudaFuncSetAttribute(small_lora_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
    });
    if (st != TFQ_OK) return st;
    CUtensorMap tmW, tmX;
    st = encode_tensor_map_2d(&tmW, CU_TENSOR_MAP_DATA_TYPE_UINT8, W_q, K, N, K, BK, 128, CU_TENSOR_MAP_SWIZZLE_128B);
    if (st == TFQ_OK)
        st = encode_tensor_map_2d(&tmX, CU_TENSOR_MAP_DATA_TYPE_UINT8, A_q, K, M, K, BK, static_cast<uint32_t>(a.Mn),
                                  CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != TFQ_OK) return st;
    return lora_launch_error(launch_cluster(small_lora_kernel, static_cast<unsigned>(tiles * a.splits), kSmallThreads,
                                            smem, a.splits, stream, tmW, tmX, a));
}

}  // namespace

// Few rows.  Its cost grows with M R, that of the path for many rows with the
// adapters that meet in a tile.  Measured on B200, 5120 x 5120 (us, few against
// many; one adapter, then 64 in any order): M = 32, R = 128 22 / 32, 28 / 62;
// M = 64, R = 64 24 / 31, 29 / 74; M = 64, R = 128 37 / 33, 48 / 106; M = 128,
// R = 32 29 / 31, 33 / 85; M = 128, R = 64 41 / 31, 50 / 95.
static bool use_small_lora(int64_t M, int64_t R, int64_t n_adapters) {
    return M <= kSmallM && (M * R <= 4096 || n_adapters > 8);
}

// The first product: fp32 for few rows, two bf16 halves up to K = kHalvesK, else
// one (the workspace formula knows no K).
constexpr int64_t kHalvesK = 512;
size_t lora_workspace_bytes(int64_t M, int64_t R) { return static_cast<size_t>(M) * static_cast<size_t>(R) * 4; }

tfq_status launch_scaled_fp8_lora(const void* A_q, const float* s_a, const void* W_q, const float* s_w,
                                  const void* bias, int64_t M, int64_t N, int64_t K, const LoraCall& l, void* out,
                                  cudaStream_t stream, DeviceState* ds) {
    if (use_small_lora(M, l.R, l.n_adapters)) return launch_small_lora(A_q, s_a, W_q, s_w, bias, M, N, K, l, out, stream, ds);
    __nv_bfloat16* t = static_cast<__nv_bfloat16*>(l.workspace);
    const bool halves = K <= kHalvesK;
    tfq_status st = launch_shrink(l, s_a, M, K, t, halves, stream, ds);
    if (st != TFQ_OK) return st;
    return launch_lora_pair_gemm(A_q, s_a, W_q, s_w, bias, M, N, K, l, t, halves, out, stream, ds);
}

}  // namespace tfq
