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
// First product, rows in tiles of 128 (lora_shrink_kernel):
//   t[m, r] = bf16(sum_k x[m,k] A[idx[m],r,k] / s_a[m]).
// A CTA takes 128 rows and streams their x through shared memory once for as
// many adapters as fit 128 accumulator columns (each Rn = R rounded up to 16
// columns wide), so a tile whose rows belong to one adapter, or to a few of
// low rank, reads x once; more adapters take further passes over x (from L2)
// or, while the grid is small, other CTAs.  Bound by HBM: x is M K bf16
// values against 2 R flops each, far below the tensor cores' ratio; the
// tensor cores are used because plain FMAs would not keep up from R = 16 on.
// Few tiles split K over a cluster of S CTAs, whose partial sums meet in
// shared memory and are added in rank order (the same bits every time).
// Roles as in the GEMM: warp 0 TMA producer, warp 1 MMA, warps 2..5 epilogue.
constexpr int kShrinkThreads = 192;
constexpr int kShrinkMaxStages = 8;
constexpr int kShrinkXStage = 128 * 128;  // 128 rows x 64 bf16

struct ShrinkArgs {
    int M, R, Rn, n_adapters;
    int per_pass;  // adapters per pass
    int stages, k_blocks, splits, pass_ctas;
    const int32_t* idx;
    const float* s_a;
    __nv_bfloat16* t;
    uint32_t* err;
};

// Shared memory behind the stages and, with splits > 1, the partial sums.
struct ShrinkTail {
    uint64_t full[kShrinkMaxStages], empty[kShrinkMaxStages];
    uint64_t tmem_full, tmem_empty, drain;
    uint32_t tmem_slot;
    int abort_flag;
    int count;
    uint32_t list[128];  // the tile's adapters, increasing
    int16_t place[128];  // a row's adapter in that list, -1: none
};

__host__ __device__ constexpr int shrink_stage_bytes(int cols) { return kShrinkXStage + cols * 128; }

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

__global__ void __launch_bounds__(kShrinkThreads)
    lora_shrink_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmA,
                       const ShrinkArgs p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int cols = p.per_pass * p.Rn;
    const int stage_bytes = shrink_stage_bytes(cols);
    float* part = reinterpret_cast<float*>(smem + p.stages * stage_bytes);  // [128][R], splits > 1
    ShrinkTail* s = reinterpret_cast<ShrinkTail*>(reinterpret_cast<uint8_t*>(part) +
                                                  (p.splits > 1 ? 128 * p.R * sizeof(float) : 0));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = p.splits > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int item = blockIdx.x / p.splits;
    const int tile = item / p.pass_ctas;
    const int first_pass = item - tile * p.pass_ctas;
    const int row0 = tile * 128;
    uint32_t tmem_cols = 32;
    while (static_cast<int>(tmem_cols) < cols) tmem_cols *= 2;

    if (threadIdx.x == 0) {
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(&s->full[i], 1);
            mbar_init(&s->empty[i], 1);
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
    if (warp == 0) {  // the tile's adapters in increasing order, and each row's place among them
        uint32_t v[4];
        int place[4] = {-1, -1, -1, -1};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int m = row0 + lane * 4 + i;
            const uint32_t a = m < p.M ? static_cast<uint32_t>(__ldg(p.idx + m)) : 0xFFFFFFFFu;
            v[i] = a < static_cast<uint32_t>(p.n_adapters) ? a : 0xFFFFFFFFu;
        }
        int n = 0;
        for (uint32_t from = 0;; ++n) {
            uint32_t a = 0xFFFFFFFFu;
#pragma unroll
            for (int i = 0; i < 4; ++i) a = min(a, v[i] >= from ? v[i] : 0xFFFFFFFFu);
            a = __reduce_min_sync(0xFFFFFFFFu, a);
            if (a == 0xFFFFFFFFu) break;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (v[i] == a) place[i] = n;
            if (lane == 0) s->list[n] = a;
            from = a + 1;
        }
        if (lane == 0) s->count = n;
#pragma unroll
        for (int i = 0; i < 4; ++i) s->place[lane * 4 + i] = static_cast<int16_t>(place[i]);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = s->tmem_slot;
    volatile int* abort_flag = &s->abort_flag;
    const int kb0 = static_cast<int>(static_cast<int64_t>(p.k_blocks) * rank / p.splits);
    const int kb1 = static_cast<int>(static_cast<int64_t>(p.k_blocks) * (rank + 1) / p.splits);
    const int count = s->count;
    int it = 0;
    bool ok = true;
    uint32_t turn = 0;  // passes done by this CTA
    for (int base = first_pass * p.per_pass; base < count; base += p.pass_ctas * p.per_pass, ++turn) {
        const int n = min(p.per_pass, count - base);
        if (warp == 0) {
            if (lane == 0) {
                for (int kb = kb0; ok && kb < kb1; ++kb, ++it) {
                    const int st = it % p.stages;
                    ok = mbar_wait(&s->empty[st], (static_cast<uint32_t>(it / p.stages) & 1u) ^ 1u, abort_flag);
                    if (!ok) {
                        *abort_flag = 1;
                        atomicOr(p.err, kErrLora);
                        break;
                    }
                    uint8_t* sx = smem + st * stage_bytes;
                    mbar_arrive_expect_tx(&s->full[st], kShrinkXStage + n * p.Rn * 128);
                    tma_load_2d(sx, &tmX, kb * 64, row0, &s->full[st]);
                    for (int i = 0; i < n; ++i)
                        tma_load_2d(sx + kShrinkXStage + i * p.Rn * 128, &tmA, kb * 64,
                                    static_cast<int>(s->list[base + i]) * p.R, &s->full[st]);
                }
            }
        } else if (warp == 1) {
            if (lane == 0) {
                if (ok) ok = mbar_wait(&s->tmem_empty, (turn & 1u) ^ 1u, abort_flag);
                tc_fence_after();
                const uint32_t idesc = make_idesc_bf16(128, n * p.Rn);
                for (int kb = kb0; ok && kb < kb1; ++kb, ++it) {
                    const int st = it % p.stages;
                    ok = mbar_wait(&s->full[st], static_cast<uint32_t>(it / p.stages) & 1u, abort_flag);
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
            const int row = quarter * 32 + lane;
            const int m = row0 + row;
            const int place = s->place[row] - base;
            const bool mine = place >= 0 && place < n;
            if (ok) ok = mbar_wait_warp(&s->tmem_full, turn & 1u, abort_flag);
            if (ok) {
                tc_fence_after();
                const float sa = mine ? __ldg(p.s_a + m) : 1.0f;
                for (int i = 0; i < n; ++i) {
                    if (!__any_sync(0xFFFFFFFFu, place == i)) continue;
                    for (int c = 0; c < p.R; c += 16) {
                        uint32_t acc[16];
                        tmem_ld_32x32b_x16(tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
                                               static_cast<uint32_t>(i * p.Rn + c),
                                           acc);
                        tmem_ld_wait();
                        if (place == i) {
#pragma unroll
                            for (int h = 0; h < 2; ++h) {  // R % 8 == 0
                                if (c + 8 * h >= p.R) continue;
                                float f[8];
#pragma unroll
                                for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(acc[8 * h + j]);
                                if (p.splits > 1) {
                                    // 16-byte units of a row rotated by the row, so that a warp's rows spread over the banks
                                    const int units = p.R / 4;
                                    float4* dst = reinterpret_cast<float4*>(part + row * p.R);
                                    dst[((c + 8 * h) / 4 + row) % units] = make_float4(f[0], f[1], f[2], f[3]);
                                    dst[((c + 8 * h) / 4 + 1 + row) % units] = make_float4(f[4], f[5], f[6], f[7]);
                                } else {
#pragma unroll
                                    for (int j = 0; j < 8; ++j) f[j] = __fdiv_rn(f[j], sa);
                                    *reinterpret_cast<uint4*>(p.t + static_cast<int64_t>(m) * p.R + c + 8 * h) =
                                        make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]),
                                                   pack2(f[6], f[7]));
                                }
                            }
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
            __syncwarp();
            cluster_sync_all();
            if (warp >= 2) {
                const int share = 128 / p.splits, units = p.R / 4;
                for (int e = threadIdx.x - 64; e < share * units; e += 128) {
                    const int row = rank * share + e / units, u = e % units;
                    const int place = s->place[row] - base;
                    if (place < 0 || place >= n) continue;
                    const uint32_t at = smem_u32(reinterpret_cast<float4*>(part + row * p.R) + (u + row) % units);
                    float4 v = ld_cluster_v4(mapa_shared(at, 0));
                    for (int q = 1; q < p.splits; ++q) {
                        const float4 w = ld_cluster_v4(mapa_shared(at, q));
                        v = make_float4(v.x + w.x, v.y + w.y, v.z + w.z, v.w + w.w);
                    }
                    const float sa = __ldg(p.s_a + row0 + row);
                    *reinterpret_cast<uint2*>(p.t + static_cast<int64_t>(row0 + row) * p.R + 4 * u) =
                        make_uint2(pack2(__fdiv_rn(v.x, sa), __fdiv_rn(v.y, sa)),
                                   pack2(__fdiv_rn(v.z, sa), __fdiv_rn(v.w, sa)));
                }
            }
            __syncwarp();
            cluster_sync_all();  // nobody overwrites or leaves what another still reads
        }
    }
    if (warp == 0 && lane == 0) {  // loads in flight must land before the CTA leaves
        for (int i = max(0, it - p.stages); i < it; ++i)
            if (!mbar_wait(&s->full[i % p.stages], static_cast<uint32_t>(i / p.stages) & 1u, nullptr))
                atomicOr(p.err, kErrGemmDrain);
    } else if (warp == 1 && lane == 0) {
        mma_commit(&s->drain);
        if (!mbar_wait(&s->drain, 0, nullptr)) atomicOr(p.err, kErrGemmDrain);
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
// lora_rows_kernel: t[m, r] = sum_k x[m,k] A[idx[m],r,k] / s_a[m] (fp32), one
// dot product per `dot_warps` warps.
//
// small_lora_kernel: the Linear with the weight as the tensor cores' M operand
// (128 output channels per CTA) and the rows as N (rounded up to 16), so that a
// tile is 128 channels wide however few rows there are, and K split over a
// cluster: N / 128 tiles times the split reach all SMs.  While the weight
// streams, the epilogue warps add up the adapters' second product on plain FMAs:
// thread n reads Bs[a, n, :] of its channel once per row.  The partial sums of
// the cluster meet in shared memory; CTA `rank` finishes its share of the rows.
constexpr int kSmallM = 64;
constexpr int kSmallThreads = 192;
constexpr int kSmallMaxStages = 6;

__global__ void __launch_bounds__(256) lora_rows_kernel(const uint4* x, const uint4* A, const int32_t* idx,
                                                        const float* s_a, int n_adapters, int R, int units,
                                                        int dot_warps, float* t) {
    __shared__ float sums[8];
    // The wait comes first: a kernel that starts after every CTA here has allowed
    // it knows that all earlier kernels of the stream are complete.
    pdl_wait();
    pdl_allow_next();
    const int dots = 8 / dot_warps;  // per CTA; divides R
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t dot = static_cast<int64_t>(blockIdx.x) * dots + warp / dot_warps;
    const int m = static_cast<int>(dot / R);
    const int r = static_cast<int>(dot - static_cast<int64_t>(m) * R);
    const uint32_t a = static_cast<uint32_t>(__ldg(idx + m));
    if (a >= static_cast<uint32_t>(n_adapters)) return;  // the whole CTA has one row
    const uint4* xr = x + static_cast<int64_t>(m) * units;
    const uint4* ar = A + (static_cast<int64_t>(a) * R + r) * units;
    float s = 0.0f;
    const int step = 32 * dot_warps;
#pragma unroll 1
    for (int base = (warp % dot_warps) * 32 + lane; base < units; base += 8 * step) {
        uint4 xv[8], av[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int u = base + j * step;
            xv[j] = u < units ? __ldg(xr + u) : make_uint4(0u, 0u, 0u, 0u);
            av[j] = u < units ? ldg_nc_v4(ar + u) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t xw[4] = {xv[j].x, xv[j].y, xv[j].z, xv[j].w}, aw[4] = {av[j].x, av[j].y, av[j].z, av[j].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s = fmaf(bf16_lo(xw[i]), bf16_lo(aw[i]), s);
                s = fmaf(bf16_hi(xw[i]), bf16_hi(aw[i]), s);
            }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if (dot_warps > 1) {
        if (lane == 0) sums[warp] = s;
        __syncthreads();
        if (warp % dot_warps != 0) return;
        for (int i = 1; i < dot_warps; ++i) s += sums[warp + i];
    }
    if (lane == 0) t[dot] = __fdiv_rn(s, __ldg(s_a + m));
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
};

__host__ __device__ constexpr int small_stage_bytes(int mn) { return (128 + mn) * BK; }

__global__ void __launch_bounds__(kSmallThreads)
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
    const uint32_t tmem_cols = p.Mn <= 32 ? 32 : 64;
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
        const int quarter = warp & 3;
        const int nl = quarter * 32 + lane, n = n0 + nl;
        const int m0 = rank * p.share, m1 = min(p.M, m0 + p.share);
        pdl_wait();  // t
        const int units = p.R / 8;
        for (int mb = m0; mb < m1; mb += 4) {
            const uint4* b[4];
            const float4* t[4];
            float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t a = mb + j < m1 ? static_cast<uint32_t>(__ldg(p.idx + mb + j)) : 0xFFFFFFFFu;
                const bool has = a < static_cast<uint32_t>(p.n_adapters) && n < p.N;
                b[j] = has ? p.Bs + (static_cast<int64_t>(a) * p.N + n) * units : nullptr;
                t[j] = reinterpret_cast<const float4*>(p.t + static_cast<int64_t>(mb + j) * p.R);
            }
#pragma unroll 2
            for (int u = 0; u < units; ++u) {
                uint4 v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (b[j] != nullptr) v[j] = __ldg(b[j] + u);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (b[j] == nullptr) continue;
                    const float4 lo = __ldg(t[j] + 2 * u), hi = __ldg(t[j] + 2 * u + 1);
                    acc[j] = fmaf(bf16_lo(v[j].x), lo.x, acc[j]);
                    acc[j] = fmaf(bf16_hi(v[j].x), lo.y, acc[j]);
                    acc[j] = fmaf(bf16_lo(v[j].y), lo.z, acc[j]);
                    acc[j] = fmaf(bf16_hi(v[j].y), lo.w, acc[j]);
                    acc[j] = fmaf(bf16_lo(v[j].z), hi.x, acc[j]);
                    acc[j] = fmaf(bf16_hi(v[j].z), hi.y, acc[j]);
                    acc[j] = fmaf(bf16_lo(v[j].w), hi.z, acc[j]);
                    acc[j] = fmaf(bf16_hi(v[j].w), hi.w, acc[j]);
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (mb + j < m1) lora[(mb + j - m0) * 128 + nl] = acc[j];
        }
        ok = mbar_wait_warp(&s->tmem_full, 0, abort_flag);
        if (ok) {
            tc_fence_after();
            for (int c = 0; c < p.Mn; c += 16) {
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
    }
    __syncwarp();
    if (p.splits > 1) cluster_sync_all();  // every CTA's partial sums are written
    if (warp >= 2) {
        const int nl = (warp & 3) * 32 + lane, n = n0 + nl;
        const int m0 = rank * p.share, m1 = min(p.M, m0 + p.share);
        if (n < p.N) {
            const float sw = __ldg(p.s_w + n);
            const float bias = p.bias != nullptr ? __bfloat162float(p.bias[n]) : 0.0f;
            for (int m = m0; m < m1; ++m) {
                float v = lora[(m - m0) * 128 + nl];
                const uint32_t at = smem_u32(part + m * 128 + nl);
                if (p.splits > 1) {
                    for (int q = 0; q < p.splits; ++q) v += ld_cluster_f32(mapa_shared(at, q));
                } else {
                    v += part[m * 128 + nl];
                }
                p.out[static_cast<int64_t>(m) * p.N + n] = __float2bfloat16_rn(fmaf(v * __ldg(p.s_a + m), sw, bias));
            }
        }
    }
    __syncwarp();
    if (p.splits > 1) cluster_sync_all();  // nobody leaves while its partial sums are read
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

tfq_status launch_shrink(const LoraCall& l, const float* s_a, int64_t M, int64_t K, __nv_bfloat16* t,
                         cudaStream_t stream, DeviceState* ds) {
    ShrinkArgs a = {};
    a.M = static_cast<int>(M);
    a.R = l.R;
    a.Rn = (l.R + 15) / 16 * 16;
    a.n_adapters = l.n_adapters;
    a.per_pass = std::max(1, std::min(128 / a.Rn, std::min(l.n_adapters, 128)));
    a.k_blocks = static_cast<int>((K + 63) / 64);
    a.idx = l.idx;
    a.s_a = s_a;
    a.t = t;
    a.err = ds->err_word;
    const int tiles = static_cast<int>((M + 127) / 128);
    // K over a cluster while that leaves every CTA four steps and the grid
    // within two CTAs per SM; then the passes of tiles with many adapters
    a.splits = 1;
    while (a.splits < 8 && tiles * a.splits * 2 <= 2 * ds->sm_count && a.k_blocks >= a.splits * 8) a.splits *= 2;
    const int passes = (std::min(l.n_adapters, 128) + a.per_pass - 1) / a.per_pass;
    a.pass_ctas = std::max(1, std::min(passes, 2 * ds->sm_count / (tiles * a.splits)));
    const int stage = shrink_stage_bytes(a.per_pass * a.Rn);
    const int rest = 1024 + static_cast<int>(sizeof(ShrinkTail)) + (a.splits > 1 ? 128 * a.R * 4 : 0);
    // two CTAs per SM where two stages fit half the shared memory
    const int budget = rest + 2 * stage <= 112 * 1024 ? 112 * 1024 : 227 * 1024;
    a.stages = std::min(kShrinkMaxStages, (budget - rest) / stage);
    if (a.stages < 2) return fail(TFQ_EUNSUPPORTED, "rank %d does not fit shared memory", l.R);
    const size_t smem = static_cast<size_t>(rest) + static_cast<size_t>(a.stages) * stage;
    if (!ds->shrink_attr_set) {
        const cudaError_t e = cudaFuncSetAttribute(lora_shrink_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
        if (e != cudaSuccess) return fail(TFQ_ECUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
        ds->shrink_attr_set = true;
    }
    CUtensorMap tmX, tmA;
    tfq_status st = encode_tensor_map_2d(&tmX, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, l.x, K, M, K * 2, 64, 128,
                                         CU_TENSOR_MAP_SWIZZLE_128B);
    if (st == TFQ_OK)
        st = encode_tensor_map_2d(&tmA, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, l.A, K,
                                  static_cast<uint64_t>(l.n_adapters) * l.R, K * 2, 64, a.Rn,
                                  CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != TFQ_OK) return st;
    return lora_launch_error(launch_cluster(lora_shrink_kernel, static_cast<unsigned>(tiles * a.pass_ctas * a.splits),
                                            kShrinkThreads, smem, a.splits, stream, tmX, tmA, a));
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
    while (dot_warps < 8 && M * l.R * dot_warps * 2 <= 32 * ds->sm_count && units >= 128 * dot_warps) dot_warps *= 2;
    const int64_t ctas = M * l.R * dot_warps / 8;
    tfq_status st = lora_launch_error(launch_cluster(lora_rows_kernel, static_cast<unsigned>(ctas), 256, 0, 1, stream,
                                                     static_cast<const uint4*>(l.x), static_cast<const uint4*>(l.A),
                                                     l.idx, s_a, l.n_adapters, l.R, units, dot_warps, t));
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
    a.stages = std::min(kSmallMaxStages, (112 * 1024 - rest) / stage);  // two CTAs per SM
    const size_t smem = static_cast<size_t>(rest) + static_cast<size_t>(a.stages) * stage;
    if (!ds->small_attr_set) {
        const cudaError_t e = cudaFuncSetAttribute(small_lora_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 112 * 1024);
        if (e != cudaSuccess) return fail(TFQ_ECUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
        ds->small_attr_set = true;
    }
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

// The first product: bf16 [M, R], or fp32 for few rows.
size_t lora_workspace_bytes(int64_t M, int64_t R) { 
    return static_cast<size_t>(M) * static_cast<size_t>(R) * (M <= kSmallM ? 4 : 2);
}

tfq_status launch_scaled_fp8_lora(const void* A_q, const float* s_a, const void* W_q, const float* s_w,
                                  const void* bias, int64_t M, int64_t N, int64_t K, const LoraCall& l, void* out,
                                  cudaStream_t stream, DeviceState* ds) {
    if (M <= kSmallM) return launch_small_lora(A_q, s_a, W_q, s_w, bias, M, N, K, l, out, stream, ds);
    __nv_bfloat16* t = static_cast<__nv_bfloat16*>(l.workspace);
    tfq_status st = launch_shrink(l, s_a, M, K, t, stream, ds);
    if (st != TFQ_OK) return st;
    return launch_lora_pair_gemm(A_q, s_a, W_q, s_w, bias, M, N, K, l, t, out, stream, ds);
}

}  // namespace tfq
