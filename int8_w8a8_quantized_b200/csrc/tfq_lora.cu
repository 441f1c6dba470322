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
    // the row that stands for "another adapter" in the second product
    if (blockIdx.x == 0 && warp >= 2)
        for (int r = threadIdx.x - 64; r < p.R; r += 128) p.t[static_cast<int64_t>(p.M) * p.R + r] = __float2bfloat16_rn(0.0f);

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
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * a.pass_ctas * a.splits));
    cfg.blockDim = dim3(kShrinkThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = TFQ_PDL;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(a.splits);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.splits > 1 ? 2 : 1;
    return lora_launch_error(cudaLaunchKernelEx(&cfg, lora_shrink_kernel, tmX, tmA, a));
}

}  // namespace

size_t lora_workspace_bytes(int64_t M, int64_t R) { return static_cast<size_t>((M + 1) * R * 2 + 15) / 16 * 16; }

tfq_status launch_scaled_fp8_lora(const void* A_q, const float* s_a, const void* W_q, const float* s_w,
                                  const void* bias, int64_t M, int64_t N, int64_t K, const LoraCall& l, void* out,
                                  cudaStream_t stream, DeviceState* ds) {
    __nv_bfloat16* t = static_cast<__nv_bfloat16*>(l.workspace);
    tfq_status st = launch_shrink(l, s_a, M, K, t, stream, ds);
    if (st != TFQ_OK) return st;
    return launch_lora_pair_gemm(A_q, s_a, W_q, s_w, bias, M, N, K, l, t, out, stream, ds);
}

}  // namespace tfq
