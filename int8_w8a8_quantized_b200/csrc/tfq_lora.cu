// tfq_lora.cu -- the scaled FP8 Linear with low-rank adapters of many
// requests beside it:
//   out[m,n] = s_a[m] s_w[n] sum_k A_q[m,k] W_q[n,k] + bias[n]
//              + scaling[a] sum_r (sum_k x[m,k] A[a,r,k]) B[a,n,r],   a = idx[m].
// The second factor is kept in units of the weight's scale, Bs = scaling B /
// s_w, and the first product in units of the row's, t[m,r] = sum_k x A / s_a,
// so that both sums share the factor s_a[m] s_w[n].
#include <cuda_bf16.h>

#include <algorithm>

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
        for (int64_t r = threadIdx.x & 31; r < R; r += 32)
            out[row * R + r] = __float2bfloat16_rn(__fdiv_rn(f * __bfloat162float(B[row * R + r]), sw));
    }
}

// t[m, r] = bf16(sum_k x[m,k] A[idx[m],r,k] / s_a[m]): a CTA per row, a warp per r.
__global__ void __launch_bounds__(256) lora_shrink_kernel(const uint4* x, const uint4* A, const int32_t* idx,
                                                          const float* s_a, int n_adapters, int R, int units,
                                                          __nv_bfloat16* t) {
    pdl_allow_next();
    pdl_wait();
    const int64_t m = blockIdx.x;
    const int a = idx[m];
    if (a < 0 || a >= n_adapters) return;
    const int lane = threadIdx.x & 31;
    for (int r = threadIdx.x >> 5; r < R; r += 8) {
        const uint4* xr = x + m * units;
        const uint4* ar = A + (static_cast<int64_t>(a) * R + r) * units;
        float s = 0.0f;
        for (int u = lane; u < units; u += 32) {
            const uint4 xv = xr[u], av = ar[u];
            const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w}, aw[4] = {av.x, av.y, av.z, av.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s = fmaf(bf16_lo(xw[i]), bf16_lo(aw[i]), s);
                s = fmaf(bf16_hi(xw[i]), bf16_hi(aw[i]), s);
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        if (lane == 0) t[m * R + r] = __float2bfloat16_rn(__fdiv_rn(s, s_a[m]));
    }
}

// out[m, n] += s_a[m] s_w[n] sum_r t[m,r] Bs[idx[m],n,r]: a CTA per row.
__global__ void __launch_bounds__(256) lora_expand_kernel(const __nv_bfloat16* t, const __nv_bfloat16* Bs,
                                                          const int32_t* idx, const float* s_a, const float* s_w,
                                                          int n_adapters, int R, int64_t N, __nv_bfloat16* out) {
    __shared__ float tr[TFQ_LORA_MAX_RANK];
    pdl_allow_next();
    pdl_wait();
    const int64_t m = blockIdx.x;
    const int a = idx[m];
    if (a < 0 || a >= n_adapters) return;
    for (int r = threadIdx.x; r < R; r += blockDim.x) tr[r] = __bfloat162float(t[m * R + r]);
    __syncthreads();
    for (int64_t n = threadIdx.x; n < N; n += blockDim.x) {
        const __nv_bfloat16* b = Bs + (a * N + n) * R;
        float s = 0.0f;
        for (int r = 0; r < R; ++r) s = fmaf(tr[r], __bfloat162float(b[r]), s);
        out[m * N + n] = __float2bfloat16_rn(fmaf(s, s_a[m] * s_w[n], __bfloat162float(out[m * N + n])));
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

size_t lora_workspace_bytes(int64_t M, int64_t R) { return static_cast<size_t>(M) * R * 2; }

tfq_status launch_scaled_fp8_lora(const void* A_q, const float* s_a, const void* W_q, const float* s_w,
                                  const void* bias, int64_t M, int64_t N, int64_t K, const LoraCall& l, void* out,
                                  cudaStream_t stream, DeviceState* ds) {
    tfq_status st = launch_scaled_fp8_gemm(A_q, s_a, W_q, s_w, bias, M, N, K, out, stream, ds);
    if (st != TFQ_OK) return st;
    __nv_bfloat16* t = static_cast<__nv_bfloat16*>(l.workspace);
    st = lora_launch_error(launch_kernel(lora_shrink_kernel, dim3(static_cast<unsigned>(M)), dim3(256), 0, stream,
                                         static_cast<const uint4*>(l.x), static_cast<const uint4*>(l.A), l.idx, s_a,
                                         l.n_adapters, l.R, static_cast<int>(K / 8), t));
    if (st != TFQ_OK) return st;
    return lora_launch_error(launch_kernel(lora_expand_kernel, dim3(static_cast<unsigned>(M)), dim3(256), 0, stream,
                                           const_cast<const __nv_bfloat16*>(t),
                                           static_cast<const __nv_bfloat16*>(l.Bs), l.idx, s_a, s_w, l.n_adapters, l.R,
                                           N, static_cast<__nv_bfloat16*>(out)));
}

}  // namespace tfq
