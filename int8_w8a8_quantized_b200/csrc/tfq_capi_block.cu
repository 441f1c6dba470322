// tfq_capi_block.cu -- the extern "C" entry points of the operators around the
// Linear (layer norm, rotary positions, low-rank adapters): argument
// validation and launches.  See include/tfq.h for the contract of every function.
#include <algorithm>
#include <cmath>

#include "tfq_args.h"
#include "tfq_internal.h"

namespace tfq {
namespace {

int type_size(int dtype) {
    switch (dtype) {
        case TFQ_DTYPE_BF16:
        case TFQ_DTYPE_FP16: return 2;
        case TFQ_DTYPE_FP32: return 4;
        default: return 0;
    }
}

bool misaligned(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(bytes)) != 0; }

constexpr int64_t kLimit = int64_t(1) << 31;

tfq_status check_norm_sizes(int64_t M, int64_t K, int64_t groups, int dtype, int w_dtype, int64_t stride, float offset) {
    if (M < 0 || K < 0) return fail(TFQ_EINVAL, "negative size (M=%lld, K=%lld)", (long long)M, (long long)K);
    if (type_size(dtype) == 0) return fail(TFQ_EINVAL, "unknown dtype %d", dtype);
    if (w_dtype != dtype && w_dtype != TFQ_DTYPE_FP32)
        return fail(TFQ_EINVAL, "w_dtype %d is neither dtype nor fp32", w_dtype);
    if (groups < 1 || M % groups != 0)
        return fail(TFQ_EINVAL, "M=%lld rows do not make %lld equal groups", (long long)M, (long long)groups);
    if (stride < K) return fail(TFQ_EINVAL, "row stride %lld below K=%lld", (long long)stride, (long long)K);
    if (!std::isfinite(offset)) return fail(TFQ_EINVAL, "weight_offset is not finite");
    if (K > TFQ_NORM_MAX_K) return fail(TFQ_EUNSUPPORTED, "K=%lld above %d", (long long)K, TFQ_NORM_MAX_K);
    if (M >= kLimit || (K > 0 && groups > (kLimit - 1) / K)) return fail(TFQ_EUNSUPPORTED, "size too large");
    return TFQ_OK;
}

tfq_status check_norm_forward(const NormCall& c) {
    tfq_status st = check_norm_sizes(c.M, c.K, c.groups, c.dtype, c.w_dtype, c.x_stride, c.offset);
    if (st != TFQ_OK) return st;
    if (!std::isfinite(c.eps) || c.eps < 0.0f) return fail(TFQ_EINVAL, "eps=%g", (double)c.eps);
    if (c.M == 0 || c.K == 0) return TFQ_OK;
    if (c.x == nullptr) return fail(TFQ_EINVAL, "null pointer");
    if (misaligned(c.x, type_size(c.dtype)) || misaligned(c.w, type_size(c.w_dtype)) ||
        misaligned(c.b, type_size(c.w_dtype)))
        return fail(TFQ_EINVAL, "pointer not aligned to its element");
    return TFQ_OK;
}

tfq_status check_rope_tensor(const RopeTensor& t, int elem, const char* name) {
    if (t.heads == 0) return TFQ_OK;
    if (t.in == nullptr || t.out == nullptr) return fail(TFQ_EINVAL, "%s: null pointer", name);
    if (misaligned(t.in, elem) || misaligned(t.out, elem))
        return fail(TFQ_EINVAL, "%s: pointer not aligned to its element", name);
    return TFQ_OK;
}

}  // namespace
}  // namespace tfq

using namespace tfq;

extern "C" {

tfq_status tfq_layer_norm(const void* x, int64_t x_stride, int dtype, const void* weight, const void* bias,
                          int w_dtype, float weight_offset, int64_t M, int64_t K, int64_t groups, float eps, void* y,
                          float* mean, float* rstd, void* stream) {
    const NormCall c = {x, x_stride, dtype, weight, bias, w_dtype, weight_offset, M, K, groups, eps, mean, rstd};
    tfq_status st = check_norm_forward(c);
    if (st != TFQ_OK || M == 0 || K == 0) return st;
    if (y == nullptr) return fail(TFQ_EINVAL, "null pointer");
    if ((mean == nullptr) != (rstd == nullptr)) return fail(TFQ_EINVAL, "mean and rstd go together");
    if (misaligned(y, type_size(dtype)) || misaligned(mean, 4) || misaligned(rstd, 4))
        return fail(TFQ_EINVAL, "pointer not aligned to its element");
    DeviceState* ds = current_device_state(&st);
    if (ds == nullptr) return st;
    return launch_layer_norm(c, y, nullptr, nullptr, 0.0f, static_cast<cudaStream_t>(stream), ds);
}

tfq_status tfq_layer_norm_quant_fp8(const void* x, int64_t x_stride, int dtype, const void* weight, const void* bias,
                                    int w_dtype, float weight_offset, int64_t M, int64_t K, int64_t groups, float eps,
                                    float qmax, void* q_e4m3, float* s, void* stream) {
    const NormCall c = {x, x_stride, dtype, weight, bias, w_dtype, weight_offset, M, K, groups, eps, nullptr, nullptr};
    tfq_status st = check_norm_forward(c);
    if (st != TFQ_OK) return st;
    if (K % 16 != 0) return fail(TFQ_EINVAL, "K=%lld is not a multiple of 16", (long long)K);
    if (!std::isfinite(qmax) || qmax < 1.0f || qmax > 448.0f)
        return fail(TFQ_EINVAL, "qmax=%g outside [1, 448]", (double)qmax);
    if (M == 0) return TFQ_OK;
    if (s == nullptr || (K > 0 && q_e4m3 == nullptr)) return fail(TFQ_EINVAL, "null pointer");
    if (!aligned16(q_e4m3) || !aligned16(s)) return fail(TFQ_EINVAL, "output not 16-byte aligned");
    DeviceState* ds = current_device_state(&st);
    if (ds == nullptr) return st;
    // rows without elements: only the floored scale, as the quantizer writes it
    if (K == 0) return launch_quant_rows(nullptr, M, 0, qmax, false, nullptr, s, static_cast<cudaStream_t>(stream), ds);
    return launch_layer_norm(c, nullptr, static_cast<uint8_t*>(q_e4m3), s, qmax, static_cast<cudaStream_t>(stream), ds);
}

size_t tfq_layer_norm_backward_workspace_bytes(int64_t M, int64_t K, int64_t groups) {
    if (M <= 0 || K <= 0 || groups < 1 || M % groups != 0 || K > TFQ_NORM_MAX_K) return 0;
    return static_cast<size_t>(layer_norm_backward_workspace(M, K, groups));
}

tfq_status tfq_layer_norm_backward(const void* dy, int64_t dy_stride, const void* x, int64_t x_stride, int dtype,
                                   const void* weight, int w_dtype, float weight_offset, const float* mean,
                                   const float* rstd, int64_t M, int64_t K, int64_t groups, void* dx, void* dweight,
                                   void* dbias, void* workspace, void* stream) {
    tfq_status st = check_norm_sizes(M, K, groups, dtype, w_dtype, std::min(x_stride, dy_stride), weight_offset);
    if (st != TFQ_OK || K == 0) return st;
    const int e = type_size(dtype), we = type_size(w_dtype);
    if (dx == nullptr && dweight == nullptr && dbias == nullptr) return TFQ_OK;
    if (misaligned(dx, e) || misaligned(dweight, we) || misaligned(dbias, we))
        return fail(TFQ_EINVAL, "pointer not aligned to its element");
    if (M > 0) {
        if (dy == nullptr || x == nullptr || mean == nullptr || rstd == nullptr)
            return fail(TFQ_EINVAL, "null pointer");
        if (misaligned(dy, e) || misaligned(x, e) || misaligned(weight, we) || misaligned(mean, 4) ||
            misaligned(rstd, 4))
            return fail(TFQ_EINVAL, "pointer not aligned to its element");
        if ((dweight != nullptr || dbias != nullptr) && (workspace == nullptr || !aligned16(workspace)))
            return fail(TFQ_EINVAL, "workspace null or not 16-byte aligned");
    }
    DeviceState* ds = current_device_state(&st);
    if (ds == nullptr) return st;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (M == 0) {  // sums over no rows
        for (void* d : {dweight, dbias}) {
            const cudaError_t err = d == nullptr ? cudaSuccess : cudaMemsetAsync(d, 0, static_cast<size_t>(groups * K * we), cs);
            if (err != cudaSuccess) return fail(TFQ_ECUDA, "clearing a gradient: %s", cudaGetErrorString(err));
        }
        return TFQ_OK;
    }
    const NormCall c = {x, x_stride, dtype, weight, nullptr, w_dtype, weight_offset, M, K, groups, 0.0f,
                        const_cast<float*>(mean), const_cast<float*>(rstd)};
    return launch_layer_norm_backward(c, dy, dy_stride, dx, dweight, dbias, static_cast<float*>(workspace), cs, ds);
}

tfq_status tfq_rope_axes(const void* q, int64_t q_row_stride, int64_t q_head_stride, int q_heads, void* q_out,
                         int64_t q_out_row_stride, int64_t q_out_head_stride, const void* k, int64_t k_row_stride,
                         int64_t k_head_stride, int k_heads, void* k_out, int64_t k_out_row_stride,
                         int64_t k_out_head_stride, int64_t M, int D, int dtype, const void* positions, int pos_is_64,
                         int64_t pos_row_stride, int64_t pos_axis_stride, int n_axes, int n_pairs,
                         const double* inv_freq, const int32_t* axis, int pairing, int inverse, void* stream) {
    if (M < 0 || q_heads < 0 || k_heads < 0 || D < 0) return fail(TFQ_EINVAL, "negative size");
    const int e = type_size(dtype);
    if (e == 0) return fail(TFQ_EINVAL, "unknown dtype %d", dtype);
    if (pairing != TFQ_ROPE_INTERLEAVED && pairing != TFQ_ROPE_HALVES)
        return fail(TFQ_EINVAL, "unknown pairing %d", pairing);
    if (n_pairs < 1 || n_pairs > D / 2) return fail(TFQ_EINVAL, "n_pairs=%d with D=%d", n_pairs, D);
    if (n_axes < 1) return fail(TFQ_EINVAL, "n_axes=%d", n_axes);
    if (D > TFQ_ROPE_MAX_D) return fail(TFQ_EUNSUPPORTED, "D=%d above %d", D, TFQ_ROPE_MAX_D);
    if (n_axes > 255) return fail(TFQ_EUNSUPPORTED, "n_axes=%d above 255", n_axes);
    if (q_heads > 65536 || k_heads > 65536 - q_heads || M >= kLimit) return fail(TFQ_EUNSUPPORTED, "size too large");
    if (inv_freq == nullptr || axis == nullptr) return fail(TFQ_EINVAL, "null frequency table");
    for (int i = 0; i < n_pairs; ++i) {
        if (!std::isfinite(inv_freq[i])) return fail(TFQ_EINVAL, "inv_freq[%d] is not finite", i);
        if (axis[i] < 0 || axis[i] >= n_axes) return fail(TFQ_EINVAL, "axis[%d]=%d outside [0, %d)", i, axis[i], n_axes);
    }
    if (M == 0 || q_heads + k_heads == 0) return TFQ_OK;
    const RopeTensor tq = {q, q_out, q_row_stride, q_head_stride, q_out_row_stride, q_out_head_stride, q_heads};
    const RopeTensor tk = {k, k_out, k_row_stride, k_head_stride, k_out_row_stride, k_out_head_stride, k_heads};
    tfq_status st = check_rope_tensor(tq, e, "q");
    if (st == TFQ_OK) st = check_rope_tensor(tk, e, "k");
    if (st != TFQ_OK) return st;
    if (positions == nullptr || misaligned(positions, pos_is_64 ? 8 : 4))
        return fail(TFQ_EINVAL, "positions null or not aligned to their element");
    DeviceState* ds = current_device_state(&st);
    if (ds == nullptr) return st;
    return launch_rope(tq, tk, M, D, dtype, positions, pos_is_64 != 0, pos_row_stride, pos_axis_stride, n_pairs,
                       inv_freq, axis, pairing == TFQ_ROPE_HALVES, inverse != 0, static_cast<cudaStream_t>(stream), ds);
}

tfq_status tfq_lora_fold(const void* lora_B, const float* scaling, const float* s_w, int64_t n_adapters, int64_t N,
                         int64_t R, void* lora_Bs, void* stream) {
    if (n_adapters < 0 || N < 0 || R < 0) return fail(TFQ_EINVAL, "negative size");
    if (n_adapters >= kLimit || N >= kLimit || R >= kLimit) return fail(TFQ_EUNSUPPORTED, "size too large");
    if (n_adapters == 0 || N == 0 || R == 0) return TFQ_OK;
    if (lora_B == nullptr || s_w == nullptr || lora_Bs == nullptr) return fail(TFQ_EINVAL, "null pointer");
    if (misaligned(lora_B, 2) || misaligned(lora_Bs, 2) || misaligned(s_w, 4) || misaligned(scaling, 4))
        return fail(TFQ_EINVAL, "pointer not aligned to its element");
    tfq_status st;
    DeviceState* ds = current_device_state(&st);
    if (ds == nullptr) return st;
    return launch_lora_fold(lora_B, scaling, s_w, n_adapters, N, R, lora_Bs, static_cast<cudaStream_t>(stream));
}

size_t tfq_scaled_fp8_linear_lora_workspace_bytes(int64_t M, int64_t R) {
    return M <= 0 || R <= 0 || R > TFQ_LORA_MAX_RANK ? 0 : lora_workspace_bytes(M, R);
}

tfq_status tfq_scaled_fp8_linear_lora(const void* A_q, const float* s_a, const void* W_q, const float* s_w,
                                      const void* bias_bf16, int64_t M, int64_t N, int64_t K, const void* x_bf16,
                                      const void* lora_A, const void* lora_Bs, const int32_t* adapter,
                                      int64_t n_adapters, int64_t R, void* out_bf16, void* workspace, void* stream) {
    tfq_status st = check_gemm_args(A_q, s_a, W_q, s_w, bias_bf16, M, N, K, out_bf16);
    if (st != TFQ_OK) return st;
    if (n_adapters < 0 || R < 0) return fail(TFQ_EINVAL, "negative size");
    if (R % 8 != 0) return fail(TFQ_EINVAL, "R=%lld is not a multiple of 8", (long long)R);
    if (R > TFQ_LORA_MAX_RANK) return fail(TFQ_EUNSUPPORTED, "R=%lld above %d", (long long)R, TFQ_LORA_MAX_RANK);
    if (n_adapters > TFQ_LORA_MAX_ADAPTERS)
        return fail(TFQ_EUNSUPPORTED, "n_adapters=%lld above %d", (long long)n_adapters, TFQ_LORA_MAX_ADAPTERS);
    if (n_adapters > 0 && n_adapters > (kLimit - 1024) / std::max<int64_t>(1, std::max(N, R)))
        return fail(TFQ_EUNSUPPORTED, "size too large");
    if (M == 0 || N == 0) return TFQ_OK;
    const bool adapters = n_adapters > 0 && R > 0;
    if (adapters) {
        if (x_bf16 == nullptr || lora_A == nullptr || lora_Bs == nullptr || adapter == nullptr || workspace == nullptr)
            return fail(TFQ_EINVAL, "null pointer");
        if (!aligned16(x_bf16) || !aligned16(lora_A) || !aligned16(lora_Bs) || !aligned16(workspace) ||
            misaligned(adapter, 4))
            return fail(TFQ_EINVAL, "misaligned pointer");
    }
    DeviceState* ds = current_device_state(&st);
    if (ds == nullptr) return st;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (!adapters) return launch_scaled_fp8_gemm(A_q, s_a, W_q, s_w, bias_bf16, M, N, K, out_bf16, cs, ds);
    const LoraCall l = {x_bf16, lora_A, lora_Bs, adapter, static_cast<int>(n_adapters), static_cast<int>(R), workspace};
    return launch_scaled_fp8_lora(A_q, s_a, W_q, s_w, bias_bf16, M, N, K, l, out_bf16, cs, ds);
}

}  // extern "C"
