// tfq_norm.cu -- layer norm around the W8A8 Linear: forward, straight to
// per-token E4M3 codes, and backward with the weight and bias gradients.
//
// For a row x[0..K) of group g (M rows in G groups of equally many rows; G = 1
// is the ordinary norm, G > 1 the adaptive norm whose weight and bias come
// from a condition of each sample):
//   mean = 1/K sum x,  rstd = 1 / sqrt(1/K sum (x - mean)^2 + eps)
//   xhat = (x - mean) rstd,  y = xhat (w[g] + offset) + b[g]
// and, with h = dy (w[g] + offset),
//   dx    = rstd (h - 1/K sum h - xhat 1/K sum h xhat)
//   dw[g] = sum over the group's rows of dy xhat,  db[g] = ... of dy.
// The quantizing form writes s = fl32(max(max |y|, 1e-12) / qmax) and the
// E4M3 code of y / s, y being the fp32 value above (not rounded to the input's
// type in between: one rounding fewer than norm and quantizer as two calls,
// and the M x K intermediate is neither written nor read).
//
// All sums, the statistics and the gradients' partial sums are fp32.  The
// variance is summed from x - mean (two passes over a row that stays in
// registers), so a large common offset costs no digits.
//
// Bound by HBM.  Rows of 16-byte units with 33 to 640 threads of 16 columns
// each (K from 513 to 10240) run the ring kernels further down, or, in the forward
// and up to K = 5120, where there are rows enough, those with one or two warps
// per row behind them.  The others (short rows, very long ones, rows of odd length
// or alignment) are read into
// registers: a row belongs to `tpr` threads, a power of two up to 32 (several
// rows per warp, no barrier) or a whole CTA of up to 1024; thread t holds the
// row's units t, t + tpr, ... (J at most).  CTAs walk consecutive rows and load
// the next row before they reduce the present one.  The weight and bias are
// read again for every row: they stay in L1 (the row loads do not allocate
// there).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "tfq_internal.h"
#include "tfq_ptx.cuh"
#include "tfq_quant_common.cuh"
#include "tfq_quant_row.cuh"

namespace tfq {
namespace {

// ------------------------------------------------- units of a row
// VEC elements of type T: one 16-byte unit (VEC * sizeof(T) == 16) or, for
// rows that are not 16-byte aligned, one element.
template <typename T>
__device__ __forceinline__ float to_float(T v) {
    if constexpr (sizeof(T) == 4) return v;
    else if constexpr (std::is_same_v<T, __half>) return __half2float(v);
    else return __bfloat162float(v);
}
template <typename T>
__device__ __forceinline__ T from_float(float v) {
    if constexpr (sizeof(T) == 4) return v;
    else if constexpr (std::is_same_v<T, __half>) return __float2half_rn(v);
    else return __float2bfloat16_rn(v);
}

// One element through the read-only path.  (The 16-bit types' own __ldg is an
// asm statement without side effects, which the compiler may move in front of
// the test that guards it: a load through a null pointer or past the row.)
template <typename T>
__device__ __forceinline__ T ldg_elem(const T* p) {
    if constexpr (sizeof(T) == 4) {
        return __ldg(p);
    } else {
        const unsigned short w = __ldg(reinterpret_cast<const unsigned short*>(p));
        return *reinterpret_cast<const T*>(&w);
    }
}

// Four fp32 values -> four E4M3 codes, the first in the low byte.
__device__ __forceinline__ uint32_t cvt_e4m3x4(float2 lo, float2 hi) {
    uint32_t r;
    asm("{\n\t.reg .b16 a, b;\n\tcvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\t"
        "mov.b32 %0, {a, b};\n\t}"
        : "=r"(r)
        : "f"(lo.x), "f"(lo.y), "f"(hi.x), "f"(hi.y));
    return r;
}

template <typename T, int VEC>
struct Unit {
    static_assert(VEC == 1 || VEC * sizeof(T) == 16, "a unit is one element or 16 bytes");
    using Raw = std::conditional_t<VEC == 1, T, uint4>;
    Raw raw;

    __device__ __forceinline__ void clear() {
        if constexpr (VEC == 1) raw = from_float<T>(0.0f);
        else raw = make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ __forceinline__ void load(const T* row, int u) {
        if constexpr (VEC == 1) raw = ldg_elem(row + u);
        else raw = ldg_nc_v4(reinterpret_cast<const uint4*>(row) + u);
    }
    __device__ __forceinline__ void get(float (&f)[VEC]) const {
        if constexpr (VEC == 1) {
            f[0] = to_float<T>(raw);
        } else {
            const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (sizeof(T) == 4) {
                    f[i] = __uint_as_float(w[i]);
                } else if constexpr (std::is_same_v<T, __half>) {
                    const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                    f[2 * i] = p.x;
                    f[2 * i + 1] = p.y;
                } else {
                    f[2 * i] = bf16_lo(w[i]);
                    f[2 * i + 1] = bf16_hi(w[i]);
                }
            }
        }
    }
    static __device__ __forceinline__ void store(T* row, int u, const float (&f)[VEC]) {
        if constexpr (VEC == 1) {
            row[u] = from_float<T>(f[0]);
        } else {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (sizeof(T) == 4) {
                    w[i] = __float_as_uint(f[i]);
                } else if constexpr (std::is_same_v<T, __half>) {
                    const __half2 p = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
                    w[i] = *reinterpret_cast<const uint32_t*>(&p);
                } else {
                    const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                    w[i] = *reinterpret_cast<const uint32_t*>(&p);
                }
            }
            reinterpret_cast<uint4*>(row)[u] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
};

// VEC values of a weight or bias row (of the input's type, or fp32) from
// column c; in the vector form their addresses are 16-byte aligned.
template <typename T, int VEC>
__device__ __forceinline__ void load_affine(float (&f)[VEC], const void* base, bool f32, int64_t at) {
    if (f32) {
        const float* p = static_cast<const float*>(base) + at;
        if constexpr (VEC == 1) {
            f[0] = __ldg(p);
        } else {
#pragma unroll
            for (int i = 0; i < VEC / 4; ++i) {
                const float4 v = __ldg(reinterpret_cast<const float4*>(p) + i);
                f[4 * i] = v.x;
                f[4 * i + 1] = v.y;
                f[4 * i + 2] = v.z;
                f[4 * i + 3] = v.w;
            }
        }
    } else {
        const T* p = static_cast<const T*>(base) + at;
        Unit<T, VEC> u;
        if constexpr (VEC == 1) u.raw = ldg_elem(p);
        else u.raw = __ldg(reinterpret_cast<const uint4*>(p));
        u.get(f);
    }
}

// ------------------------------------------------- sums over a row's threads
// kWarpRow: the row's tpr (a power of two, <= 32) lanes; otherwise the whole
// CTA, through `red` (32 floats per reduction, zero past the CTA's warps).
// Every thread gets the result, summed in an order that depends only on the
// launch shape.  Consecutive calls need different `red` buffers: a buffer may
// be written again only after another reduction's barrier.
struct SumOp {
    static __device__ __forceinline__ float apply(float a, float b) { return a + b; }
};
struct MaxOp {
    static __device__ __forceinline__ float apply(float a, float b) { return fmaxf(a, b); }
};

template <bool kWarpRow, typename Op, int N>
__device__ __forceinline__ void row_reduce(float (&v)[N], int tpr, float* red) {
    if constexpr (kWarpRow) {
        for (int o = tpr >> 1; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = Op::apply(v[i], __shfl_xor_sync(0xFFFFFFFFu, v[i], o));
    } else {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = Op::apply(v[i], __shfl_xor_sync(0xFFFFFFFFu, v[i], o));
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) red[32 * i + (threadIdx.x >> 5)] = v[i];
        __syncthreads();
        const int quads = (static_cast<int>(blockDim.x >> 5) + 3) >> 2;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float s = 0.0f;
            for (int q = 0; q < quads; ++q) {
                const float4 p = *reinterpret_cast<const float4*>(red + 32 * i + 4 * q);
                s = Op::apply(s, Op::apply(Op::apply(p.x, p.y), Op::apply(p.z, p.w)));
            }
            v[i] = s;
        }
    }
}

struct NormArgs {
    const void* x;
    int64_t x_stride;  // elements between rows
    const void* w;     // [G, K] or null
    const void* b;     // [G, K] or null
    int w_f32;         // w and b (and their gradients) are fp32, else of the input's type
    float offset;
    int64_t M;
    int64_t group_rows;
    int K;
    int tpr;    // threads per row
    float eps;
    float* mean;  // [M] or null (written by the forward, read by the backward)
    float* rstd;
    // forward
    void* y;  // [M, K]
    // quantizing forward
    uint8_t* q;  // [M, K]
    float* s;    // [M]
    float qmax;
    int clamp;  // qmax is not an E4M3 value
    // backward
    const void* dy;
    int64_t dy_stride;
    void* dx;        // [M, K] or null
    float* part_dw;  // [G, parts, K] partial sums, or null
    float* part_db;
    int parts;
};

// Rows per CTA at a time, and this thread's place: row slot and lane in it.
template <bool kWarpRow>
__device__ __forceinline__ void my_place(int tpr, int& slots, int& slot, int& t) {
    if constexpr (kWarpRow) {
        slots = blockDim.x / tpr;
        slot = threadIdx.x / tpr;
        t = threadIdx.x & (tpr - 1);
    } else {
        slots = 1;
        slot = 0;
        t = threadIdx.x;
    }
}

template <typename T, int VEC, int J, bool kWarpRow, bool kQuant>
__global__ void __launch_bounds__(J > 4 ? 1024 : 512)
    norm_forward_kernel(const NormArgs p) {
    __shared__ __align__(16) float red[3][32];
    int slots, slot, t;
    my_place<kWarpRow>(p.tpr, slots, slot, t);
    if constexpr (!kWarpRow)
        for (int i = threadIdx.x; i < 96; i += blockDim.x) (&red[0][0])[i] = 0.0f;
    pdl_allow_next();
    pdl_wait();
    const int units = p.K / VEC;
    // consecutive rows per CTA, so that a group's weight and bias stay in L1
    const int64_t chunk = (p.M + static_cast<int64_t>(gridDim.x) * slots - 1) / (static_cast<int64_t>(gridDim.x) * slots) * slots;
    const int64_t first = blockIdx.x * chunk;
    const int64_t last = min(p.M, first + chunk);
    const float inv_k = 1.0f / static_cast<float>(p.K);
    Unit<T, VEC> cur[J];
    const auto fetch = [&](Unit<T, VEC>(&v)[J], int64_t r) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int u = t + p.tpr * j;
            v[j].clear();
            if (r < last && u < units) v[j].load(static_cast<const T*>(p.x) + r * p.x_stride, u);
        }
    };
    if constexpr (!kWarpRow) __syncthreads();  // red cleared
    fetch(cur, first + slot);
    for (int64_t base = first; base < last; base += slots) {
        const int64_t r = base + slot;
        Unit<T, VEC> next[J];
        fetch(next, r + slots);
        float acc[1] = {0.0f};
#pragma unroll
        for (int j = 0; j < J; ++j) {
            float f[VEC];
            cur[j].get(f);
#pragma unroll
            for (int i = 0; i < VEC; ++i) acc[0] += f[i];
        }
        row_reduce<kWarpRow, SumOp>(acc, p.tpr, red[0]);
        const float mean = acc[0] * inv_k;
        acc[0] = 0.0f;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            if (t + p.tpr * j < units) {
                float f[VEC];
                cur[j].get(f);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float d = f[i] - mean;
                    acc[0] = fmaf(d, d, acc[0]);
                }
            }
        }
        row_reduce<kWarpRow, SumOp>(acc, p.tpr, red[1]);
        const float rstd = __frsqrt_rn(fmaf(acc[0], inv_k, p.eps));
        const bool row_ok = r < last;
        if (p.mean != nullptr && row_ok && t == 0) {
            p.mean[r] = mean;
            p.rstd[r] = rstd;
        }
        int64_t affine = 0;  // M < 2^31: a 32-bit division
        if (p.group_rows != p.M && row_ok)
            affine = static_cast<int64_t>(static_cast<uint32_t>(r) / static_cast<uint32_t>(p.group_rows)) * p.K;
        const auto value = [&](int j, float(&y)[VEC]) {
            const int64_t at = affine + static_cast<int64_t>(t + p.tpr * j) * VEC;
            cur[j].get(y);
#pragma unroll
            for (int i = 0; i < VEC; ++i) y[i] = (y[i] - mean) * rstd;
            if (p.w != nullptr) {
                float w[VEC];
                load_affine<T, VEC>(w, p.w, p.w_f32, at);
#pragma unroll
                for (int i = 0; i < VEC; ++i) y[i] *= w[i] + p.offset;
            }
            if (p.b != nullptr) {
                float b[VEC];
                load_affine<T, VEC>(b, p.b, p.w_f32, at);
#pragma unroll
                for (int i = 0; i < VEC; ++i) y[i] += b[i];
            }
        };
        if constexpr (!kQuant) {
            if (row_ok) {
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    if (t + p.tpr * j < units) {
                        float y[VEC];
                        value(j, y);
                        Unit<T, VEC>::store(static_cast<T*>(p.y) + r * p.K, t + p.tpr * j, y);
                    }
                }
            }
        } else {
            // up to four units a thread the values wait in registers for the
            // row's maximum; more are computed a second time
            constexpr bool kKeep = J * VEC <= 32;
            float y[kKeep ? J : 1][VEC];
            float amax[1] = {0.0f};
#pragma unroll
            for (int j = 0; j < J; ++j) {
                if (t + p.tpr * j < units) {
                    value(j, y[kKeep ? j : 0]);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) amax[0] = fmaxf(amax[0], fabsf(y[kKeep ? j : 0][i]));
                }
            }
            row_reduce<kWarpRow, MaxOp>(amax, p.tpr, red[2]);
            const float sc = __fdiv_rn(fmaxf(amax[0], 1e-12f), p.qmax);
            if (row_ok) {
                if (t == 0) p.s[r] = sc;
                const float rcp = __frcp_rn(sc);
                const float rcp_lo = rcp_low(sc, rcp);
                const bool ieee = !(sc <= kDivMaxScale);
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const int u = t + p.tpr * j;
                    if (u >= units) continue;
                    if constexpr (!kKeep) value(j, y[0]);
                    const float(&yj)[VEC] = y[kKeep ? j : 0];
                    uint32_t codes[(VEC + 1) / 2];
#pragma unroll
                    for (int i = 0; i < VEC; i += 2) {
                        const float a = yj[i], b = VEC > 1 ? yj[(i + 1) % VEC] : 0.0f;
                        float2 d = ieee ? make_float2(__fdiv_rn(a, sc), __fdiv_rn(b, sc))
                                        : div2_rn_unsigned_zero(make_float2(a, b), sc, rcp, rcp_lo);
                        if (p.clamp) {
                            d.x = fminf(fmaxf(d.x, -p.qmax), p.qmax);
                            d.y = fminf(fmaxf(d.y, -p.qmax), p.qmax);
                        }
                        codes[i / 2] = cvt_e4m3x2(d.x, d.y);
                    }
                    uint8_t* out = p.q + r * p.K;
                    if constexpr (VEC == 8) {
                        reinterpret_cast<uint2*>(out)[u] =
                            make_uint2(codes[0] | (codes[1] << 16), codes[2] | (codes[3] << 16));
                    } else if constexpr (VEC == 4) {
                        reinterpret_cast<uint32_t*>(out)[u] = codes[0] | (codes[1] << 16);
                    } else {
                        out[u] = static_cast<uint8_t>(codes[0]);
                    }
                }
            }
        }
#pragma unroll
        for (int j = 0; j < J; ++j) cur[j] = next[j];
    }
}

// Backward.  Grid G * parts: CTA (g, i) walks the i-th share of group g's
// rows; a thread owns the same columns of every row, so the sums for dw and db
// stay in its registers and leave once per CTA, as fp32 partials [g][i][K]
// that norm_partials_kernel adds up in order of i.
template <typename T, int VEC, int J, bool kWarpRow>
__global__ void __launch_bounds__(J > 4 ? 1024 : 512)
    norm_backward_kernel(const NormArgs p) {
    __shared__ __align__(16) float red[2][64];
    int slots, slot, t;
    my_place<kWarpRow>(p.tpr, slots, slot, t);
    if constexpr (!kWarpRow)
        for (int i = threadIdx.x; i < 128; i += blockDim.x) (&red[0][0])[i] = 0.0f;
    pdl_allow_next();
    pdl_wait();
    const int units = p.K / VEC;
    const int64_t g = blockIdx.x / static_cast<unsigned>(p.parts);
    const int64_t part = blockIdx.x % static_cast<unsigned>(p.parts);
    const int64_t chunk = (p.group_rows + p.parts - 1) / p.parts;
    const int64_t first = g * p.group_rows + part * chunk;
    const int64_t last = min((g + 1) * p.group_rows, first + chunk);
    const float inv_k = 1.0f / static_cast<float>(p.K);
    float dw[J][VEC], db[J][VEC];
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) dw[j][i] = db[j][i] = 0.0f;
    if constexpr (!kWarpRow) __syncthreads();  // red cleared
    int turn = 0;
    for (int64_t base = first; base < last; base += slots, turn ^= 1) {
        const int64_t r = base + slot;
        const bool row_ok = r < last;
        Unit<T, VEC> ux[J], ud[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int u = t + p.tpr * j;
            ux[j].clear();
            ud[j].clear();
            if (row_ok && u < units) {
                ux[j].load(static_cast<const T*>(p.x) + r * p.x_stride, u);
                ud[j].load(static_cast<const T*>(p.dy) + r * p.dy_stride, u);
            }
        }
        const float mean = row_ok ? __ldg(p.mean + r) : 0.0f;
        const float rstd = row_ok ? __ldg(p.rstd + r) : 0.0f;
        float acc[2] = {0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < J; ++j) {
            if (row_ok && t + p.tpr * j < units) {
                float x[VEC], d[VEC], w[VEC];
                ux[j].get(x);
                ud[j].get(d);
                if (p.w != nullptr) load_affine<T, VEC>(w, p.w, p.w_f32, g * p.K + (t + p.tpr * j) * VEC);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float xhat = (x[i] - mean) * rstd;
                    dw[j][i] = fmaf(d[i], xhat, dw[j][i]);
                    db[j][i] += d[i];
                    const float h = p.w != nullptr ? d[i] * (w[i] + p.offset) : d[i];
                    acc[0] += h;
                    acc[1] = fmaf(h, xhat, acc[1]);
                }
            }
        }
        if (p.dx != nullptr) {
            row_reduce<kWarpRow, SumOp>(acc, p.tpr, red[turn]);
            const float c1 = acc[0] * inv_k, c2 = acc[1] * inv_k;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                if (row_ok && t + p.tpr * j < units) {
                    float x[VEC], d[VEC], w[VEC];
                    ux[j].get(x);
                    ud[j].get(d);
                    if (p.w != nullptr) load_affine<T, VEC>(w, p.w, p.w_f32, g * p.K + (t + p.tpr * j) * VEC);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        const float xhat = (x[i] - mean) * rstd;
                        const float h = p.w != nullptr ? d[i] * (w[i] + p.offset) : d[i];
                        d[i] = rstd * (h - c1 - xhat * c2);
                    }
                    Unit<T, VEC>::store(static_cast<T*>(p.dx) + r * p.K, t + p.tpr * j, d);
                }
            }
        }
    }
    if (p.part_dw == nullptr && p.part_db == nullptr) return;
    const int64_t out = (g * p.parts + part) * p.K;
    if constexpr (!kWarpRow) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int u = t + p.tpr * j;
            if (u < units) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    if (p.part_dw != nullptr) p.part_dw[out + u * VEC + i] = dw[j][i];
                    if (p.part_db != nullptr) p.part_db[out + u * VEC + i] = db[j][i];
                }
            }
        }
    } else {
        // the rows of one warp by shuffles, then the warps in order
        __shared__ float cols[2][32 * J * VEC];
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                for (int o = p.tpr; o < 32; o <<= 1) {
                    dw[j][i] += __shfl_xor_sync(0xFFFFFFFFu, dw[j][i], o);
                    db[j][i] += __shfl_xor_sync(0xFFFFFFFFu, db[j][i], o);
                }
        const int lane = threadIdx.x & 31;
        for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) {
            if (static_cast<int>(threadIdx.x >> 5) == w && lane < p.tpr) {
#pragma unroll
                for (int j = 0; j < J; ++j)
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        const int c = (t + p.tpr * j) * VEC + i;
                        cols[0][c] = (w == 0 ? 0.0f : cols[0][c]) + dw[j][i];
                        cols[1][c] = (w == 0 ? 0.0f : cols[1][c]) + db[j][i];
                    }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < p.K; c += blockDim.x) {
            if (p.part_dw != nullptr) p.part_dw[out + c] = cols[0][c];
            if (p.part_db != nullptr) p.part_db[out + c] = cols[1][c];
        }
    }
}

// dw[g, c] = sum over i of part_dw[g][i][c], and db likewise: 32 columns per
// CTA, the parts split over its warps and joined in order.  (Bound by latency:
// 7 us for 888 parts of 1536 columns; with 8 warps the backward of 32760 x
// 1536 took 10 us longer.)
constexpr int kPartWarps = 32;
template <typename T>
__global__ void __launch_bounds__(32 * kPartWarps) norm_partials_kernel(const float* part_dw, const float* part_db, int K,
                                                            int parts, int w_f32, void* dw, void* db) {
    __shared__ float sums[kPartWarps][33];
    pdl_allow_next();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned blocks = static_cast<unsigned>(K + 31) / 32;
    const int c = static_cast<int>(blockIdx.x % blocks) * 32 + lane;
    const int64_t g = blockIdx.x / blocks;
    const float* part = blockIdx.y == 0 ? part_dw : part_db;
    void* dst = blockIdx.y == 0 ? dw : db;
    if (part == nullptr) return;
    float s = 0.0f;
    if (c < K) {
        const float* at = part + g * parts * K + c;
#pragma unroll 8
        for (int i = warp; i < parts; i += kPartWarps) s += at[static_cast<int64_t>(i) * K];
    }
    sums[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < K) {
        s = sums[0][lane];
#pragma unroll
        for (int i = 1; i < kPartWarps; ++i) s += sums[i][lane];
        if (w_f32) static_cast<float*>(dst)[g * K + c] = s;
        else static_cast<T*>(dst)[g * K + c] = from_float<T>(s);
    }
}

// ------------------------------------------------- rows through shared memory
// The kernels of wide rows (16-byte units, 33 to 640 threads a row).  Thread t
// owns 16 columns of every row (units t, t + T, ...), whose weight, bias and,
// in the backward, gradient sums stay in its registers while the CTA walks
// consecutive rows.  The rows themselves arrive in a ring of shared-memory
// slots by bulk copies several rows ahead, which keeps enough bytes in flight
// for HBM whatever the CTA is waiting for (loads into registers one row ahead
// reached 2 TB/s on the quantizing norm of 75600 x 5120).
//
// The forward has one barrier per row: a warp forms the sum of its columns, its
// own mean and the squares about that (all by shuffles); the warps' three
// numbers are joined behind the barrier, sum (x - mean)^2 = sum over the warps
// of M2_w + n_w (mean_w - mean)^2, which never subtracts large squares.
// Arithmetic is on pairs (fp32x2 instructions): at some seven instructions per
// value the quantizing form would otherwise be bound by them, not by HBM.
constexpr int kRingCols = 16;     // columns per thread
constexpr int kRingMaxSlots = 8;
constexpr int kRingSmall = 320;   // threads per CTA of the variant with two CTAs' registers per SM
constexpr int kRingLarge = 640;   // ... with one

// A thread's columns as pairs; column pair i is in unit i / (VEC / 2).
template <typename T>
struct RingRow {
    static constexpr int VEC = 16 / sizeof(T);
    static constexpr int J = kRingCols / VEC;
    static constexpr int P = kRingCols / 2;
    __device__ static __forceinline__ void get(float2 (&f)[P], const uint8_t* slot, int t, int threads, int units) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int u = t + threads * j;
            Unit<T, VEC> raw;
            raw.clear();
            if (u < units) raw.raw = reinterpret_cast<const uint4*>(slot)[u];
            float v[VEC];
            raw.get(v);
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) f[j * (VEC / 2) + i] = make_float2(v[2 * i], v[2 * i + 1]);
        }
    }
    __device__ static __forceinline__ void put(const float2 (&f)[P], T* row, int t, int threads, int units) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int u = t + threads * j;
            float v[VEC];
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) {
                v[2 * i] = f[j * (VEC / 2) + i].x;
                v[2 * i + 1] = f[j * (VEC / 2) + i].y;
            }
            if (u < units) Unit<T, VEC>::store(row, u, v);
        }
    }
    // Weight or bias of group g: w + offset, or `missing` without one.
    __device__ static __forceinline__ void affine(float2 (&f)[P], const void* base, bool f32, int64_t at, float offset,
                                                  float missing, int t, int threads, int units) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int u = t + threads * j;
            float v[VEC];
            if (base != nullptr && u < units) load_affine<T, VEC>(v, base, f32, at + static_cast<int64_t>(u) * VEC);
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i)
                f[j * (VEC / 2) + i] = base != nullptr && u < units ? make_float2(v[2 * i] + offset, v[2 * i + 1] + offset)
                                                                   : make_float2(missing, missing);
        }
    }
};

// A warp's bounded wait for a row slot, and what it does after giving up: it
// records that, its thread that issues the copies (if it has one) waits out
// those of the next `in_flight` slots, and the warp leaves its rows.
__device__ __forceinline__ bool ring_wait(uint64_t* full, uint32_t phase) {
    return __all_sync(0xFFFFFFFFu, mbar_wait(full, phase, nullptr));
}
__device__ __forceinline__ void ring_give_up(uint64_t* full, int slot, int slots, uint32_t phase, bool issuer,
                                             int64_t in_flight, uint32_t* err) {
    atomicOr(err, kErrNorm);
    for (int i = 0; issuer && i < slots && i < in_flight; ++i) {
        const bool wrapped = slot + i >= slots;
        mbar_wait(&full[wrapped ? slot + i - slots : slot + i], phase ^ (wrapped ? 1u : 0u), nullptr);
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// A number per warp, zero past the CTA's warps, read whole by every thread.
template <int kMaxThreads>
struct PerWarp {
    static constexpr int kQuads = (kMaxThreads / 32 + 3) / 4;
    float4 v[kQuads];
    __device__ __forceinline__ float& operator[](int i) { return reinterpret_cast<float*>(v)[i]; }
    __device__ __forceinline__ float sum() const {
        float4 q[kQuads];
#pragma unroll
        for (int i = 0; i < kQuads; ++i) q[i] = v[i];
        float2 a = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < kQuads; ++i)
            a = __fadd2_rn(a, __fadd2_rn(make_float2(q[i].x, q[i].y), make_float2(q[i].z, q[i].w)));
        return a.x + a.y;
    }
    __device__ __forceinline__ float max() const {  // of values >= 0
        float4 q[kQuads];
#pragma unroll
        for (int i = 0; i < kQuads; ++i) q[i] = v[i];
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < kQuads; ++i) m = fmaxf(m, fmaxf(fmaxf(q[i].x, q[i].y), fmaxf(q[i].z, q[i].w)));
        return m;
    }
};

template <int kMaxThreads>
struct RingShared {
    PerWarp<kMaxThreads> sum[2], m2[2], amax, count, inv_count;  // count: a warp's columns
    uint64_t full[kRingMaxSlots];
    // sum over the warps of m2 + count (sum / count - mean)^2
    __device__ __forceinline__ float squares(int par, float mean) const {
        float2 a = make_float2(0.0f, 0.0f);
        const float2 neg = make_float2(-mean, -mean);
#pragma unroll
        for (int i = 0; i < PerWarp<kMaxThreads>::kQuads; ++i) {
            const float4 q = sum[par].v[i], n = count.v[i], r = inv_count.v[i], m = m2[par].v[i];
            const float2 d0 = __ffma2_rn(make_float2(q.x, q.y), make_float2(r.x, r.y), neg);
            const float2 d1 = __ffma2_rn(make_float2(q.z, q.w), make_float2(r.z, r.w), neg);
            a = __fadd2_rn(a, __ffma2_rn(__fmul2_rn(make_float2(n.x, n.y), d0), d0, make_float2(m.x, m.y)));
            a = __fadd2_rn(a, __ffma2_rn(__fmul2_rn(make_float2(n.z, n.w), d1), d1, make_float2(m.z, m.w)));
        }
        return a.x + a.y;
    }
};

// kMode: 0 = values out, 1 = codes, 2 = codes of values clamped to +-qmax first
// (qmax is not an E4M3 value).
template <typename T, int kMode, int kMaxThreads>
__global__ void __launch_bounds__(kMaxThreads, kMaxThreads <= kRingSmall ? 2 : 1)
    norm_ring_kernel(const NormArgs p, int slots, uint32_t* err) {
    using Row = RingRow<T>;
    constexpr int P = Row::P, VEC = Row::VEC, J = Row::J;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ RingShared<kMaxThreads> s;
    const int t = threadIdx.x, threads = blockDim.x, warp = t >> 5, lane = t & 31;
    const int units = p.K / VEC;
    const uint32_t row_bytes = static_cast<uint32_t>(p.K * sizeof(T));
    if (t == 0) {
        for (int i = 0; i < slots; ++i) mbar_init(&s.full[i], 1);
        fence_mbar_init();
    }
    int mine = 0;
    bool valid[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        valid[j] = t + threads * j < units;
        mine += valid[j] ? VEC : 0;
    }
    const float n_warp = warp_sum(static_cast<float>(mine));
    const float inv_n_warp = n_warp > 0.0f ? 1.0f / n_warp : 0.0f;
    if (t < 4 * PerWarp<kMaxThreads>::kQuads) {
        s.sum[0][t] = s.sum[1][t] = s.m2[0][t] = s.m2[1][t] = 0.0f;
        s.amax[t] = s.count[t] = s.inv_count[t] = 0.0f;
    }
    __syncthreads();
    if (lane == 0) {
        s.count[warp] = n_warp;
        s.inv_count[warp] = inv_n_warp;
    }
    __syncthreads();
    pdl_allow_next();
    pdl_wait();
    const int64_t chunk = (p.M + gridDim.x - 1) / gridDim.x;
    const int64_t first = blockIdx.x * chunk;
    const int64_t last = min(p.M, first + chunk);
    const auto fetch = [&](int64_t r, int slot) {
        mbar_arrive_expect_tx(&s.full[slot], row_bytes);
        bulk_g2s(ring + static_cast<size_t>(slot) * row_bytes, static_cast<const T*>(p.x) + r * p.x_stride, row_bytes,
                 &s.full[slot]);
    };
    if (t == 0)
        for (int i = 0; i < slots && first + i < last; ++i) fetch(first + i, i);
    const float inv_k = 1.0f / static_cast<float>(p.K);
    int64_t group = -1;
    float2 w[P], b[P];
    int slot = 0;
    uint32_t phase = 0;
    for (int64_t r = first; r < last; ++r) {
        const int64_t g = p.group_rows == p.M ? 0 : static_cast<uint32_t>(r) / static_cast<uint32_t>(p.group_rows);
        if (g != group) {
            group = g;
            Row::affine(w, p.w, p.w_f32, g * p.K, p.offset, 1.0f, t, threads, units);
            Row::affine(b, p.b, p.w_f32, g * p.K, 0.0f, 0.0f, t, threads, units);
#pragma unroll
            for (int i = 0; i < P; ++i)  // a column past the row gives 0, which no maximum sees
                if (!valid[i / (VEC / 2)]) w[i] = make_float2(0.0f, 0.0f);
        }
        if (!ring_wait(&s.full[slot], phase)) {  // the barriers below do not count warps that have left
            ring_give_up(s.full, slot, slots, phase, t == 0, last - r, err);
            break;
        }
        float2 x[P];
        Row::get(x, ring + static_cast<size_t>(slot) * row_bytes, t, threads, units);
        float2 acc = x[0];
#pragma unroll
        for (int i = 1; i < P; ++i) acc = __fadd2_rn(acc, x[i]);
        const float sum_w = warp_sum(acc.x + acc.y);
        const float mean_w = sum_w * inv_n_warp;
        acc = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const float2 d = __fadd2_rn(x[i], make_float2(-mean_w, -mean_w));
            if (valid[i / (VEC / 2)]) acc = __ffma2_rn(d, d, acc);
        }
        const float m2_w = warp_sum(acc.x + acc.y);
        const int par = static_cast<int>(r & 1);
        if (lane == 0) {
            s.sum[par][warp] = sum_w;
            s.m2[par][warp] = m2_w;
        }
        __syncthreads();
        // every thread has its columns: the slot takes the row `slots` further on
        if (t == 0 && r + slots < last) fetch(r + slots, slot);
        const float mean = s.sum[par].sum() * inv_k;
        const float rstd = rsqrtf(fmaf(s.squares(par, mean), inv_k, p.eps));
        if (p.mean != nullptr && t == 0) {
            p.mean[r] = mean;
            p.rstd[r] = rstd;
        }
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const float2 xhat = __fmul2_rn(__fadd2_rn(x[i], make_float2(-mean, -mean)), make_float2(rstd, rstd));
            x[i] = __ffma2_rn(xhat, w[i], b[i]);
        }
        if constexpr (kMode == 0) {
            Row::put(x, static_cast<T*>(p.y) + r * p.K, t, threads, units);
        } else {
            float m = 0.0f;
#pragma unroll
            for (int i = 0; i < P; ++i) m = fmaxf(m, fmaxf(fabsf(x[i].x), fabsf(x[i].y)));
            // non-negative floats compare as their bits do
            const uint32_t m_w = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(m));
            if (lane == 0) s.amax[warp] = __uint_as_float(m_w);
            __syncthreads();
            const float sc = __fdiv_rn(fmaxf(s.amax.max(), 1e-12f), p.qmax);
            if (t == 0) p.s[r] = sc;
            float rcp;  // 1 ulp; with the product's half the quotient is good to 1.5
            asm("rcp.approx.f32 %0, %1;" : "=f"(rcp) : "f"(sc));
#pragma unroll
            for (int i = 0; i < P; ++i) {
                x[i] = __fmul2_rn(x[i], make_float2(rcp, rcp));
                if constexpr (kMode == 2) {
                    x[i].x = fminf(fmaxf(x[i].x, -p.qmax), p.qmax);
                    x[i].y = fminf(fmaxf(x[i].y, -p.qmax), p.qmax);
                }
            }
            uint8_t* out = p.q + r * p.K;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int u = t + threads * j;
                uint32_t c[VEC / 4];
#pragma unroll
                for (int i = 0; i < VEC / 4; ++i) {
                    const float2 lo = x[j * (VEC / 2) + 2 * i], hi = x[j * (VEC / 2) + 2 * i + 1];
                    c[i] = cvt_e4m3x4(lo, hi);
                }
                if (valid[j]) {
                    if constexpr (VEC == 8) reinterpret_cast<uint2*>(out)[u] = make_uint2(c[0], c[1]);
                    else reinterpret_cast<uint32_t*>(out)[u] = c[0];
                }
            }
        }
        if (++slot == slots) {
            slot = 0;
            phase ^= 1u;
        }
    }
}

// Backward through the ring (a slot holds a row of x, then its row of dy); grid
// and partial sums as in norm_backward_kernel.  (Measured on B200, 32760 x 5120
// bf16: 160 us, 6.3 TB/s, bound by HBM; 16384 x 1536 fp16 34 us, 4.5 TB/s,
// start and partial sums included.)
template <typename T, int kMaxThreads>
__global__ void __launch_bounds__(kMaxThreads, kMaxThreads <= kRingSmall ? 2 : 1)
    norm_backward_ring_kernel(const NormArgs p, int slots, uint32_t* err) {
    using Row = RingRow<T>;
    constexpr int P = Row::P, VEC = Row::VEC, J = Row::J;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ uint64_t full[kRingMaxSlots];
    __shared__ PerWarp<kMaxThreads> sums[2][2];
    const int t = threadIdx.x, threads = blockDim.x, warp = t >> 5, lane = t & 31;
    const int units = p.K / VEC;
    const uint32_t row_bytes = static_cast<uint32_t>(p.K * sizeof(T));
    if (t == 0) {
        for (int i = 0; i < slots; ++i) mbar_init(&full[i], 1);
        fence_mbar_init();
    }
    if (t < 4 * PerWarp<kMaxThreads>::kQuads) sums[0][0][t] = sums[0][1][t] = sums[1][0][t] = sums[1][1][t] = 0.0f;
    __syncthreads();
    pdl_allow_next();
    pdl_wait();
    const int64_t g = blockIdx.x / static_cast<unsigned>(p.parts);
    const int64_t part = blockIdx.x % static_cast<unsigned>(p.parts);
    const int64_t chunk = (p.group_rows + p.parts - 1) / p.parts;
    const int64_t first = g * p.group_rows + part * chunk;
    const int64_t last = min((g + 1) * p.group_rows, first + chunk);
    const auto fetch = [&](int64_t r, int slot) {
        mbar_arrive_expect_tx(&full[slot], 2 * row_bytes);
        uint8_t* dst = ring + static_cast<size_t>(slot) * 2 * row_bytes;
        bulk_g2s(dst, static_cast<const T*>(p.x) + r * p.x_stride, row_bytes, &full[slot]);
        bulk_g2s(dst + row_bytes, static_cast<const T*>(p.dy) + r * p.dy_stride, row_bytes, &full[slot]);
    };
    if (t == 0)
        for (int i = 0; i < slots && first + i < last; ++i) fetch(first + i, i);
    const float inv_k = 1.0f / static_cast<float>(p.K);
    float2 w[P], dw[P], db[P];
    Row::affine(w, p.w, p.w_f32, g * p.K, p.offset, 1.0f, t, threads, units);
#pragma unroll
    for (int i = 0; i < P; ++i) dw[i] = db[i] = make_float2(0.0f, 0.0f);
    float mean = first < last ? __ldg(p.mean + first) : 0.0f, rstd = first < last ? __ldg(p.rstd + first) : 0.0f;
    int slot = 0;
    uint32_t phase = 0;
    for (int64_t r = first; r < last; ++r) {
        const float next_mean = r + 1 < last ? __ldg(p.mean + r + 1) : 0.0f;
        const float next_rstd = r + 1 < last ? __ldg(p.rstd + r + 1) : 0.0f;
        if (!ring_wait(&full[slot], phase)) {
            ring_give_up(full, slot, slots, phase, t == 0, last - r, err);
            break;
        }
        const uint8_t* src = ring + static_cast<size_t>(slot) * 2 * row_bytes;
        float2 xhat[P], h[P];
        Row::get(xhat, src, t, threads, units);
        Row::get(h, src + row_bytes, t, threads, units);
        float2 s1 = make_float2(0.0f, 0.0f), s2 = s1;
#pragma unroll
        for (int i = 0; i < P; ++i) {  // past the row dy is 0, and so is h
            xhat[i] = __fmul2_rn(__fadd2_rn(xhat[i], make_float2(-mean, -mean)), make_float2(rstd, rstd));
            dw[i] = __ffma2_rn(h[i], xhat[i], dw[i]);
            db[i] = __fadd2_rn(db[i], h[i]);
            h[i] = __fmul2_rn(h[i], w[i]);
            s1 = __fadd2_rn(s1, h[i]);
            s2 = __ffma2_rn(h[i], xhat[i], s2);
        }
        const float a1 = warp_sum(s1.x + s1.y), a2 = warp_sum(s2.x + s2.y);
        const int par = static_cast<int>(r & 1);
        if (lane == 0) {
            sums[par][0][warp] = a1;
            sums[par][1][warp] = a2;
        }
        __syncthreads();
        if (t == 0 && r + slots < last) fetch(r + slots, slot);
        if (p.dx != nullptr) {
            const float c1 = sums[par][0].sum() * inv_k, c2 = sums[par][1].sum() * inv_k;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const float2 e = __ffma2_rn(xhat[i], make_float2(-c2, -c2), __fadd2_rn(h[i], make_float2(-c1, -c1)));
                h[i] = __fmul2_rn(e, make_float2(rstd, rstd));
            }
            Row::put(h, static_cast<T*>(p.dx) + r * p.K, t, threads, units);
        }
        mean = next_mean;
        rstd = next_rstd;
        if (++slot == slots) {
            slot = 0;
            phase ^= 1u;
        }
    }
    const int64_t out = (g * p.parts + part) * p.K;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int u = t + threads * j;
        if (u >= units) continue;
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i) {
            const float2 lo = dw[j * (VEC / 2) + 2 * i], hi = dw[j * (VEC / 2) + 2 * i + 1];
            if (p.part_dw != nullptr)
                reinterpret_cast<float4*>(p.part_dw + out)[u * (VEC / 4) + i] = make_float4(lo.x, lo.y, hi.x, hi.y);
            const float2 lo2 = db[j * (VEC / 2) + 2 * i], hi2 = db[j * (VEC / 2) + 2 * i + 1];
            if (p.part_db != nullptr)
                reinterpret_cast<float4*>(p.part_db + out)[u * (VEC / 4) + i] = make_float4(lo2.x, lo2.y, hi2.x, hi2.y);
        }
    }
}

// ------------------------------------------------- one or two warps per row
// Many wide rows (16-byte units, K up to 64 * 80): a row is held as fp32 pairs by
// W warps (1 or 2), C columns a lane, so that the sums are shuffles and at most
// one barrier of two warps joins them; a row costs some 1500 instructions of a
// warp (those of the ring above 4000).  The weight (with its offset) and bias
// lie in shared memory as fp32, which every row of the CTA reads.  Each row's
// warps have one or two row slots of their own and copy the next rows into
// them while they work on the present one.  A CTA stays within one group.
// (Measured on B200, 75600 x 5120 bf16 to codes: 231 us, 5.0 TB/s; the ring
// 394 us; W = 1, C = 160, with spills, 270 us.  32760 x 5120 to values 118 us,
// 5.7 TB/s.  Bound by instruction issue and HBM together.)
constexpr int kRowWarps = 16;  // warps per CTA, one CTA per SM

__device__ __forceinline__ float max3_abs(float a, float b, float c) {
    float d;
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

template <typename T, bool kQuant, int C, int W>
__global__ void __launch_bounds__(32 * kRowWarps, 1) norm_rows_kernel(const NormArgs p, int slots, uint32_t* err) {
    constexpr int VEC = 16 / sizeof(T), J = C / VEC, P = C / 2, R = kRowWarps / W;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t full[R][2];
    __shared__ float joined[2][R][W][2];
    __shared__ uint32_t joined_max[R][W];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int row = warp / W, sub = warp % W, place = sub * 32 + lane;  // of the CTA's rows; of the row's threads
    const int units = p.K / VEC;
    const uint32_t row_bytes = static_cast<uint32_t>(p.K * sizeof(T));
    // weight + offset, then bias, each quad q of a 16-byte unit in a plane of its
    // own, so that a warp's accesses are consecutive
    float4* sw = reinterpret_cast<float4*>(smem);
    float4* sb = sw + p.K / 4;
    uint8_t* ring = smem + 8 * static_cast<size_t>(p.K) + static_cast<size_t>(row * slots) * row_bytes;
    if (place == 0) {
        mbar_init(&full[row][0], 1);
        mbar_init(&full[row][1], 1);
        fence_mbar_init();
    }
    pdl_allow_next();
    pdl_wait();
    const int64_t g = blockIdx.x / static_cast<unsigned>(p.parts);
    const int64_t part = blockIdx.x % static_cast<unsigned>(p.parts);
    // the group's rows, dealt to its parts * R rows at a time in turn
    const int64_t first = g * p.group_rows + part * R + row, last = (g + 1) * p.group_rows;
    const int64_t step = static_cast<int64_t>(p.parts) * R;
    const auto fetch = [&](int64_t r, int slot) {
        mbar_arrive_expect_tx(&full[row][slot], row_bytes);
        bulk_g2s(ring + slot * row_bytes, static_cast<const T*>(p.x) + r * p.x_stride, row_bytes, &full[row][slot]);
    };
    if (place == 0)
        for (int i = 0; i < slots && first + i * step < last; ++i) fetch(first + i * step, i);
    for (int c = t; c < p.K; c += 32 * kRowWarps) {
        const int64_t at = g * p.K + c;
        float w[1] = {1.0f}, b[1] = {0.0f};
        if (p.w != nullptr) {
            load_affine<T, 1>(w, p.w, p.w_f32, at);
            w[0] += p.offset;
        }
        if (p.b != nullptr) load_affine<T, 1>(b, p.b, p.w_f32, at);
        const int to = ((c % VEC / 4) * units + c / VEC) * 4 + c % 4;
        reinterpret_cast<float*>(sw)[to] = w[0];
        reinterpret_cast<float*>(sb)[to] = b[0];
    }
    bool valid[J];
    int mine = 0;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        valid[j] = place + 32 * W * j < units;
        mine += valid[j] ? VEC : 0;
    }
    // columns of this warp and of the row's other one
    const float n_warp = warp_sum(static_cast<float>(mine)), n_other = static_cast<float>(p.K) - n_warp;
    const float inv_n_warp = n_warp > 0.0f ? 1.0f / n_warp : 0.0f, inv_n_other = n_other > 0.0f ? 1.0f / n_other : 0.0f;
    __syncthreads();
    const auto row_sync = [&]() {
        if constexpr (W == 1) __syncwarp();
        else named_bar_sync(1 + row, 32 * W);
    };
    const float inv_k = 1.0f / static_cast<float>(p.K);
    int slot = 0, par = 0;
    uint32_t phase = 0;
    for (int64_t r = first; r < last; r += step, par ^= 1) {
        if (!ring_wait(&full[row][slot], phase)) {
            ring_give_up(full[row], slot, slots, phase, place == 0, r + step < last ? 2 : 1, err);
            if constexpr (W == 2) {  // the row's other warp is or will be at its barrier: it leaves too
                if (lane == 0) joined[par][row][sub][1] = -1.0f;
                row_sync();
            }
            break;
        }
        float2 x[P];
        const uint4* src = reinterpret_cast<const uint4*>(ring + slot * row_bytes);
#pragma unroll
        for (int j = 0; j < J; ++j) {
            Unit<T, VEC> raw;
            raw.clear();
            if (valid[j]) raw.raw = src[place + 32 * W * j];
            float v[VEC];
            raw.get(v);
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) x[j * (VEC / 2) + i] = make_float2(v[2 * i], v[2 * i + 1]);
        }
        float2 a0 = x[0], a1 = x[1];
#pragma unroll
        for (int i = 2; i < P; i += 2) {
            a0 = __fadd2_rn(a0, x[i]);
            a1 = __fadd2_rn(a1, x[i + 1]);
        }
        a0 = __fadd2_rn(a0, a1);
        const float sum_w = warp_sum(a0.x + a0.y);
        const float mean_w = sum_w * inv_n_warp;
        a0 = a1 = make_float2(0.0f, 0.0f);
        const float2 neg_w = make_float2(-mean_w, -mean_w);
#pragma unroll
        for (int j = 0; j < J; ++j) {
#pragma unroll
            for (int i = j * (VEC / 2); i < (j + 1) * (VEC / 2); i += 2) {
                const float2 d0 = __fadd2_rn(x[i], neg_w), d1 = __fadd2_rn(x[i + 1], neg_w);
                if (valid[j]) {
                    a0 = __ffma2_rn(d0, d0, a0);
                    a1 = __ffma2_rn(d1, d1, a1);
                }
            }
        }
        a0 = __fadd2_rn(a0, a1);
        float m2 = warp_sum(a0.x + a0.y), mean = mean_w;
        if constexpr (W == 2) {
            if (lane == 0) {
                joined[par][row][sub][0] = sum_w;
                joined[par][row][sub][1] = m2;
            }
            row_sync();
            if (joined[par][row][sub ^ 1][1] < 0.0f) {  // no sum of squares: the other warp gave up
                ring_give_up(full[row], slot, slots, phase, place == 0, r + step < last ? 2 : 1, err);
                break;
            }
            // both warps get the same bits: the terms are added in the warps' order
            const float s0 = joined[par][row][0][0], s1 = joined[par][row][1][0];
            mean = (s0 + s1) * inv_k;
            const float n0 = sub == 0 ? n_warp : n_other, n1 = sub == 0 ? n_other : n_warp;
            const float d0 = fmaf(s0, sub == 0 ? inv_n_warp : inv_n_other, -mean);
            const float d1 = fmaf(s1, sub == 0 ? inv_n_other : inv_n_warp, -mean);
            m2 = fmaf(n0 * d0, d0, joined[par][row][0][1]) + fmaf(n1 * d1, d1, joined[par][row][1][1]);
        } else {
            row_sync();
        }
        // every lane has its columns: the slot takes the row `slots` steps on
        if (place == 0 && r + slots * step < last) fetch(r + slots * step, slot);
        const float rstd = rsqrtf(fmaf(m2, inv_k, p.eps));
        if (p.mean != nullptr && place == 0) {
            p.mean[r] = mean;
            p.rstd[r] = rstd;
        }
        const float2 rs = make_float2(rstd, rstd), neg = make_float2(-mean, -mean);
        float m0 = 0.0f, m1 = 0.0f;
#pragma unroll
        for (int j = 0; j < J; ++j) {
#pragma unroll
            for (int q = 0; q < VEC / 4; ++q) {
                const int i = j * (VEC / 2) + 2 * q, at = q * units + place + 32 * W * j;
                float4 w = make_float4(0.0f, 0.0f, 0.0f, 0.0f), b = w;
                if (valid[j]) {
                    w = sw[at];
                    b = sb[at];
                }
                x[i] = __ffma2_rn(__fmul2_rn(__fadd2_rn(x[i], neg), rs), make_float2(w.x, w.y), make_float2(b.x, b.y));
                x[i + 1] = __ffma2_rn(__fmul2_rn(__fadd2_rn(x[i + 1], neg), rs), make_float2(w.z, w.w),
                                      make_float2(b.z, b.w));
                if constexpr (kQuant) {
                    m0 = max3_abs(m0, x[i].x, x[i].y);
                    m1 = max3_abs(m1, x[i + 1].x, x[i + 1].y);
                }
            }
        }
        if constexpr (!kQuant) {
            T* out = static_cast<T*>(p.y) + r * p.K;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                float v[VEC];
#pragma unroll
                for (int i = 0; i < VEC / 2; ++i) {
                    v[2 * i] = x[j * (VEC / 2) + i].x;
                    v[2 * i + 1] = x[j * (VEC / 2) + i].y;
                }
                if (valid[j]) Unit<T, VEC>::store(out, place + 32 * W * j, v);
            }
        } else {
            // non-negative floats compare as their bits do
            uint32_t bits = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(fmaxf(m0, m1)));
            if constexpr (W == 2) {
                if (lane == 0) joined_max[row][sub] = bits;
                row_sync();
                bits = max(joined_max[row][0], joined_max[row][1]);
            }
            const float sc = __fdiv_rn(fmaxf(__uint_as_float(bits), 1e-12f), p.qmax);
            if (place == 0) p.s[r] = sc;
            float rcp;  // 1 ulp; with the product's half the quotient is good to 1.5
            asm("rcp.approx.f32 %0, %1;" : "=f"(rcp) : "f"(sc));
            const float2 rc = make_float2(rcp, rcp);
            uint8_t* out = p.q + r * p.K;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                uint32_t c[VEC / 4];
#pragma unroll
                for (int q = 0; q < VEC / 4; ++q) {
                    const int i = j * (VEC / 2) + 2 * q;
                    c[q] = cvt_e4m3x4(__fmul2_rn(x[i], rc), __fmul2_rn(x[i + 1], rc));
                }
                const int u = place + 32 * W * j;
                if (valid[j]) {
                    if constexpr (VEC == 8) reinterpret_cast<uint2*>(out)[u] = make_uint2(c[0], c[1]);
                    else reinterpret_cast<uint32_t*>(out)[u] = c[0];
                }
            }
        }
        if (++slot == slots) {
            slot = 0;
            phase ^= 1u;
        }
    }
}

// ------------------------------------------------- launch shapes
struct NormShape {
    bool vec;   // 16-byte units
    int j;      // units per thread
    int tpr;    // threads per row
    int block;  // threads per CTA
};

// Threads per row: a power of two up to 32 where J = 2 units each cover the
// row, else whole warps; J = 2, or more where a row needs over 512 threads.
NormShape norm_shape(int64_t K, int elem, bool vec) {
    const int units = static_cast<int>(vec ? K * elem / 16 : K);
    if (units <= 64) {
        int tpr = 1;
        while (2 * tpr < units) tpr *= 2;
        return {vec, 2, tpr, 256};
    }
    for (int j : {2, 4, 8}) {
        if (j == 4 && !vec) continue;
        const int tpr = ((units + j - 1) / j + 31) / 32 * 32;
        if (tpr <= (j <= 4 ? 512 : 1024)) return {vec, j, tpr, tpr};
    }
    return {vec, 32, 1024, 1024};  // scalar units, K <= TFQ_NORM_MAX_K
}

tfq_status launch_error(const char* what, cudaError_t e) {
    if (e == cudaSuccess) e = cudaGetLastError();
    return e == cudaSuccess ? TFQ_OK : fail(TFQ_ECUDA, "%s launch: %s", what, cudaGetErrorString(e));
}

using NormKernel = void (*)(const NormArgs);
using RingKernel = void (*)(const NormArgs, int, uint32_t*);

// The ring kernels' shape for rows of K elements (0 threads: not for them).
struct RingShape {
    int threads;
    int per_sm;  // CTAs per SM by registers
    int slots;
    size_t smem;
};

RingShape ring_shape(int64_t K, int elem, bool vec, int rows_per_slot) {
    const int threads = static_cast<int>((K + kRingCols - 1) / kRingCols + 31) / 32 * 32;
    if (!vec || threads <= 32 || threads > kRingLarge) return {0, 0, 0, 0};
    const int64_t slot = K * elem * rows_per_slot;
    // At 96 registers five warps fit each of the SM's four schedulers.  (A grid
    // for 21 ran a second wave: 32760 x 1536 backward 71 us against 62.)
    const int per_sm = std::min(10, std::max(1, 20 / (threads / 32)));
    // about 144 KB of rows in flight per SM
    const int slots = static_cast<int>(std::max<int64_t>(2, std::min<int64_t>(kRingMaxSlots, 144 * 1024 / (slot * per_sm))));
    return {threads, per_sm, slots, static_cast<size_t>(slot * slots)};
}

template <typename T, bool kQuant>
NormKernel forward_kernel(const NormShape& s) {
    constexpr int V = 16 / sizeof(T);
    if (s.vec) {
        if (s.block == 256 && s.tpr <= 32) return norm_forward_kernel<T, V, 2, true, kQuant>;
        // between these and the longest rows lie the ring's
        constexpr int kMid = sizeof(T) == 4 ? 2 : 4;
        return s.j == kMid ? norm_forward_kernel<T, V, kMid, false, kQuant> : norm_forward_kernel<T, V, 8, false, kQuant>;
    }
    if (s.block == 256 && s.tpr <= 32) return norm_forward_kernel<T, 1, 2, true, kQuant>;
    if (s.j == 2) return norm_forward_kernel<T, 1, 2, false, kQuant>;
    return s.j == 8 ? norm_forward_kernel<T, 1, 8, false, kQuant> : norm_forward_kernel<T, 1, 32, false, kQuant>;
}

template <typename T>
NormKernel backward_kernel(const NormShape& s) {
    constexpr int V = 16 / sizeof(T);
    if (s.vec) {
        if (s.block == 256 && s.tpr <= 32) return norm_backward_kernel<T, V, 2, true>;
        constexpr int kMid = sizeof(T) == 4 ? 2 : 4;
        return s.j == kMid ? norm_backward_kernel<T, V, kMid, false> : norm_backward_kernel<T, V, 8, false>;
    }
    if (s.block == 256 && s.tpr <= 32) return norm_backward_kernel<T, 1, 2, true>;
    if (s.j == 2) return norm_backward_kernel<T, 1, 2, false>;
    return s.j == 8 ? norm_backward_kernel<T, 1, 8, false> : norm_backward_kernel<T, 1, 32, false>;
}

template <typename T>
RingKernel ring_forward(bool quant, bool clamp, bool small) {
    if (clamp) return small ? norm_ring_kernel<T, 2, kRingSmall> : norm_ring_kernel<T, 2, kRingLarge>;
    if (quant) return small ? norm_ring_kernel<T, 1, kRingSmall> : norm_ring_kernel<T, 1, kRingLarge>;
    return small ? norm_ring_kernel<T, 0, kRingSmall> : norm_ring_kernel<T, 0, kRingLarge>;
}
template <typename T>
RingKernel ring_backward(bool small) {
    return small ? norm_backward_ring_kernel<T, kRingSmall> : norm_backward_ring_kernel<T, kRingLarge>;
}

// The kernels of one or two warps per row: up to 80 columns a lane.
struct RowsShape {
    RingKernel kernel;  // null: not for these rows
    int rows;           // rows per CTA at a time
    int slots;
    size_t smem;
};
constexpr int kRingSmem = 160 * 1024;
constexpr int kRowsSmem = 226 * 1024;
constexpr int kRowsMaxK = 64 * 80;

template <typename T, bool kQuant>
RowsShape rows_shape(int64_t K) {
    RowsShape s = {nullptr, K <= 32 * 80 ? kRowWarps : kRowWarps / 2, 2, 0};
    const int64_t row = K * sizeof(T);
    if (8 * K + s.rows * 2 * row > kRowsSmem) s.slots = 1;
    s.smem = static_cast<size_t>(8 * K + s.rows * s.slots * row);
    if (s.smem > kRowsSmem || K > kRowsMaxK) return s;
    s.kernel = K <= 32 * 32   ? norm_rows_kernel<T, kQuant, 32, 1>
               : K <= 32 * 48 ? norm_rows_kernel<T, kQuant, 48, 1>
               : K <= 32 * 64 ? norm_rows_kernel<T, kQuant, 64, 1>
               : K <= 32 * 80 ? norm_rows_kernel<T, kQuant, 80, 1>
               : K <= 64 * 48 ? norm_rows_kernel<T, kQuant, 48, 2>
               : K <= 64 * 64 ? norm_rows_kernel<T, kQuant, 64, 2>
                              : norm_rows_kernel<T, kQuant, 80, 2>;
    return s;
}

// Opt-in shared memory of the kernels with row slots (once per device).
template <typename T>
cudaError_t ring_attributes_of() {
    cudaError_t e = cudaSuccess;
    for (bool small : {true, false}) {
        const RingKernel k[4] = {ring_forward<T>(false, false, small), ring_forward<T>(true, false, small),
                                 ring_forward<T>(true, true, small), ring_backward<T>(small)};
        for (RingKernel f : k)
            if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingSmem);
    }
    for (int K : {32 * 32, 32 * 48, 32 * 64, 32 * 80, 64 * 48, 64 * 64, 64 * 80}) {
        const RingKernel k[2] = {rows_shape<T, false>(K).kernel, rows_shape<T, true>(K).kernel};
        for (RingKernel f : k)
            if (e == cudaSuccess && f != nullptr)
                e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kRowsSmem);
    }
    return e;
}
tfq_status ring_attributes(DeviceState* ds) {
    return once_per_device(ds->norm_attr_set, [] {
        cudaError_t e = ring_attributes_of<float>();
        if (e == cudaSuccess) e = ring_attributes_of<__half>();
        if (e == cudaSuccess) e = ring_attributes_of<__nv_bfloat16>();
        return e;
    });
}

int elem_size(int dtype) { return dtype == TFQ_DTYPE_FP32 ? 4 : 2; }

// The vector form needs every row of every operand on a 16-byte boundary.
bool rows_aligned(const void* p, int64_t stride, int elem) { return p == nullptr || (aligned16(p) && stride * elem % 16 == 0); }

bool norm_vector_ok(const NormCall& c, const void* out, int64_t out_elem) {
    const int e = elem_size(c.dtype);
    const int we = elem_size(c.w_dtype);
    return c.K * e % 16 == 0 && rows_aligned(c.x, c.x_stride, e) && rows_aligned(c.w, c.K, we) &&
           rows_aligned(c.b, c.K, we) && (out == nullptr || aligned16(out)) && out_elem * c.K % 4 == 0;
}

NormArgs norm_args(const NormCall& c, const NormShape& s) {
    NormArgs a = {};
    a.x = c.x;
    a.x_stride = c.x_stride;
    a.w = c.w;
    a.b = c.b;
    a.w_f32 = c.w_dtype == TFQ_DTYPE_FP32;
    a.offset = c.offset;
    a.M = c.M;
    a.group_rows = c.M / c.groups;
    a.K = static_cast<int>(c.K);
    a.tpr = s.tpr;
    a.eps = c.eps;
    a.mean = c.mean;
    a.rstd = c.rstd;
    return a;
}

// CTAs per SM worth launching: about 1536 threads.
int64_t norm_grid(const NormShape& s, int64_t rows, int sm_count) {
    const int64_t slots = s.block / s.tpr;
    return std::min<int64_t>((rows + slots - 1) / slots, static_cast<int64_t>(sm_count) * std::max(1, 1536 / s.block));
}

}  // namespace

// Row shares per group of the kernels of one or two warps per row: of one to four
// waves of a CTA per SM the number whose turns of `at_once` rows, times the waves,
// are fewest, a CTA's start counting as two of them.  (One wave alone, its shares
// rounded down, left 68 SMs without work at 80 groups.  Us, that and this: 32768 x
// 1536, 4 groups 39, 39, 50 groups 46, 45, 80 54, 45, 149 61, 54; 32768 x 5120, 80
// groups 170, 138, 110 128, 132, 149 188, 167; to codes 80 groups 183, 140.)
static int64_t rows_parts(int64_t rows, int64_t groups, int at_once, int sms) {
    int64_t best = 1, least = INT64_MAX;
    for (int waves = 1; waves <= 4; ++waves) {
        const int64_t n = std::max<int64_t>(1, std::min<int64_t>(rows / at_once, static_cast<int64_t>(sms) * waves / groups));
        const int64_t cost = (groups * n + sms - 1) / sms * ((rows + n * at_once - 1) / (n * at_once) + 2);
        if (cost < least) {
            least = cost;
            best = n;
        }
    }
    return best;
}

tfq_status launch_layer_norm(const NormCall& c, void* y, uint8_t* q, float* s, float qmax, cudaStream_t stream,
                             DeviceState* ds) {
    const int e = elem_size(c.dtype);
    const NormShape sh = norm_shape(c.K, e, norm_vector_ok(c, q != nullptr ? q : y, q != nullptr ? 1 : e));
    NormArgs a = norm_args(c, sh);
    a.y = y;
    a.q = q;
    a.s = s;
    a.qmax = qmax;
    a.clamp = q != nullptr && !is_e4m3_value(qmax);
    const RingShape ring = ring_shape(c.K, e, sh.vec, 1);
    // One or two warps per row where every SM has rows for all of its warps twice
    // over, and every group some too (fewer rows finish sooner with a CTA each:
    // 8 x 5120 to codes 6.2 us against 8.1); a qmax that needs a clamp goes
    // with the ring.
    if (ring.threads > 0 && a.clamp == 0 && c.M >= 2 * kRowWarps * ds->sm_count && c.M / c.groups >= 4 * kRowWarps) {
        RowsShape rows;
        if (c.dtype == TFQ_DTYPE_FP32) rows = q ? rows_shape<float, true>(c.K) : rows_shape<float, false>(c.K);
        else if (c.dtype == TFQ_DTYPE_FP16) rows = q ? rows_shape<__half, true>(c.K) : rows_shape<__half, false>(c.K);
        else rows = q ? rows_shape<__nv_bfloat16, true>(c.K) : rows_shape<__nv_bfloat16, false>(c.K);
        if (rows.kernel != nullptr) {
            const tfq_status st = ring_attributes(ds);
            if (st != TFQ_OK) return st;
            a.parts = static_cast<int>(rows_parts(c.M / c.groups, c.groups, rows.rows, ds->sm_count));
            return launch_error("layer norm", launch_kernel(rows.kernel, dim3(static_cast<unsigned>(a.parts * c.groups)),
                                                            dim3(32 * kRowWarps), rows.smem, stream, a, rows.slots,
                                                            ds->err_word));
        }
    }
    if (ring.threads > 0) {
        const bool small = ring.threads <= kRingSmall;
        RingKernel rk;
        if (c.dtype == TFQ_DTYPE_FP32) rk = ring_forward<float>(q != nullptr, a.clamp != 0, small);
        else if (c.dtype == TFQ_DTYPE_FP16) rk = ring_forward<__half>(q != nullptr, a.clamp != 0, small);
        else rk = ring_forward<__nv_bfloat16>(q != nullptr, a.clamp != 0, small);
        const tfq_status st = ring_attributes(ds);
        if (st != TFQ_OK) return st;
        const int64_t grid = std::min<int64_t>(c.M, static_cast<int64_t>(ds->sm_count) * ring.per_sm);
        return launch_error("layer norm", launch_kernel(rk, dim3(static_cast<unsigned>(grid)), dim3(ring.threads),
                                                        ring.smem, stream, a, ring.slots, ds->err_word));
    }
    NormKernel k;
    if (c.dtype == TFQ_DTYPE_FP32) k = q ? forward_kernel<float, true>(sh) : forward_kernel<float, false>(sh);
    else if (c.dtype == TFQ_DTYPE_FP16) k = q ? forward_kernel<__half, true>(sh) : forward_kernel<__half, false>(sh);
    else k = q ? forward_kernel<__nv_bfloat16, true>(sh) : forward_kernel<__nv_bfloat16, false>(sh);
    return launch_error("layer norm", launch_kernel(k, dim3(static_cast<unsigned>(norm_grid(sh, c.M, ds->sm_count))),
                                                    dim3(sh.block), 0, stream, a));
}

// Row shares per group of the backward.  The CTAs run in whole waves of the GPU's
// places: of one to four waves the number is taken whose rows per CTA, times the
// waves, are fewest (a few CTAs more than a wave run alone behind it: 32760 x
// 5120 in 5 groups, 300 CTAs on 296 places, took 244 us, 295 take 160).  A CTA's
// partial sums count as kPartRows rows.
constexpr int kNormMaxSms = 160;  // the workspace formula knows no device: more SMs add no parts
constexpr int kNormSms = 148;     // B200: the waves are chosen for it, whatever the device has
constexpr int kPartRows = 4;
static int64_t backward_parts(int64_t M, int64_t K, int64_t groups, int elem, bool vec, int sm_count) {
    const NormShape s = norm_shape(K, elem, vec);
    const RingShape ring = ring_shape(K, elem, vec, 2);
    const int64_t slots = ring.threads > 0 ? 1 : s.block / s.tpr;
    const int per_sm = ring.threads > 0 ? ring.per_sm : std::max(1, std::min(8, 1024 / s.block));
    const int64_t rows = M / groups, most = (rows + slots - 1) / slots;
    const auto parts = [&](int sms, int waves) {
        return std::max<int64_t>(1, std::min<int64_t>(most, static_cast<int64_t>(sms) * per_sm * waves / groups));
    };
    int best = 1;
    int64_t least = INT64_MAX;
    for (int waves = 1; waves <= 4; ++waves) {
        const int64_t n = parts(kNormSms, waves), places = static_cast<int64_t>(kNormSms) * per_sm;
        const int64_t cost = (groups * n + places - 1) / places * ((rows + n - 1) / n + kPartRows);
        if (cost < least) {
            least = cost;
            best = waves;
        }
    }
    return parts(std::min(sm_count, kNormMaxSms), best);
}

int64_t layer_norm_backward_workspace(int64_t M, int64_t K, int64_t groups) {
    int64_t parts = 1;  // the most that any type and alignment of the operands takes
    for (int e : {2, 4})
        for (bool vec : {true, false}) parts = std::max(parts, backward_parts(M, K, groups, e, vec, kNormMaxSms));
    return 2 * groups * parts * K * 4;
}

tfq_status launch_layer_norm_backward(const NormCall& c, const void* dy, int64_t dy_stride, void* dx, void* dw,
                                      void* db, float* workspace, cudaStream_t stream, DeviceState* ds) {
    const int e = elem_size(c.dtype);
    const bool vec = norm_vector_ok(c, dx, e) && rows_aligned(dy, dy_stride, e);
    const NormShape sh = norm_shape(c.K, e, vec);
    NormArgs a = norm_args(c, sh);
    a.dy = dy;
    a.dy_stride = dy_stride;
    a.dx = dx;
    const RingShape ring = ring_shape(c.K, e, vec, 2);
    a.parts = static_cast<int>(backward_parts(c.M, c.K, c.groups, e, vec, ds->sm_count));
    const int64_t n = c.groups * a.parts * c.K;
    a.part_dw = dw != nullptr ? workspace : nullptr;
    a.part_db = db != nullptr ? workspace + (dw != nullptr ? n : 0) : nullptr;
    const dim3 grid(static_cast<unsigned>(a.parts * c.groups));
    tfq_status st;
    if (ring.threads > 0) {
        const bool small = ring.threads <= kRingSmall;
        RingKernel rk = c.dtype == TFQ_DTYPE_FP32 ? ring_backward<float>(small)
                        : c.dtype == TFQ_DTYPE_FP16 ? ring_backward<__half>(small) : ring_backward<__nv_bfloat16>(small);
        st = ring_attributes(ds);
        if (st != TFQ_OK) return st;
        st = launch_error("layer norm backward", launch_kernel(rk, grid, dim3(ring.threads), ring.smem, stream, a,
                                                               ring.slots, ds->err_word));
    } else {
        NormKernel k = c.dtype == TFQ_DTYPE_FP32 ? backward_kernel<float>(sh)
                       : c.dtype == TFQ_DTYPE_FP16 ? backward_kernel<__half>(sh) : backward_kernel<__nv_bfloat16>(sh);
        st = launch_error("layer norm backward", launch_kernel(k, grid, dim3(sh.block), 0, stream, a));
    }
    if (st != TFQ_OK || (dw == nullptr && db == nullptr)) return st;
    auto join = c.dtype == TFQ_DTYPE_FP32 ? norm_partials_kernel<float>
                : c.dtype == TFQ_DTYPE_FP16 ? norm_partials_kernel<__half> : norm_partials_kernel<__nv_bfloat16>;
    const dim3 jgrid(static_cast<unsigned>((c.K + 31) / 32 * c.groups), 2);
    return launch_error("layer norm gradient", launch_kernel(join, jgrid, dim3(32 * kPartWarps), 0, stream,
                                                             const_cast<const float*>(a.part_dw),
                                                             const_cast<const float*>(a.part_db), a.K, a.parts,
                                                             a.w_f32, dw, db));
}

}  // namespace tfq
