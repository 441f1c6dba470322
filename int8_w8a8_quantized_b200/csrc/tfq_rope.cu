// tfq_rope.cu -- rotary positions with several axes (time, height, width, ...)
// on the queries and keys of an attention layer, in one launch.
//
// Rotated pair i of a head (i < P) belongs to one axis of the token's
// position: angle = position[axis[i]] * inv_freq[i], and
//   (a, b) -> (a cos - b sin, a sin + b cos)
// with (a, b) = elements (2 i, 2 i + 1) or (i, P + i) of the head; elements
// from 2 P on are copied.  The inverse rotation (sin negated) is the
// operator's gradient: a rotation's transpose is its inverse.
//
// Positions reach millions of turns, where an fp32 angle has lost its
// fraction: the angle is formed in fp64 as position * (inv_freq / 2 pi), its
// whole turns are dropped there, and the fraction goes to fp32 for sincospi
// (what that rounding takes off is put back for fp32 outputs).  That costs one
// fp64 product per token and pair, not per element.
//
// Bound by HBM: every element is read and written once.  A CTA takes a few
// tokens; its threads form the tokens' cos/sin table in shared memory (one
// or a few entries each), then stream the heads: a thread stays at one place
// within the head, so it finds its place once and keeps four heads' loads in
// flight.  (Measured on B200: 75600 tokens, 40 + 40 heads of 128 bf16 516 us,
// 6.0 TB/s; 6889 tokens, 28 + 4 heads fp16 25 us, 4.5 TB/s, start and end of
// a launch weighing more; 7 tokens 2.5 us in a graph.)
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "tfq_internal.h"
#include "tfq_ptx.cuh"
#include "tfq_quant_common.cuh"

namespace tfq {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeBytes = 96 * 1024;  // heads of a CTA's tokens
constexpr int kRopeSpread = 8;         // CTAs per SM where there are tokens for them

struct RopeArgs {
    RopeTensor q, k;
    int64_t M;
    int D;
    int pairs;
    int items;       // places within a head: units of the rotated part, then of the copied part
    int rot_items;   // the first of them that rotate
    int head_lanes;  // heads of one token processed at a time
    int tokens;      // tokens per CTA
    int inverse;
    const void* pos;
    int pos64;
    int64_t pos_row_stride, pos_axis_stride;
    double inv_turn[TFQ_ROPE_MAX_PAIRS];  // inv_freq / (2 pi)
    uint8_t axis[TFQ_ROPE_MAX_PAIRS];
};

template <typename T, int VEC>
struct Chunk {  // VEC elements of T, moved as one 16-byte access (VEC > 1) or one element
    using Raw = std::conditional_t<VEC == 1, T, uint4>;
    Raw raw;
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (VEC == 1) {
            raw = *p;
        } else {  // not the read-only path: the call may be in place
            asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(raw.x), "=r"(raw.y), "=r"(raw.z), "=r"(raw.w)
                         : "l"(p));
        }
    }
    __device__ __forceinline__ void store(T* p) const {
        if constexpr (VEC == 1) *p = raw;
        else *reinterpret_cast<uint4*>(p) = raw;
    }
    __device__ __forceinline__ void get(float (&f)[VEC]) const {
        const T* e = reinterpret_cast<const T*>(&raw);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            if constexpr (sizeof(T) == 4) f[i] = e[i];
            else if constexpr (std::is_same_v<T, __half>) f[i] = __half2float(e[i]);
            else f[i] = __bfloat162float(e[i]);
        }
    }
    __device__ __forceinline__ void set(const float (&f)[VEC]) {
        T* e = reinterpret_cast<T*>(&raw);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            if constexpr (sizeof(T) == 4) e[i] = f[i];
            else if constexpr (std::is_same_v<T, __half>) e[i] = __float2half_rn(f[i]);
            else e[i] = __float2bfloat16_rn(f[i]);
        }
    }
};

// kHalves: an item is the VEC elements at i and their partners at P + i, else
// VEC consecutive elements (VEC / 2 pairs), two single ones in the form
// without alignment (VEC == 1).  A thread has one place within a head and
// walks (token, head) pairs, kBatch of them in flight; the first batch's loads
// are issued before the table is formed.
template <typename T, int VEC, bool kHalves>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs p) {
    constexpr bool kTwo = kHalves || VEC == 1;  // an item is two chunks
    constexpr int kPairs = kTwo ? VEC : VEC / 2;
    constexpr int kBatch = 4;
    extern __shared__ float2 table[];           // [tokens][pairs] (cos, sin)
    pdl_allow_next();
    pdl_wait();
    const int64_t m0 = static_cast<int64_t>(blockIdx.x) * p.tokens;
    const int here = static_cast<int>(min(static_cast<int64_t>(p.tokens), p.M - m0));
    const int heads = p.q.heads + p.k.heads;
    const int per_token = p.items * p.head_lanes;
    const int slot = threadIdx.x / per_token;
    const int slots = kRopeThreads / per_token;
    const int in_token = threadIdx.x - slot * per_token;
    const int h0 = in_token / p.items;
    const int item = in_token - h0 * p.items;
    const bool rotates = item < p.rot_items;
    // element offsets of the item's chunks within a head
    int o0, o1;
    if (!rotates) {
        o0 = o1 = 2 * p.pairs + (item - p.rot_items) * VEC;
    } else if constexpr (kHalves) {
        o0 = item * VEC;
        o1 = p.pairs + o0;
    } else if constexpr (kTwo) {
        o0 = 2 * item;
        o1 = o0 + 1;
    } else {
        o0 = o1 = item * VEC;
    }
    Chunk<T, VEC> a[kBatch], b[kTwo ? kBatch : 1];
    T* out[kBatch];
    int tokens[kBatch];  // of the batch's items, -1: none
    int tok = slot < slots ? slot : here, h = h0;  // the next (token, head)
    const auto load = [&]() {
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            tokens[j] = -1;
            if (tok < here) {
                const bool is_k = h >= p.q.heads;
                const RopeTensor& t = is_k ? p.k : p.q;
                const int hl = is_k ? h - p.q.heads : h;
                const int64_t m = m0 + tok;
                const T* in = static_cast<const T*>(t.in) + m * t.row_stride + hl * t.head_stride;
                out[j] = static_cast<T*>(t.out) + m * t.out_row_stride + hl * t.out_head_stride;
                a[j].load(in + o0);
                if constexpr (kTwo)
                    if (rotates) b[j].load(in + o1);
                tokens[j] = tok;
                h += p.head_lanes;
                if (h >= heads) {
                    h = h0;
                    tok += slots;
                }
            }
        }
    };
    load();
    for (int e = threadIdx.x; e < here * p.pairs; e += kRopeThreads) {
        const int row = e / p.pairs, i = e - row * p.pairs;
        const int64_t at = (m0 + row) * p.pos_row_stride + p.axis[i] * p.pos_axis_stride;
        const double pos = p.pos64 ? static_cast<double>(static_cast<const int64_t*>(p.pos)[at])
                                   : static_cast<double>(static_cast<const int32_t*>(p.pos)[at]);
        const double turns = pos * p.inv_turn[i];
        const double half_turns = 2.0 * (turns - rint(turns));
        const float angle = static_cast<float>(half_turns);
        float s, c;
        sincospif(angle, &s, &c);
        if constexpr (sizeof(T) == 4) {
            // The angle's rounding, up to 9e-8 rad, is more than a table entry's
            // own: taken back to first order (rms error of the rotation 5.5e-8 ->
            // 4.1e-8, with a table rounded from 64 bits 4.2e-8).  Outputs of 16
            // bits are rounded at 2^-12 and more, where it does not show (and
            // costs 5 to 9 % of the time).
            const float rest = 3.14159265f * static_cast<float>(half_turns - angle), s0 = s;
            s = fmaf(c, rest, s);
            c = fmaf(-s0, rest, c);
        }
        table[e] = make_float2(c, p.inverse ? -s : s);
    }
    __syncthreads();
    while (tokens[0] >= 0) {
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            if (tokens[j] < 0) continue;
            if (rotates) {
                float2 cs[kPairs];
#pragma unroll
                for (int i = 0; i < kPairs; ++i) cs[i] = table[tokens[j] * p.pairs + item * kPairs + i];
                float fa[VEC];
                a[j].get(fa);
                if constexpr (kTwo) {
                    float fb[VEC];
                    b[j].get(fb);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        const float x = fa[i], y = fb[i];
                        fa[i] = fmaf(x, cs[i].x, -(y * cs[i].y));
                        fb[i] = fmaf(x, cs[i].y, y * cs[i].x);
                    }
                    b[j].set(fb);
                    b[j].store(out[j] + o1);
                } else {
#pragma unroll
                    for (int i = 0; i < kPairs; ++i) {
                        const float x = fa[2 * i], y = fa[2 * i + 1];
                        fa[2 * i] = fmaf(x, cs[i].x, -(y * cs[i].y));
                        fa[2 * i + 1] = fmaf(x, cs[i].y, y * cs[i].x);
                    }
                }
                a[j].set(fa);
            }
            a[j].store(out[j] + o0);
        }
        load();
    }
}

using RopeKernel = void (*)(const RopeArgs);

template <typename T>
RopeKernel rope_kernel_for(bool vec, bool halves) {
    constexpr int V = 16 / sizeof(T);
    if (vec) return halves ? rope_kernel<T, V, true> : rope_kernel<T, V, false>;
    return halves ? rope_kernel<T, 1, true> : rope_kernel<T, 1, false>;
}

bool rope_aligned(const RopeTensor& t, int e) {
    return t.heads == 0 || (aligned16(t.in) && aligned16(t.out) && t.row_stride * e % 16 == 0 &&
                            t.head_stride * e % 16 == 0 && t.out_row_stride * e % 16 == 0 &&
                            t.out_head_stride * e % 16 == 0);
}

}  // namespace

tfq_status launch_rope(const RopeTensor& q, const RopeTensor& k, int64_t M, int D, int dtype, const void* pos,
                       bool pos64, int64_t pos_row_stride, int64_t pos_axis_stride, int pairs, const double* inv_freq,
                       const int32_t* axis, bool halves, bool inverse, cudaStream_t stream, DeviceState* ds) {
    const int heads = q.heads + k.heads;
    const int e = dtype == TFQ_DTYPE_FP32 ? 4 : 2;
    const int V = 16 / e;
    // 16-byte accesses need aligned heads whose rotated part (each half of it
    // in the halves pairing) and copied part are whole units
    const bool vec = rope_aligned(q, e) && rope_aligned(k, e) && D % V == 0 &&
                     (halves ? pairs % V == 0 : 2 * pairs % V == 0);
    RopeArgs a = {};
    a.q = q;
    a.k = k;
    a.M = M;
    a.D = D;
    a.pairs = pairs;
    a.rot_items = vec ? (halves ? pairs / V : 2 * pairs / V) : pairs;
    a.items = a.rot_items + (D - 2 * pairs) / (vec ? V : 1);
    a.head_lanes = std::max(1, std::min(heads, kRopeThreads / a.items));
    a.inverse = inverse;
    a.pos = pos;
    a.pos64 = pos64;
    a.pos_row_stride = pos_row_stride;
    a.pos_axis_stride = pos_axis_stride;
    constexpr double kInvTwoPi = 0.15915494309189533577;  // 1 / (2 pi)
    for (int i = 0; i < pairs; ++i) {
        a.inv_turn[i] = inv_freq[i] * kInvTwoPi;
        a.axis[i] = static_cast<uint8_t>(axis[i]);
    }
    // Tokens per CTA: a table entry for every thread while the tokens' heads stay
    // within kRopeBytes, work for every token slot, and few enough that every SM
    // gets kRopeSpread CTAs.  (Measured on B200, us in a graph, by the table alone
    // and so: 7 tokens, 18 heads of 80 fp32 5.2, 2.5; 1000 tokens, 80 heads of 32,
    // 8 pairs 17.4, 4.5; 2000 tokens, 40 heads of 256, 8 pairs 53, 13, one pair 2252,
    // 59; 30000 tokens, 40 heads of 128, 8 pairs 131, 101; 75600 tokens, 80 heads of
    // 128 505 both.  One token per CTA there 558; four CTAs per SM 8.4 for 1200
    // tokens, 32 heads of 128, eight 6.4.)
    const int slots = kRopeThreads / (a.items * a.head_lanes);
    const int table_tokens = std::max(1, kRopeThreads / std::max(1, pairs));
    const int64_t token_bytes = static_cast<int64_t>(heads) * D * e;
    const int64_t tokens = std::max<int64_t>(slots, std::min<int64_t>(table_tokens, kRopeBytes / token_bytes));
    const int64_t spread = static_cast<int64_t>(kRopeSpread) * ds->sm_count;
    a.tokens = static_cast<int>(std::max<int64_t>(1, std::min(tokens, (M + spread - 1) / spread)));
    const size_t smem = static_cast<size_t>(a.tokens) * pairs * sizeof(float2);
    const int64_t blocks = (M + a.tokens - 1) / a.tokens;
    auto kernel = dtype == TFQ_DTYPE_FP32   ? rope_kernel_for<float>(vec, halves)
                  : dtype == TFQ_DTYPE_FP16 ? rope_kernel_for<__half>(vec, halves)
                                            : rope_kernel_for<__nv_bfloat16>(vec, halves);
    cudaError_t err = launch_kernel(kernel, dim3(static_cast<unsigned>(blocks)), dim3(kRopeThreads), smem, stream, a);
    if (err == cudaSuccess) err = cudaGetLastError();
    return err == cudaSuccess ? TFQ_OK : fail(TFQ_ECUDA, "rotary launch: %s", cudaGetErrorString(err));
}

}  // namespace tfq
