// Paged 8-bit cache: what its two attention kernels share.
#pragma once

#include "cache8.h"

namespace kvb {
namespace c8 {

constexpr float BIAS = 7.f;    // weights are taken against 2^-7 of the reference
constexpr float MARGIN = 8.f;  // a reference is raised past this much (base 2)
constexpr float NO_REF = -3.0e38f;

__device__ __forceinline__ float ex2(float x) {  // relative error about 2^-22
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void store_out(__nv_bfloat16* p, float4 v) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}
__device__ __forceinline__ void store_out(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }

// The rows and keys of one CTA: row = token * g + head of the group, so the rows
// of a block are close in position; keys [k0, k1) of the last row's visible ones.
struct RowBlock {
    int64_t row0;
    int nrows, tok0, pos;
    int pos_lo;        // position of the block's first row
    int k0, k1, active;  // active: chunks that have keys (at least one)
    // index of a row in [n_layers][Hq][T]
    __device__ __forceinline__ int64_t row_of(const AttnParams& P, int64_t hq0, int row) const {
        const int64_t gr = row0 + row, i = gr / P.g;
        return (hq0 + (gr - i * P.g)) * P.q.T + tok0 + i;
    }
};

// false where the block has no rows or the chunk no keys.
__device__ __forceinline__ bool row_block(const AttnParams& P, int s, int rb, int rows, int split, RowBlock& B) {
    const SeqView sv = seq_view(P.q, s, P.err);
    const int64_t total = static_cast<int64_t>(sv.n) * P.g;
    B.row0 = static_cast<int64_t>(rb) * rows;
    if (B.row0 >= total) return false;
    B.nrows = static_cast<int>(min(static_cast<int64_t>(rows), total - B.row0));
    B.tok0 = sv.tok0;
    B.pos = sv.pos;
    int64_t kv = P.q.kv_len ? static_cast<int64_t>(__ldg(P.q.kv_len + s)) : static_cast<int64_t>(sv.pos) + sv.n;
    if (kv > P.q.max_kv) {
        if (threadIdx.x == 0) err_set(P.err, DEV_ERR_BAD_SEQ);
        kv = P.q.max_kv;
    }
    const int64_t pos_hi = sv.pos + (B.row0 + B.nrows - 1) / P.g;  // position of the block's last row
    B.pos_lo = sv.pos + static_cast<int>(B.row0 / P.g);
    const int kv_end = static_cast<int>(max(static_cast<int64_t>(0), min(kv, pos_hi + 1)));
    B.active = max(1, static_cast<int>((static_cast<int64_t>(kv_end) + P.chunk - 1) / P.chunk));
    if (split >= B.active) return false;
    B.k0 = split * P.chunk;
    B.k1 = static_cast<int>(min(static_cast<int64_t>(kv_end), static_cast<int64_t>(B.k0) + P.chunk));
    return true;
}

// Parts of one row's result, each with its references: first every part's
// reference(), then every part's add().  st = (m, mv, sum, -).  A part that saw
// nothing has NO_REF references and adds zeros; a NaN reaches the result.
struct Joined {
    float m = NO_REF, mv = NO_REF, sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    __device__ __forceinline__ void reference(const float4& st) {
        m = fmaxf(m, st.x);
        mv = fmaxf(mv, st.y);
    }
    __device__ __forceinline__ void add(const float4& st, const float4& o) {
        const float f = ex2(st.y - mv);
        sum = fmaf(ex2(st.x - m), st.z, sum);
        acc.x = fmaf(f, o.x, acc.x);
        acc.y = fmaf(f, o.y, acc.y);
        acc.z = fmaf(f, o.z, acc.z);
        acc.w = fmaf(f, o.w, acc.w);
    }
    // acc / sum * 2^(mv - m), the power in two halves: it may pass the range of one float
    __device__ __forceinline__ float4 output() const {
        const float half = ex2(0.5f * (mv - m)), f = sum == 0.f ? 0.f : half / sum;
        return make_float4(acc.x * f * half, acc.y * f * half, acc.z * f * half, acc.w * f * half);
    }
    __device__ __forceinline__ float lse() const {
        return sum == 0.f ? -INFINITY : (m - BIAS + log2f(sum)) * 0.693147180559945f;
    }
};

// After a chunk's partial results are written: the last CTA of the unit to
// arrive joins the chunks, in order.  Called by the CTA's first NTHREADS threads
// (SOME: there are others, so they meet at named barrier 9).
template <typename T, int D, int ROWS, int NTHREADS, bool SOME = false>
__device__ __forceinline__ void join_splits(const AttnParams& P, const RowBlock& B, int64_t unit, int64_t hq0, int* s_last) {
    auto meet = [] {
        if constexpr (SOME) named_bar_sync(9, NTHREADS);
        else __syncthreads();
    };
    __threadfence();
    meet();
    if (threadIdx.x == 0) {
        const int n = atomicAdd(P.counters + unit, 1);
        *s_last = n == B.active - 1;
        if (n == B.active - 1) P.counters[unit] = 0;
    }
    meet();
    if (!*s_last) return;
    __threadfence();
    const int64_t u0 = unit * P.splits * ROWS;
    T* out = static_cast<T*>(P.out);
    for (int e = threadIdx.x; e < B.nrows * (D / 4); e += NTHREADS) {
        const int row = e / (D / 4), d4 = e % (D / 4);
        Joined z;
        for (int i = 0; i < B.active; ++i) z.reference(__ldcg(P.part_stat + u0 + static_cast<int64_t>(i) * ROWS + row));
#pragma unroll 4
        for (int i = 0; i < B.active; ++i) {
            const int64_t p = u0 + static_cast<int64_t>(i) * ROWS + row;
            z.add(__ldcg(P.part_stat + p), __ldcg(reinterpret_cast<const float4*>(P.partial + p * D) + d4));
        }
        const int64_t o = B.row_of(P, hq0, row);
        store_out(out + o * D + 4 * d4, z.output());
        if (d4 == 0 && P.lse) P.lse[o] = z.lse();
    }
}

}  // namespace c8
}  // namespace kvb
