// Attention over the paged cache of the model's own type: what its kernels share.
#pragma once

#include <cfloat>

#include "cache8_attn.cuh"
#include "paged.h"

namespace kvb {
namespace paged {

using c8::ex2;
using c8::LineStart;
using c8::Pieces;
using c8::RowBlock;

constexpr float MARGIN = 8.f;       // a reference is raised past this much (base 2)
constexpr float LOWEST = -FLT_MAX;  // reference of a row that has seen nothing

// Outputs and statistics of one row's parts, each with a reference.
struct Joined {
    float m = LOWEST, sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    __device__ __forceinline__ void reference(float2 st) { m = fmaxf(m, st.x); }
    __device__ __forceinline__ void add(float2 st, float4 o) {
        const float w = ex2(st.x - m);
        sum = fmaf(w, st.y, sum);
        weigh(w, o);
    }
    __device__ __forceinline__ void weigh(float w, float4 o) {
        acc.x = fmaf(w, o.x, acc.x);
        acc.y = fmaf(w, o.y, acc.y);
        acc.z = fmaf(w, o.z, acc.z);
        acc.w = fmaf(w, o.w, acc.w);
    }
    __device__ __forceinline__ float4 output() const {
        if (sum == 0.f) return make_float4(0.f, 0.f, 0.f, 0.f);  // whatever the values that it does not see are
        const float f = 1.f / sum;
        return make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
    }
    __device__ __forceinline__ float lse() const { return sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.693147180559945f; }
};

// Keys that some rows of a block see and others do not (the last of several new tokens) may have values
// that are not finite: 0 times them is NaN, for rows that do not see them too.  Such values become 0 where
// they lie in shared memory, and are added afterwards to the rows that see them: any weight of them is the same.
__device__ __forceinline__ bool not_finite(float x) { return (__float_as_uint(x) & 0x7f800000u) == 0x7f800000u; }
template <typename T>
__device__ __forceinline__ uint32_t finite_or_0(uint32_t w) {  // an fp32 number, or two of bf16
    if constexpr (sizeof(T) == 4) return (w & 0x7f800000u) == 0x7f800000u ? 0u : w;
    else return w & (((w & 0x7f80u) == 0x7f80u ? 0u : 0xffffu) | ((w & 0x7f800000u) == 0x7f800000u ? 0u : 0xffff0000u));
}
template <typename T>
__device__ __forceinline__ bool make_finite(uint4& v) {  // whether it was not
    const uint4 x = make_uint4(finite_or_0<T>(v.x), finite_or_0<T>(v.y), finite_or_0<T>(v.z), finite_or_0<T>(v.w));
    const bool odd = ((v.x ^ x.x) | (v.y ^ x.y) | (v.z ^ x.z) | (v.w ^ x.w)) != 0;
    if (odd) v = x;
    return odd;
}
// Element `dim` of the value of key j, 0 if its page is not there.
template <typename T>
__device__ __forceinline__ float value_of(const AttnParams& P, int s, int l, int h, int j, int dim) {
    const int p = j >> P.c.page_log2;
    if (p >= P.q.max_pages || !c8::table_in_bounds(P.q, P.err, s, p)) return 0.f;
    const int pid = __ldg(P.q.page_table + static_cast<int64_t>(s) * P.q.max_pages + p);
    const int64_t blocks = (static_cast<int64_t>(P.c.l_begin) + P.c.n_layers) * P.c.n_pages * P.c.H;
    const int64_t block = ((static_cast<int64_t>(P.c.l_begin) + l) * P.c.n_pages + pid) * P.c.H + h;
    if (pid < 0 || pid >= P.c.n_pages || !KVB_IN_BOUNDS(P.err, block, 1, blocks)) return 0.f;
    const int64_t at = (((block << P.c.page_log2) + (j & (P.c.page - 1))) << P.c.d_log2) + dim;
    return static_cast<float>(static_cast<const T*>(P.c.kv[1])[at]);
}

// Row `row` of a unit, in rows with strides and in [n_layers][Hq][T].
struct RowPlace {
    int head, token;
};
__device__ __forceinline__ RowPlace place_of(const AttnParams& P, const RowBlock& B, int h, int row) {
    const int gr = B.row0 + row, i = gr / P.g;
    return RowPlace{h * P.g + (gr - i * P.g), B.tok0 + i};
}
template <typename T>
__device__ __forceinline__ T* address(const Rows& r, int l, RowPlace at) {
    return static_cast<T*>(r.data) + (l * r.l + at.head * r.h + at.token * r.t);
}
template <typename T>
__device__ __forceinline__ void write_row(const AttnParams& P, int l, RowPlace at, int d4, const Joined& z) {
    const int64_t row = (static_cast<int64_t>(l) * P.c.H * P.g + at.head) * P.q.T + at.token;
    if (!KVB_IN_BOUNDS(P.err, row, 1, c8::rows_of(P))) return;
    c8::store_out(address<T>(P.out, l, at) + 4 * d4, z.output());
    if (d4 == 0 && P.lse) P.lse[row] = z.lse();
}

// After a piece of a unit is written: the last CTA of the unit to arrive joins the pieces, in
// order.  All pieces' statistics go to shared memory (`buf`, `cap` floats, free) and become their weights,
// then each of the NT threads adds its columns, with the loads of each part in flight together.
template <typename T, int D, int ROWS, int NT>
__device__ __forceinline__ void join_pieces(const AttnParams& P, const RowBlock& B, const Pieces& pieces, int64_t unit, int l, int h,
                                            int* s_last, float* buf, int cap) {
    const int tid = threadIdx.x;
    __syncthreads();
    if (tid == 0) {  // its fences, with the barriers, order what all threads wrote and will read
        *s_last = false;
        __threadfence();
        if (KVB_IN_BOUNDS(P.err, unit, 1, P.units) && c8::pieces_in_bounds(P, pieces)) {
            const int n = atomicAdd(P.counters + unit, 1);
            *s_last = n == pieces.n - 1;
            if (n == pieces.n - 1) P.counters[unit] = 0;
        }
        __threadfence();
    }
    __syncthreads();
    if (!*s_last) return;
    const int n = pieces.n, lane = tid & 31;
    float2* whole = reinterpret_cast<float2*>(buf);              // [ROWS] reference, 1 / sum
    int64_t* to = reinterpret_cast<int64_t*>(buf + 2 * ROWS);    // [ROWS] element of P.out, or -1
    float2* part = reinterpret_cast<float2*>(buf + 4 * ROWS);    // [row][piece] reference (then weight / sum), sum
    const bool listed = n <= (cap - 4 * ROWS) / (2 * ROWS);
    auto stat = [&](int row, int i) { return __ldcg(P.part_stat + pieces.slot(i) * ROWS + row); };
    // what a row needs once
    auto finish = [&](int row, float m, float sum) {
        const RowPlace at = place_of(P, B, h, row);
        const int64_t r = (static_cast<int64_t>(l) * P.c.H * P.g + at.head) * P.q.T + at.token;
        const bool inside = KVB_IN_BOUNDS(P.err, r, 1, c8::rows_of(P));
        to[row] = inside ? l * P.out.l + at.head * P.out.h + at.token * P.out.t : -1;
        if (inside && P.lse) P.lse[r] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.693147180559945f;
        const float by = sum == 0.f ? 0.f : 1.f / sum;
        whole[row] = make_float2(m, by);
        return by;
    };
    if (listed) {
#pragma unroll 4
        for (int i = tid; i < B.nrows * n; i += NT) part[i] = stat(i / n, i % n);
        __syncthreads();
    }
    if (listed && n <= 8) {  // a thread a row
        for (int row = tid; row < B.nrows; row += NT) {
            float2* mine = part + row * n;
            float m = LOWEST, sum = 0.f;
            for (int i = 0; i < n; ++i) m = fmaxf(m, mine[i].x);
            for (int i = 0; i < n; ++i) {
                const float w = ex2(mine[i].x - m);
                sum = fmaf(w, mine[i].y, sum);
                mine[i].x = w;
            }
            const float by = finish(row, m, sum);
            for (int i = 0; i < n; ++i) mine[i].x *= by;
        }
    } else {  // a warp a row
        for (int row = tid >> 5; row < B.nrows; row += NT / 32) {
            auto at = [&](int i) { return listed ? part[row * n + i] : stat(row, i); };
            float m = LOWEST, sum = 0.f;
            for (int i = lane; i < n; i += 32) m = fmaxf(m, at(i).x);
#pragma unroll
            for (int x = 1; x < 32; x <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
            for (int i = lane; i < n; i += 32) {
                const float2 y = at(i);
                const float w = ex2(y.x - m);
                sum = fmaf(w, y.y, sum);
                if (listed) part[row * n + i].x = w;
            }
#pragma unroll
            for (int x = 1; x < 32; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
            float by = 0.f;
            if (lane == 0) by = finish(row, m, sum);
            by = __shfl_sync(0xffffffffu, by, 0);
            if (listed)
                for (int i = lane; i < n; i += 32) part[row * n + i].x *= by;
        }
    }
    __syncthreads();
    // a thread's items side by side, AT_ONCE loads and more in flight: one after another they took 1000
    // cycles each
    constexpr int AT_ONCE = 8;
    const int items = B.nrows * (D / 4);
    for (int i0 = tid; i0 < items; i0 += AT_ONCE * NT) {
        float4 acc[AT_ONCE];
        int row[AT_ONCE];
        const float4* from[AT_ONCE];
#pragma unroll
        for (int x = 0; x < AT_ONCE; ++x) {
            const int i = min(i0 + x * NT, items - 1);
            row[x] = i / (D / 4);
            from[x] = reinterpret_cast<const float4*>(P.partial) + i;
            acc[x] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        auto add = [&](int p, auto weight) {
            const int64_t slot = pieces.slot(p) * (ROWS * (D / 4));
            float4 v[AT_ONCE];
#pragma unroll
            for (int x = 0; x < AT_ONCE; ++x) v[x] = __ldcg(from[x] + slot);
#pragma unroll
            for (int x = 0; x < AT_ONCE; ++x) {
                const float w = weight(x);
                acc[x].x = fmaf(w, v[x].x, acc[x].x);
                acc[x].y = fmaf(w, v[x].y, acc[x].y);
                acc[x].z = fmaf(w, v[x].z, acc[x].z);
                acc[x].w = fmaf(w, v[x].w, acc[x].w);
            }
        };
        if (listed) {
#pragma unroll 2
            for (int p = 0; p < n; ++p) add(p, [&](int x) { return part[row[x] * n + p].x; });
        } else {
            for (int p = 0; p < n; ++p) add(p, [&](int x) { return ex2(stat(row[x], p).x - whole[row[x]].x) * whole[row[x]].y; });
        }
#pragma unroll
        for (int x = 0; x < AT_ONCE; ++x)
            if (i0 + x * NT < items && to[row[x]] >= 0) {
                const bool seen = whole[row[x]].y != 0.f;  // else 0, whatever the values that it does not see are
                const float4 o = seen ? acc[x] : make_float4(0.f, 0.f, 0.f, 0.f);
                c8::store_out(static_cast<T*>(P.out.data) + to[row[x]] + 4 * ((i0 + x * NT) % (D / 4)), o);
            }
    }
}

}  // namespace paged
}  // namespace kvb
