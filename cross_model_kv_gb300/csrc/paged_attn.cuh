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
        const float f = sum == 0.f ? 0.f : 1.f / sum;
        return make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
    }
    __device__ __forceinline__ float lse() const { return sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.693147180559945f; }
};

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
// order.  A warp takes a row's references and sum, the weights of all pieces go to shared memory (`buf`,
// `cap` floats, free), then each thread adds its columns with its loads in flight together.
// meet(): the NT threads, numbered from 0, meet.
template <typename T, int D, int ROWS, int NT, class Meet>
__device__ __forceinline__ void join_pieces(const AttnParams& P, const RowBlock& B, const Pieces& pieces, int64_t unit, int l, int h,
                                            int* s_last, float* buf, int cap, Meet meet) {
    const int tid = threadIdx.x;
    __threadfence();
    meet();
    if (tid == 0) {
        *s_last = false;
        if (KVB_IN_BOUNDS(P.err, unit, 1, P.units) && c8::pieces_in_bounds(P, pieces)) {
            const int n = atomicAdd(P.counters + unit, 1);
            *s_last = n == pieces.n - 1;
            if (n == pieces.n - 1) P.counters[unit] = 0;
        }
    }
    meet();
    if (!*s_last) return;
    __threadfence();
    const int n = pieces.n, lane = tid & 31;
    float2* whole = reinterpret_cast<float2*>(buf);  // [ROWS] reference, sum
    float* weight = buf + 2 * ROWS;                  // [row][piece]
    const bool listed = n <= (cap - 2 * ROWS) / ROWS;
    auto stat = [&](int row, int i) { return __ldcg(P.part_stat + pieces.slot(i) * ROWS + row); };
    for (int row = tid >> 5; row < B.nrows; row += NT / 32) {
        float m = LOWEST, sum = 0.f;
        float2 st[2];  // of 64 pieces; more are read again
#pragma unroll
        for (int i = 0; i < 2; ++i) st[i] = lane + 32 * i < n ? stat(row, lane + 32 * i) : make_float2(LOWEST, 0.f);
        m = fmaxf(st[0].x, st[1].x);
        for (int i = lane + 64; i < n; i += 32) m = fmaxf(m, stat(row, i).x);
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
        for (int i = lane, c = 0; i < n; i += 32, ++c) {
            const float2 y = c == 0 ? st[0] : c == 1 ? st[1] : stat(row, i);
            const float w = ex2(y.x - m);
            sum = fmaf(w, y.y, sum);
            if (listed) weight[row * n + i] = w;
        }
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        if (lane == 0) whole[row] = make_float2(m, sum);
    }
    meet();
    for (int i = tid; i < B.nrows * (D / 4); i += NT) {
        const int row = i / (D / 4), d4 = i % (D / 4);
        Joined z;
        z.m = whole[row].x;
        z.sum = whole[row].y;
#pragma unroll 16
        for (int p = 0; p < n; ++p)
            z.weigh(listed ? weight[row * n + p] : ex2(stat(row, p).x - z.m),
                    __ldcg(reinterpret_cast<const float4*>(P.partial + (pieces.slot(p) * ROWS + row) * D) + d4));
        write_row<T>(P, l, place_of(P, B, h, row), d4, z);
    }
}

}  // namespace paged
}  // namespace kvb
