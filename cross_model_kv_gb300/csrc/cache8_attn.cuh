// Attention over paged caches: what the two kernels of the 8-bit cache share.  The row blocks, the
// line of tiles and the pieces serve the pages of the model's own type too (Params: its AttnParams).
#pragma once

#include "cache8.h"

namespace kvb {
namespace c8 {

constexpr float BIAS = 7.f;    // weights are taken against 2^-7 of the reference
constexpr float MARGIN = 8.f;  // a reference is raised past this much (base 2)
constexpr float NO_REF = -3.0e38f;
constexpr float WIDE_QUERY = 256.f;  // a row's factor above this may pass fp32 with a key scale (2^119 at most)
constexpr int MIN_TILES = 4;       // a CTA's least share of the line of tiles, but for few keys
constexpr int PREFILL_ROWS = 256;  // rows of a unit in the tcgen05 kernel

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

// A block of query rows of one sequence and head: row = token * g + head of the
// group, so the rows of a block are close in position.
struct RowBlock {
    int row0;
    int nrows, tok0, pos;  // nrows 0: the sequence has no such rows
    int pos_lo;            // position of the block's first row
    int kv_end;            // keys that its last row may see
    // index of a row in [n_layers][Hq][T]
    template <class Params>
    __device__ __forceinline__ int64_t row_of(const Params& P, int64_t hq0, int row) const {
        const int gr = row0 + row, i = gr / P.g;
        return (hq0 + (gr - i * P.g)) * P.q.T + tok0 + i;
    }
};

// Rows of q, out and lse.
template <class Params>
__device__ __forceinline__ int64_t rows_of(const Params& P) {
    return static_cast<int64_t>(P.c.n_layers) * P.c.H * P.g * P.q.T;
}

template <class Params>
__device__ __forceinline__ RowBlock row_block(const Params& P, int s, int rb, int rows) {
    RowBlock B{};
    const SeqView sv = seq_view(P.q, s, P.err);
    const int total = sv.n * P.g;  // and rows of a call, and tiles of its line, stay below 2^30
    B.row0 = rb * rows;
    if (B.row0 >= total) return B;
    B.nrows = min(rows, total - B.row0);
    B.tok0 = sv.tok0;
    B.pos = sv.pos;
    int64_t kv = P.q.kv_len ? static_cast<int64_t>(__ldg(P.q.kv_len + s)) : static_cast<int64_t>(sv.pos) + sv.n;
    if (kv > P.q.max_kv) {
        err_set(P.err, DEV_ERR_BAD_SEQ);
        kv = P.q.max_kv;
    }
    const int64_t pos_hi = sv.pos + (B.row0 + B.nrows - 1) / P.g;  // position of the block's last row
    B.pos_lo = sv.pos + B.row0 / P.g;
    B.kv_end = static_cast<int>(max(static_cast<int64_t>(0), min(kv, pos_hi + 1)));
    return B;
}

// Tiles of TILE keys of a unit: one at least, so that rows that see nothing are written; EXTRA: in front of them,
// those that the unit itself counts as.
template <int TILE, int EXTRA = 0>
__device__ __forceinline__ int unit_tiles(const RowBlock& B) {
    return B.nrows == 0 ? 0 : EXTRA + max(1, (B.kv_end + TILE - 1) / TILE);
}

// Inclusive scan / sum over the CTA's NTHREADS threads (scratch: one value a warp).
__device__ __forceinline__ int block_scan(int v, int* scratch) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, v, x);
        if (lane >= x) v += o;
    }
    __syncthreads();  // scratch is free
    if (lane == 31) scratch[warp] = v;
    __syncthreads();
    for (int w = 0; w < warp; ++w) v += scratch[w];
    return v;
}
template <int NTHREADS>
__device__ __forceinline__ int block_sum(int v, int* scratch) {
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) v += __shfl_xor_sync(0xffffffffu, v, x);
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0;
    for (int w = 0; w < NTHREADS / 32; ++w) v += scratch[w];
    return v;
}

struct LineStart {
    int found, before, total;
};

// The units' tiles form one line: layer, then entry (sequence, row block), then
// head.  This CTA takes tiles [at, stop) of it, the first of them tile `first` of unit
// (l, e, h); share is every CTA's number.  false: nothing is left for this CTA.
// A_LANE: entries a lane of a warp looks at, where there are few enough for every warp to look by itself.  The 8-bit
// kernels have one: with four, prefill_kernel<128> spills 108 bytes instead of 24 and 1024 tokens over 16K take 507 us
// instead of 497, one token of 40 sequences of 2000 keys 42.6 instead of 42.0.
template <int ROWS, int TILE, int NTHREADS, int EXTRA = 0, int A_LANE = 1, class Params>
__device__ __forceinline__ bool line_start(const Params& P, int* scratch, LineStart* found, int& at, int& stop, int& share,
                                           int& l, int& e, int& h, int& first) {
    const int entries = P.q.n_seq * P.row_blocks;
    auto tiles_of = [&](int i) { return unit_tiles<TILE, EXTRA>(row_block(P, i / P.row_blocks, i % P.row_blocks, ROWS)); };
    int before = 0, want;  // tiles of the entries before e, times H; and up to this CTA's first
    auto place = [&](int per_layer) {
        const int all = per_layer * P.c.n_layers;
        share = max(P.min_tiles, (all + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x));
        at = static_cast<int>(blockIdx.x) * share;
        if (at >= all) return false;
        stop = min(all, at + share);
        l = at / per_layer;
        want = at - l * per_layer;
        return true;
    };
    if (entries <= 32 * A_LANE) {  // every warp for itself: no barrier
        const int lane = threadIdx.x & 31, per = A_LANE == 1 ? 1 : (entries + 31) / 32;
        int mine[A_LANE], sum = 0;
#pragma unroll
        for (int x = 0; x < A_LANE; ++x) mine[x] = x < per && lane * per + x < entries ? tiles_of(lane * per + x) * P.c.H : 0;
#pragma unroll
        for (int x = 0; x < A_LANE; ++x) sum += mine[x];
        int incl = sum;
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, incl, x);
            if (lane >= x) incl += o;
        }
        if (!place(__shfl_sync(0xffffffffu, incl, 31))) return false;
        const uint32_t hit = __ballot_sync(0xffffffffu, want >= incl - sum && want < incl);
        if (hit == 0) return false;  // not reached while the call's arrays stay as they are
        int first_of = incl - sum, at_entry = lane * per;  // the lane's entry that holds `want`
#pragma unroll
        for (int x = 0; x < A_LANE - 1; ++x)
            if (x + 1 < per && want >= first_of + mine[x] && at_entry == lane * per + x) {
                first_of += mine[x];
                ++at_entry;
            }
        e = __shfl_sync(0xffffffffu, at_entry, __ffs(hit) - 1);
        before = __shfl_sync(0xffffffffu, first_of, __ffs(hit) - 1);
    } else {
        const int mine0 = static_cast<int>(threadIdx.x) < entries ? tiles_of(threadIdx.x) : 0;
        int per_layer = mine0;
        for (int i = threadIdx.x + NTHREADS; i < entries; i += NTHREADS) per_layer += tiles_of(i);
        if (!place(block_sum<NTHREADS>(per_layer, scratch) * P.c.H)) return false;
        e = -1;
        for (int e0 = 0; e < 0; e0 += NTHREADS) {
            if (e0 >= entries) return false;  // likewise
            const int i = e0 + threadIdx.x;
            const int mine = (e0 == 0 ? mine0 : i < entries ? tiles_of(i) : 0) * P.c.H;
            const int incl = before + block_scan(mine, scratch);
            if (threadIdx.x == 0) found->found = -1;
            __syncthreads();
            if (want >= incl - mine && want < incl) {
                found->found = i;
                found->before = incl - mine;
            }
            if (threadIdx.x == NTHREADS - 1) found->total = incl;
            __syncthreads();
            e = found->found;
            before = e < 0 ? found->total : found->before;
            __syncthreads();
        }
    }
    const int tiles = tiles_of(e);
    h = (want - before) / tiles;
    first = want - before - h * tiles;
    return true;
}

// The partial results of one unit, in the order of its keys: CTAs c0 .. c0 + n - 1
// share it; a CTA's slot is 2c for the piece that it begins with and 2c + 1 for one that
// it ends with.
struct Pieces {
    int n, c0;
    __device__ __forceinline__ int64_t slot(int i) const { return i == 0 ? 2 * c0 + 1 : 2 * (c0 + i); }
};

// All of them (the checked build).
template <class Params>
__device__ __forceinline__ bool pieces_in_bounds(const Params& P, const Pieces& pieces) {
    return KVB_IN_BOUNDS(P.err, pieces.slot(0), 1, P.slots) && KVB_IN_BOUNDS(P.err, pieces.slot(pieces.n - 1), 1, P.slots);
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
        sum = fmaf(ex2(st.x - m), st.z, sum);
        weigh(ex2(st.y - mv), o);
    }
    __device__ __forceinline__ void weigh(float f, const float4& o) {
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

// After a piece of a unit is written: the last CTA of the unit to arrive joins
// the pieces, in order.  Called by all NTHREADS threads; buf: shared memory of
// `cap` floats, free once they have met.  A warp takes a row's references and sum, the
// weights of all chunks go to shared memory, then each thread adds its columns with
// its loads in flight together: 64 pieces one after another took 15 us.
template <typename T, int D, int ROWS, int NTHREADS>
__device__ __forceinline__ void join_splits(const AttnParams& P, const RowBlock& B, const Pieces& pieces, int64_t unit, int64_t hq0, int* s_last,
                                            float* buf, int cap) {
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
        *s_last = false;
        if (KVB_IN_BOUNDS(P.err, unit, 1, P.units) && pieces_in_bounds(P, pieces)) {
            const int n = atomicAdd(P.counters + unit, 1);
            *s_last = n == pieces.n - 1;
            if (n == pieces.n - 1) P.counters[unit] = 0;
        }
    }
    __syncthreads();
    if (!*s_last) return;
    __threadfence();
    const int active = pieces.n, lane = threadIdx.x & 31;
    float4* ref = reinterpret_cast<float4*>(buf);  // [ROWS] (m, mv, sum, -)
    float* weight = buf + 4 * ROWS;                // [row][piece]
    const bool listed = active <= (cap - 4 * ROWS) / ROWS;
    auto stat = [&](int row, int i) { return __ldcg(P.part_stat + pieces.slot(i) * ROWS + row); };
    for (int row = threadIdx.x >> 5; row < B.nrows; row += NTHREADS / 32) {
        float m = NO_REF, mv = NO_REF, sum = 0.f;
        for (int i = lane; i < active; i += 32) {
            const float4 st = stat(row, i);
            m = fmaxf(m, st.x);
            mv = fmaxf(mv, st.y);
        }
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) {
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
            mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, x));
        }
        for (int i = lane; i < active; i += 32) {
            const float4 st = stat(row, i);
            sum = fmaf(ex2(st.x - m), st.z, sum);
            if (listed) weight[row * active + i] = ex2(st.y - mv);
        }
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        if (lane == 0) ref[row] = make_float4(m, mv, sum, 0.f);
    }
    __syncthreads();
    T* out = static_cast<T*>(P.out);
    for (int e = threadIdx.x; e < B.nrows * (D / 4); e += NTHREADS) {
        const int row = e / (D / 4), d4 = e % (D / 4);
        const float4 st = ref[row];
        Joined z;
        z.m = st.x;
        z.mv = st.y;
        z.sum = st.z;
#pragma unroll 8
        for (int i = 0; i < active; ++i)
            z.weigh(listed ? weight[row * active + i] : ex2(stat(row, i).y - z.mv), 
                    __ldcg(reinterpret_cast<const float4*>(P.partial + (pieces.slot(i) * ROWS + row) * D) + d4));
        const int64_t o = B.row_of(P, hq0, row);
        if (!KVB_IN_BOUNDS(P.err, o, 1, rows_of(P))) continue;
        store_out(out + o * D + 4 * d4, z.output());
        if (d4 == 0 && P.lse) P.lse[o] = z.lse();
    }
}

}  // namespace c8
}  // namespace kvb
