// Paged 8-bit cache: what its kernels share.
//
// Codes are e4m3 in pages, [layer][page][kv head][slot][dim], with one
// power-of-two scale for each (layer, page, head) block of K and of V.
#pragma once

#include <cuda_fp16.h>

#include <string>

#include "kvb_internal.h"

namespace kvb {
namespace c8 {

constexpr int E_MIN = -117;  // 2^-9 (the least code) * 2^-117 is the least normal float
constexpr int E_MAX = 119;   // 448 * 2^119 is finite

// Positions of a sequence are counted in 32 bits.  The attention kernels name keys that lie past
// the last one (and do not read them): up to 382 with tiles asked for two ahead.
constexpr int64_t MAX_KEYS = 0x7ffffc00;

// The error word of the context and its host mirror (pinned, written by the
// kernel that finds the error, so that a call needs no copy back).
struct Err {
    int* word;
    int* mirror;
    uint64_t timeout_ns;
};

struct Cache {
    uint8_t* code[2];  // K, V
    float* scale[2];
    int64_t n_pages;
    int H, d, d_log2, page, page_log2;
    int l_begin, n_layers;
};

struct Seqs {
    const int* page_table;
    const int* off;
    const int* pos;
    const int* kv_len;
    int n_seq, max_pages, max_tokens, max_kv;
    int64_t T;
};

// ------------------------------------------------------------ launchers
cudaError_t launch_write(const Cache& c, const Seqs& q, kvb_dtype dtype, const void* k, const void* v, const Err& err,
                         cudaStream_t s);
cudaError_t launch_read(const Cache& c, const Seqs& q, kvb_dtype dtype, void* k, void* v, const Err& err,
                        cudaStream_t s);

struct AttnParams {
    Cache c;
    Seqs q;
    const void* query;  // [n_layers][Hq][T][d]
    void* out;
    float* lse;  // or null
    int g;       // query heads of a KV head
    int row_blocks;
    int min_tiles;      // a CTA's least share of the line of tiles
    float scale_log2;   // scale * log2(e)
    int* counters;      // [units], 0 before and after a call
    int2* shared_by;    // [units], tcgen05 kernel: CTAs that share the unit, the first of them
    float* partial;     // [slots][rows][d] outputs in units of 2^mv
    float4* part_stat;  // [slots][rows] (m, mv, sum, -)
    int64_t units, slots;
    Err err;
};

// How a call is cut: blocks of `rows` query rows, and their keys over CTAs.
struct AttnPlan {
    bool tensor;  // the tcgen05 kernel
    bool few;     // the other one: few keys
    int rows, row_blocks, min_tiles;
    int ctas;
    int64_t units;  // (layer, sequence, row block, head)
    int64_t slots;  // partial results: two a CTA
    double tiles;   // of all units, at most
    size_t counter_bytes, partial_bytes, unit_bytes;
};
AttnPlan plan_attention(const Cache& c, const Seqs& q, kvb_dtype dtype, int g, int num_sms);
cudaError_t launch_decode(const AttnParams& P, kvb_dtype dtype, const AttnPlan& p, cudaStream_t s);
cudaError_t launch_prefill(const AttnParams& P, const AttnPlan& p, cudaStream_t s);  // bf16, d 64 and 128

#ifdef __CUDACC__

__device__ __forceinline__ void err_set(const Err& e, int code) {
    if (atomicCAS(e.word, 0, code) == 0) {
        *reinterpret_cast<volatile int*>(e.mirror) = code;
        __threadfence_system();
    }
}

// The checked build's index checks (KVB_IN_BOUNDS) on this error record.
__device__ __forceinline__ bool check_bounds(const Err& e, int64_t first, int64_t count, int64_t size) {
    if (first >= 0 && count >= 0 && first + count <= size) return true;
    err_set(e, DEV_ERR_BOUNDS);
    return false;
}
// Entry p of sequence s's row of the page table.
__device__ __forceinline__ bool table_in_bounds(const Seqs& q, const Err& e, int s, int64_t p) {
    return KVB_IN_BOUNDS(e, s, 1, q.n_seq) && KVB_IN_BOUNDS(e, p, 1, q.max_pages);
}
// Blocks (layer, page, head) that a call may touch.
__device__ __forceinline__ int64_t blocks_of(const Cache& c) {
    return (static_cast<int64_t>(c.l_begin) + c.n_layers) * c.n_pages * c.H;
}

// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }
// e of a normal power of two.
__device__ __forceinline__ int exponent_of(float scale) { return (__float_as_int(scale) >> 23) - 127; }
// The smallest e in [E_MIN, E_MAX] with amax <= 448 * 2^e (448 = 1.75 * 2^8): the
// exponent of amax less 8, one more where its fraction is above 0.75.
__device__ __forceinline__ int exponent_for(float amax) {
    const int e = ((__float_as_int(amax) + 0x1FFFFF) >> 23) - 135;
    return min(max(e, E_MIN), E_MAX);
}

// Ask for `bytes` (a multiple of 16, 16-byte aligned) to be brought to L2.
__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// Two e4m3 codes (low byte: a), to nearest even, saturating.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}
// The two fp16 numbers (exact) of the codes in the low / high half of w.
__device__ __forceinline__ uint32_t half2_of_lo(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
    return r;
}
__device__ __forceinline__ uint32_t half2_of_hi(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(w));
    return r;
}
__device__ __forceinline__ float2 float2_of(uint32_t h2) {
    return __half22float2(*reinterpret_cast<const __half2*>(&h2));
}

// Sequence s of a call: its tokens and their first position.  n = 0 and an
// error recorded where it does not fit what the call described.
struct SeqView {
    int tok0, n, pos;
};
__device__ __forceinline__ SeqView seq_view(const Seqs& q, int s, const Err& err) {
    if (!KVB_IN_BOUNDS(err, s, 1, q.n_seq)) return SeqView{};
    const int a = __ldg(q.off + s), b = __ldg(q.off + s + 1);
    SeqView v{a, a < 0 || b < a ? 0 : b - a, __ldg(q.pos + s)};
    if (a < 0 || b < a || b > q.T || v.n > q.max_tokens || v.pos > 0x7fffffff - v.n) {
        err_set(err, DEV_ERR_BAD_SEQ);
        v.tok0 = v.n = 0;
    }
    return v;
}

#endif  // __CUDACC__

}  // namespace c8
}  // namespace kvb
