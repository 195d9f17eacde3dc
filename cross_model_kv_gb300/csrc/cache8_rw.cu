// Writing tokens into the paged 8-bit cache and reading them back.
//
// Both are bound by HBM: a write reads 2 (bf16) or 4 (fp32) bytes and writes 1
// per element, a read the reverse; the arithmetic is a handful of operations
// per element.
#include "cache8.h"

namespace kvb {
namespace c8 {

namespace {

constexpr int NT = 256;    // threads per CTA (512 where a block needs them all)
constexpr int CHUNKS = 4;  // 8-element chunks that one thread holds: 16 registers of bf16, 32 of fp32

struct RwParams {
    Cache c;
    Seqs q;
    const void* src[2];  // write
    void* dst[2];        // read
    int items;           // blocks that one sequence can touch
    int64_t total;       // items * n_seq * H * n_layers * 2
    Err err;
};

// Block `idx` of a call: the K or V block of one page that one sequence's tokens touch.
struct Item {
    int kv, l, h, s, i;
};
__device__ __forceinline__ Item item_of(const RwParams& P, int64_t idx) {
    uint32_t x = static_cast<uint32_t>(idx);  // total < 2^31
    Item it;
    it.i = x % P.items;
    x /= P.items;
    it.s = x % P.q.n_seq;
    x /= P.q.n_seq;
    it.h = x % P.c.H;
    x /= P.c.H;
    it.l = x % P.c.n_layers;
    it.kv = x / P.c.n_layers;
    return it;
}

// Eight elements as they lie in memory, and as fp32 with those that are not finite as 0.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
    uint4 u;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = __ldcs(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void get(float (&o)[8]) const {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o[2 * i] = __uint_as_float(w[i] << 16);
            o[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};
template <>
struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = __ldcs(reinterpret_cast<const float4*>(p));
        b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void get(float (&o)[8]) const {
        o[0] = a.x; o[1] = a.y; o[2] = a.z; o[3] = a.w;
        o[4] = b.x; o[5] = b.y; o[6] = b.z; o[7] = b.w;
    }
};
__device__ __forceinline__ bool finite(float x) { return fabsf(x) < __int_as_float(0x7f800000); }

// One block per group of GS threads: its new values stay in registers, as they
// lay in memory, between the maximum and the rounding, so they are read once and
// enough CTAs are resident to keep HBM busy (holding them as fp32, eight chunks
// a thread, left two CTAs an SM and 3.1 TB/s).
template <typename T, int GS>
__global__ void __launch_bounds__(GS > NT ? GS : NT) write_kernel(const __grid_constant__ RwParams P) {
    constexpr int PER = GS > NT ? 1 : NT / GS;
    const int64_t idx = static_cast<int64_t>(blockIdx.x) * PER + threadIdx.x / GS;
    const int t = threadIdx.x % GS;
    if (idx >= P.total) return;  // whole groups leave together, here and below
    const Item it = item_of(P, idx);
    const SeqView sv = seq_view(P.q, it.s, P.err);
    if (sv.n == 0) return;
    if (sv.pos < 0) {
        if (t == 0) err_set(P.err, DEV_ERR_BAD_SEQ);
        return;
    }
    const int64_t logical = (sv.pos >> P.c.page_log2) + it.i;
    const int64_t p0 = logical << P.c.page_log2;
    const int64_t end = static_cast<int64_t>(sv.pos) + sv.n;
    const int lo = it.i == 0 ? sv.pos - static_cast<int>(p0) : 0;  // first slot written
    const int m = static_cast<int>(min(end - p0, static_cast<int64_t>(P.c.page))) - lo;
    if (m <= 0) return;
    const int pid = logical < P.q.max_pages ? __ldg(P.q.page_table + static_cast<int64_t>(it.s) * P.q.max_pages + logical) : -1;
    if (pid < 0 || pid >= P.c.n_pages) {
        if (t == 0) err_set(P.err, DEV_ERR_BAD_SEQ);
        return;
    }
    const int64_t tok = sv.tok0 + (p0 + lo - sv.pos);
    const int64_t head = static_cast<int64_t>(it.l) * P.c.H + it.h;
    const T* src = static_cast<const T*>(P.src[it.kv]) + ((head * P.q.T + tok) << P.c.d_log2);
    const int n8 = (m << P.c.d_log2) >> 3;

    Raw8<T> raw[CHUNKS];
    float amax = 0.f;
    bool bad = false;
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c)
        if (c * GS + t < n8) raw[c].load(src + 8 * (c * GS + t));
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c)
        if (c * GS + t < n8) {
            float x[8];
            raw[c].get(x);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                bad |= !finite(x[i]);
                amax = fmaxf(amax, finite(x[i]) ? fabsf(x[i]) : 0.f);
            }
        }
    if (bad) err_set(P.err, DEV_ERR_NONFINITE);
    // non-negative floats order as their bits
    int top = __reduce_max_sync(0xffffffffu, __float_as_int(amax));

    const int64_t block = ((static_cast<int64_t>(P.c.l_begin) + it.l) * P.c.n_pages + pid) * P.c.H + it.h;
    float* scale = P.c.scale[it.kv] + block;
    uint8_t* codes = P.c.code[it.kv] + ((block << P.c.page_log2) << P.c.d_log2);
    int e_old = E_MIN;
    if (lo > 0) e_old = min(max(exponent_of(*scale), E_MIN), E_MAX);
    if constexpr (GS > 32) {
        __shared__ int tops[PER][GS / 32];
        const int group = threadIdx.x / GS;
        if ((t & 31) == 0) tops[group][t >> 5] = top;
        named_bar_sync(1 + group, GS);  // also: every thread has read the old scale
#pragma unroll
        for (int w = 0; w < GS / 32; ++w) top = max(top, tops[group][w]);
    } else {
        __syncwarp();
    }
    const int e = max(e_old, exponent_for(__int_as_float(top)));
    if (t == 0) *scale = pow2(e);
    const float inv = pow2(-e);
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c)
        if (c * GS + t < n8) {
            float x[8];
            raw[c].get(x);
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = finite(x[i]) ? x[i] * inv : 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = e4m3x2(x[2 * i], x[2 * i + 1]);
            *reinterpret_cast<uint2*>(codes + (lo << P.c.d_log2) + 8 * (c * GS + t)) =
                make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
        }
    if (lo > 0 && e > e_old) {  // the slots before the new tokens, under the larger scale
        const float f = pow2(max(e_old - e, -126));
        for (int c = t; c < (lo << P.c.d_log2) >> 3; c += GS) {
            uint2* p = reinterpret_cast<uint2*>(codes) + c;
            const uint2 u = *p;
            uint32_t r[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float2 a = float2_of(half2_of_lo(i ? u.y : u.x)), b = float2_of(half2_of_hi(i ? u.y : u.x));
                r[i] = e4m3x2(a.x * f, a.y * f) | (e4m3x2(b.x * f, b.y * f) << 16);
            }
            *p = make_uint2(r[0], r[1]);
        }
    }
}

__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                   pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7])));
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(x[0], x[1], x[2], x[3]));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(x[4], x[5], x[6], x[7]));
}

// One block per group of GS threads; code * 2^e is exact in fp32 and in bf16.
template <typename T, int GS>
__global__ void __launch_bounds__(NT) read_kernel(const __grid_constant__ RwParams P) {
    const int64_t idx = static_cast<int64_t>(blockIdx.x) * (NT / GS) + threadIdx.x / GS;
    const int t = threadIdx.x % GS;
    if (idx >= P.total) return;
    const Item it = item_of(P, idx);
    const SeqView sv = seq_view(P.q, it.s, P.err);
    if (sv.n == 0) return;
    if (sv.pos < 0 && t == 0) err_set(P.err, DEV_ERR_BAD_SEQ);
    const int pos = max(sv.pos, 0);
    const int64_t logical = (pos >> P.c.page_log2) + it.i;
    const int64_t p0 = logical << P.c.page_log2;
    const int64_t end = static_cast<int64_t>(pos) + sv.n;
    const int lo = it.i == 0 ? pos - static_cast<int>(p0) : 0;
    const int m = static_cast<int>(min(end - p0, static_cast<int64_t>(P.c.page))) - lo;
    if (m <= 0) return;
    int pid = logical < P.q.max_pages ? __ldg(P.q.page_table + static_cast<int64_t>(it.s) * P.q.max_pages + logical) : -1;
    const bool have = pid >= 0 && pid < P.c.n_pages && sv.pos >= 0;
    if (!have) {
        if (t == 0) err_set(P.err, DEV_ERR_BAD_SEQ);
        pid = 0;
    }
    const int64_t tok = sv.tok0 + (p0 + lo - pos);
    const int64_t head = static_cast<int64_t>(it.l) * P.c.H + it.h;
    T* dst = static_cast<T*>(P.dst[it.kv]) + ((head * P.q.T + tok) << P.c.d_log2);
    const int64_t block = ((static_cast<int64_t>(P.c.l_begin) + it.l) * P.c.n_pages + pid) * P.c.H + it.h;
    const uint8_t* codes = P.c.code[it.kv] + ((block << P.c.page_log2) << P.c.d_log2) + (lo << P.c.d_log2);
    const float f = have ? __ldg(P.c.scale[it.kv] + block) : 0.f;
    const int n8 = (m << P.c.d_log2) >> 3;
    for (int c = t; c < n8; c += GS) {
        float x[8] = {};
        if (have) {
            const uint2 u = __ldcs(reinterpret_cast<const uint2*>(codes) + c);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float2 a = float2_of(half2_of_lo(i ? u.y : u.x)), b = float2_of(half2_of_hi(i ? u.y : u.x));
                x[4 * i] = a.x * f;
                x[4 * i + 1] = a.y * f;
                x[4 * i + 2] = b.x * f;
                x[4 * i + 3] = b.y * f;
            }
        }
        store8(dst + 8 * c, x);
    }
}

// Blocks that one sequence of a call can touch, wherever its first token lies in a page.
int items_of(const Cache& c, const Seqs& q) {
    return static_cast<int>((static_cast<int64_t>(q.max_tokens) + c.page - 2) / c.page + 1);
}

// Threads for a block: enough to hold the most new values that a block can get, four
// chunks each, so that a few tokens take a warp a block and a whole page a CTA.
int group_size(const Cache& c, const Seqs& q) {
    const int values = (q.max_tokens < c.page ? q.max_tokens : c.page) * c.d;
    int gs = 32;
    while (gs * CHUNKS * 8 < values) gs *= 2;
    return gs;  // at most 512: 128 tokens of 128
}

RwParams params(const Cache& c, const Seqs& q, const Err& err) {
    RwParams P{};
    P.c = c;
    P.q = q;
    P.items = items_of(c, q);
    P.total = static_cast<int64_t>(P.items) * q.n_seq * c.H * c.n_layers * 2;
    P.err = err;
    return P;
}

template <typename T, int GS>
cudaError_t launch_write_gs(const RwParams& P, cudaStream_t s) {
    constexpr int PER = GS > NT ? 1 : NT / GS;
    write_kernel<T, GS><<<static_cast<unsigned>((P.total + PER - 1) / PER), GS > NT ? GS : NT, 0, s>>>(P);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_write_t(const RwParams& P, int gs, cudaStream_t s) {
    switch (gs) {
        case 32: return launch_write_gs<T, 32>(P, s);
        case 64: return launch_write_gs<T, 64>(P, s);
        case 128: return launch_write_gs<T, 128>(P, s);
        case 256: return launch_write_gs<T, 256>(P, s);
        default: return launch_write_gs<T, 512>(P, s);
    }
}

template <typename T>
cudaError_t launch_read_t(const RwParams& P, int gs, cudaStream_t s) {
    const int per = gs == 32 ? NT / 32 : 1;
    const unsigned grid = static_cast<unsigned>((P.total + per - 1) / per);
    if (gs == 32) read_kernel<T, 32><<<grid, NT, 0, s>>>(P);
    else read_kernel<T, NT><<<grid, NT, 0, s>>>(P);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_write(const Cache& c, const Seqs& q, kvb_dtype dtype, const void* k, const void* v, const Err& err,
                         cudaStream_t s) {
    RwParams P = params(c, q, err);
    P.src[0] = k;
    P.src[1] = v;
    return dtype == KVB_BF16 ? launch_write_t<__nv_bfloat16>(P, group_size(c, q), s)
                             : launch_write_t<float>(P, group_size(c, q), s);
}

cudaError_t launch_read(const Cache& c, const Seqs& q, kvb_dtype dtype, void* k, void* v, const Err& err,
                        cudaStream_t s) {
    RwParams P = params(c, q, err);
    P.dst[0] = k;
    P.dst[1] = v;
    return dtype == KVB_BF16 ? launch_read_t<__nv_bfloat16>(P, group_size(c, q), s)
                             : launch_read_t<float>(P, group_size(c, q), s);
}

}  // namespace c8
}  // namespace kvb
