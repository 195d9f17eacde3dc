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
// 8-element chunks of K, and of V, that one thread of a group of gs holds: 32
// registers in all, where the largest group suffices.
__host__ __device__ constexpr int chunks_of(size_t element, int gs) { return element == 4 && gs < 512 ? 2 : 4; }

struct RwParams {
    Cache c;
    Seqs q;
    const void* src[2];  // write
    void* dst[2];        // read
    int items;           // pages that one sequence can touch
    int64_t total;       // items * n_seq * H * n_layers
    Err err;
};

// Item `idx` of a call: the K and V blocks of one page that one sequence's tokens touch.
struct Item {
    int l, h, s, i;
};
__device__ __forceinline__ Item item_of(const RwParams& P, int64_t idx) {
    uint32_t x = static_cast<uint32_t>(idx);  // total < 2^31
    Item it;
    it.i = x % P.items;
    x /= P.items;
    it.s = x % P.q.n_seq;
    x /= P.q.n_seq;
    it.h = x % P.c.H;
    it.l = x / P.c.H;
    return it;
}

constexpr int INF_BITS = 0x7f800000;

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {  // two products in one instruction
    float2 d;
    asm("{\n\t.reg .b64 x, y, w;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mul.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// Eight elements as they lie in memory.  top(): the largest magnitude as the bits of
// an fp32 number (non-negative floats order as their bits, infinities and NaN above
// all others); get(): the elements as fp32.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
    uint4 u;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = __ldcs(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ int top() const {
        const uint32_t a = 0x7fff7fffu;
        const uint32_t m = __vmaxu2(__vmaxu2(u.x & a, u.y & a), __vmaxu2(u.z & a, u.w & a));
        return static_cast<int>(max(m << 16, m & 0xffff0000u));
    }
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
    __device__ __forceinline__ int top() const {
        float o[8];
        get(o);
        int m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_int(o[i]) & 0x7fffffff);
        return m;
    }
    __device__ __forceinline__ void get(float (&o)[8]) const {
        o[0] = a.x; o[1] = a.y; o[2] = a.z; o[3] = a.w;
        o[4] = b.x; o[5] = b.y; o[6] = b.z; o[7] = b.w;
    }
};
__device__ __forceinline__ bool finite(float x) { return (__float_as_int(x) & 0x7fffffff) < INF_BITS; }

// What a group of threads does for one item.
struct Place {
    int lo, m;       // the page's slots [lo, lo + m) are the call's
    int64_t row;     // first of them in [n_layers][H][T]
    int64_t block;   // in [L_tgt][n_pages][H]; negative: the page is bad
};
// false: the item has no tokens.  pos < 0 counts as a bad page.
__device__ __forceinline__ bool place_of(const RwParams& P, const Item& it, bool report, Place& o) {
    const SeqView sv = seq_view(P.q, it.s, P.err);
    if (sv.n == 0) return false;
    const int pos = max(sv.pos, 0);
    const int64_t logical = (pos >> P.c.page_log2) + it.i;
    const int64_t p0 = logical << P.c.page_log2;
    o.lo = it.i == 0 ? pos - static_cast<int>(p0) : 0;
    o.m = static_cast<int>(min(static_cast<int64_t>(pos) + sv.n - p0, static_cast<int64_t>(P.c.page))) - o.lo;
    if (o.m <= 0) return false;
    o.row = (static_cast<int64_t>(it.l) * P.c.H + it.h) * P.q.T + sv.tok0 + (p0 + o.lo - pos);
    const int pid = logical < P.q.max_pages && table_in_bounds(P.q, P.err, it.s, logical) ? __ldg(P.q.page_table + static_cast<int64_t>(it.s) * P.q.max_pages + logical) : -1;
    const bool bad = pid < 0 || pid >= P.c.n_pages || sv.pos < 0;
    if (bad && report) err_set(P.err, DEV_ERR_BAD_SEQ);
    o.block = bad ? -1 : ((static_cast<int64_t>(P.c.l_begin) + it.l) * P.c.n_pages + pid) * P.c.H + it.h;
    // every access of the item lies in these rows, and in these slots of this block
    return KVB_IN_BOUNDS(P.err, o.row, o.m, static_cast<int64_t>(P.c.n_layers) * P.c.H * P.q.T) &&
           KVB_IN_BOUNDS(P.err, max(o.block, static_cast<int64_t>(0)), 1, blocks_of(P.c)) &&
           KVB_IN_BOUNDS(P.err, o.lo, o.m, P.c.page);
}

// One page's K and V blocks per group of GS threads.  Their new values stay in
// registers, as they lay in memory, between the maximum and the rounding, so they
// are read once; what bounds the kernel is how many loads are in flight (fp32
// copies of eight chunks a thread: two CTAs an SM, 3.1 TB/s; raw, K and V as items of their
// own: 4.7; together, one set of look-ups for twice the bytes: 6.8, 64 layers of 8192 tokens in
// 474 us).
template <typename T, int GS>
__global__ void __launch_bounds__(GS > NT ? GS : NT) write_kernel(const __grid_constant__ RwParams P) {
    constexpr int PER = GS > NT ? 1 : NT / GS, CHUNKS = chunks_of(sizeof(T), GS);
    const int64_t idx = static_cast<int64_t>(blockIdx.x) * PER + threadIdx.x / GS;
    const int t = threadIdx.x % GS;
    if (idx >= P.total) return;  // whole groups leave together, here and below
    const Item it = item_of(P, idx);
    Place at;
    if (!place_of(P, it, t == 0, at) || at.block < 0) return;
    const int n8 = (at.m << P.c.d_log2) >> 3;

    Raw8<T> raw[2][CHUNKS];
#pragma unroll
    for (int kv = 0; kv < 2; ++kv)
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c)
            if (c * GS + t < n8) raw[kv][c].load(static_cast<const T*>(P.src[kv]) + (at.row << P.c.d_log2) + 8 * (c * GS + t));
    int e_old[2] = {E_MIN, E_MIN};
    if (at.lo > 0)
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) e_old[kv] = min(max(exponent_of(P.c.scale[kv][at.block]), E_MIN), E_MAX);
    // the group's largest magnitudes; the barrier also lets every thread read the old scales
    auto over_group = [&](int (&top)[2]) {
        top[0] = __reduce_max_sync(0xffffffffu, top[0]);
        top[1] = __reduce_max_sync(0xffffffffu, top[1]);
        if constexpr (GS > 32) {
            __shared__ int tops[PER][2][GS / 32];
            const int group = threadIdx.x / GS;
            if ((t & 31) == 0) {
                tops[group][0][t >> 5] = top[0];
                tops[group][1][t >> 5] = top[1];
            }
            named_bar_sync(1 + group, GS);
#pragma unroll
            for (int w = 0; w < GS / 32; ++w) {
                top[0] = max(top[0], tops[group][0][w]);
                top[1] = max(top[1], tops[group][1][w]);
            }
        } else {
            __syncwarp();
        }
    };
    int top[2] = {0, 0};
#pragma unroll
    for (int kv = 0; kv < 2; ++kv)
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c)
            if (c * GS + t < n8) top[kv] = max(top[kv], raw[kv][c].top());
    over_group(top);
    const bool odd = max(top[0], top[1]) >= INF_BITS;  // the group's: some value is not finite
    if (odd) {
        if constexpr (GS > 32) named_bar_sync(1 + threadIdx.x / GS, GS);  // the maxima have been read
        bool bad = false;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            top[kv] = 0;
#pragma unroll
            for (int c = 0; c < CHUNKS; ++c)
                if (c * GS + t < n8) {
                    float x[8];
                    raw[kv][c].get(x);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        bad |= !finite(x[i]);
                        if (finite(x[i])) top[kv] = max(top[kv], __float_as_int(x[i]) & 0x7fffffff);
                    }
                }
        }
        if (bad) err_set(P.err, DEV_ERR_NONFINITE);
        over_group(top);
    }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        uint8_t* codes = P.c.code[kv] + ((at.block << P.c.page_log2) << P.c.d_log2);
        const int e = max(e_old[kv], exponent_for(__int_as_float(top[kv])));
        if (t == 0) P.c.scale[kv][at.block] = pow2(e);
        const float inv = pow2(-e);
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c)
            if (c * GS + t < n8) {
                float x[8];
                raw[kv][c].get(x);
                if (odd) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = finite(x[i]) ? x[i] : 0.f;
                }
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 y = mul2(make_float2(x[2 * i], x[2 * i + 1]), make_float2(inv, inv));
                    w[i] = e4m3x2(y.x, y.y);
                }
                *reinterpret_cast<uint2*>(codes + (at.lo << P.c.d_log2) + 8 * (c * GS + t)) =
                    make_uint2(__byte_perm(w[0], w[1], 0x5410), __byte_perm(w[2], w[3], 0x5410));
            }
        if (at.lo > 0 && e > e_old[kv]) {  // the slots before the new tokens, under the larger scale
            const float f = pow2(max(e_old[kv] - e, -126));
            for (int c = t; c < (at.lo << P.c.d_log2) >> 3; c += GS) {
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
}

// 16 bytes of output from as many codes as give them.
__device__ __forceinline__ uint2 load_codes(const uint8_t* p, __nv_bfloat16) { return __ldcs(reinterpret_cast<const uint2*>(p)); }
__device__ __forceinline__ uint2 load_codes(const uint8_t* p, float) {
    return make_uint2(__ldcs(reinterpret_cast<const uint32_t*>(p)), 0u);
}
__device__ __forceinline__ void store_values(__nv_bfloat16* p, uint2 u, float f) {
    const float2 a = float2_of(half2_of_lo(u.x)), b = float2_of(half2_of_hi(u.x));
    const float2 c = float2_of(half2_of_lo(u.y)), d = float2_of(half2_of_hi(u.y));
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(pack_bf16x2(a.x * f, a.y * f), pack_bf16x2(b.x * f, b.y * f),
                                                   pack_bf16x2(c.x * f, c.y * f), pack_bf16x2(d.x * f, d.y * f)));
}
__device__ __forceinline__ void store_values(float* p, uint2 u, float f) {
    const float2 a = float2_of(half2_of_lo(u.x)), b = float2_of(half2_of_hi(u.x));
    __stcs(reinterpret_cast<float4*>(p), make_float4(a.x * f, a.y * f, b.x * f, b.y * f));
}

// One page's K and V blocks per group of GS threads; every store of a thread is 16
// bytes next to its neighbour's, several of them in flight; code * 2^e is exact in
// fp32 and in bf16.  64 layers of 8192 tokens to bf16: 470 us, the copy rate.
template <typename T, int GS>
__global__ void __launch_bounds__(NT) read_kernel(const __grid_constant__ RwParams P) {
    const int64_t idx = static_cast<int64_t>(blockIdx.x) * (NT / GS) + threadIdx.x / GS;
    const int t = threadIdx.x % GS;
    if (idx >= P.total) return;
    const Item it = item_of(P, idx);
    Place at;
    if (!place_of(P, it, t == 0, at)) return;
    const bool have = at.block >= 0;
    const int64_t block = have ? at.block : 0;
    const uint8_t* codes[2];
    T* dst[2];
    float f[2];
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        codes[kv] = P.c.code[kv] + ((block << P.c.page_log2) << P.c.d_log2) + (at.lo << P.c.d_log2);
        dst[kv] = static_cast<T*>(P.dst[kv]) + (at.row << P.c.d_log2);
        f[kv] = have ? __ldg(P.c.scale[kv] + block) : 0.f;
    }
    constexpr int VEC = 16 / sizeof(T), AHEAD = sizeof(T);  // codes of a store; stores in flight, of K and of V
    const int n = (at.m << P.c.d_log2) / VEC;
    for (int c0 = t; c0 < n; c0 += AHEAD * GS) {
        uint2 u[2][AHEAD];
#pragma unroll
        for (int kv = 0; kv < 2; ++kv)
#pragma unroll
            for (int j = 0; j < AHEAD; ++j)
                u[kv][j] = have && c0 + j * GS < n ? load_codes(codes[kv] + VEC * (c0 + j * GS), T()) : make_uint2(0, 0);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv)
#pragma unroll
            for (int j = 0; j < AHEAD; ++j)
                if (c0 + j * GS < n) store_values(dst[kv] + VEC * (c0 + j * GS), u[kv][j], f[kv]);
    }
}

// Pages that one sequence of a call can touch, wherever its first token lies in a page.
int items_of(const Cache& c, const Seqs& q) {
    return static_cast<int>((static_cast<int64_t>(q.max_tokens) + c.page - 2) / c.page + 1);
}

// Threads for an item: enough to hold the most new values that a block can get, so
// that a few tokens take a warp an item and a whole page a CTA.
int group_size(const Cache& c, const Seqs& q, size_t element) {
    const int values = (q.max_tokens < c.page ? q.max_tokens : c.page) * c.d;
    int gs = 32;
    while (gs * chunks_of(element, gs) * 8 < values) gs *= 2;
    return gs;  // at most 512: 128 tokens of 128
}

RwParams params(const Cache& c, const Seqs& q, const Err& err) {
    RwParams P{};
    P.c = c;
    P.q = q;
    P.items = items_of(c, q);
    P.total = static_cast<int64_t>(P.items) * q.n_seq * c.H * c.n_layers;
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
    return dtype == KVB_BF16 ? launch_write_t<__nv_bfloat16>(P, group_size(c, q, 2), s)
                             : launch_write_t<float>(P, group_size(c, q, 4), s);
}

cudaError_t launch_read(const Cache& c, const Seqs& q, kvb_dtype dtype, void* k, void* v, const Err& err,
                        cudaStream_t s) {
    RwParams P = params(c, q, err);
    P.dst[0] = k;
    P.dst[1] = v;
    return dtype == KVB_BF16 ? launch_read_t<__nv_bfloat16>(P, group_size(c, q, 2), s)
                             : launch_read_t<float>(P, group_size(c, q, 2), s);
}

}  // namespace c8
}  // namespace kvb
