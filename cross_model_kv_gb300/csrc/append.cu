// Appending keys and values to the paged caches, with the position rotation applied on the way.
//
// A row x at position p becomes (pairs i, i + d/2)
//     x'_i = x_i c_i - x_{i+d/2} s_i,  x'_{i+d/2} = x_{i+d/2} c_i + x_i s_i
// with (c_i, s_i) of position p from the context's table.  A thread owns 16 bytes of the low half
// of a row and the 16 bytes of the high half that they pair with.  Each product and each sum is
// rounded by itself: what fp32 tensors multiplied and added element by element give, bit for
// bit, so that a block's scale in the 8-bit cache does not hang on the order of an FMA.
// Memory bounds both kernels: 3 flops an element against 3 to 8 bytes.  8192 tokens of a layer, 64 query and 8 KV heads of
// 128, bf16: 54.3 us (6.2 TB/s moved, 0.91 of the copy rate), into 8 bits 57.7 (5.5 TB/s); 64 layers without rotation 620
// us (6.9 TB/s); one token 2.7 us, a launch.
#include "paged.h"

namespace kvb {
namespace paged {

namespace {

constexpr int NT = 256;
// CTAs an SM to share the jobs of the same tokens among: 8192 tokens of 64 + 16 heads take 55.9 us with 4, 54.3 with 12 and 24.
constexpr double CTAS_AN_SM = 12;

template <typename T>
struct Vec;  // 16 bytes of a row
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void get(const uint4& u, float (&x)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 put(const float (&x)[8]) {
        return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    }
};
template <>
struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void get(const uint4& u, float (&x)[4]) {
        x[0] = __uint_as_float(u.x);
        x[1] = __uint_as_float(u.y);
        x[2] = __uint_as_float(u.z);
        x[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ uint4 put(const float (&x)[4]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
};

__device__ __forceinline__ uint4 load16(const void* p) { return __ldcs(static_cast<const uint4*>(p)); }

// The table's entries of N pairs from pair i0 of position p on.
template <int N>
struct Turn {
    float c[N], s[N];
    __device__ __forceinline__ void load(const float2* tab, int64_t at) {
        const float4* t = reinterpret_cast<const float4*>(tab + at);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const float4 x = __ldg(t + i);
            c[2 * i] = x.x;
            s[2 * i] = x.y;
            c[2 * i + 1] = x.z;
            s[2 * i + 1] = x.w;
        }
    }
    __device__ __forceinline__ void apply(float (&lo)[N], float (&hi)[N]) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {  // (as f32x2 the products are fused with the sums)
            const float a = lo[i], b = hi[i];
            lo[i] = __fsub_rn(__fmul_rn(a, c[i]), __fmul_rn(b, s[i]));
            hi[i] = __fadd_rn(__fmul_rn(b, c[i]), __fmul_rn(a, s[i]));
        }
    }
};

// How rows are spread over CTAs.  A CTA has NT / chunks row slots: `tokens` of them take as many
// tokens of one sequence, the rest (lanes) share their heads.  A job is a KV head's k and v, or
// two query heads; `groups` CTAs share the jobs of the same tokens.
struct Spread {
    int chunks_log2, tokens_log2, lanes, jobs, kv_jobs, groups;
    int blocks;  // of tokens, a sequence
    int64_t ctas;
};

struct RowArgs {
    AppendParams P;
    Spread S;
};

// CTA `cta` of S.ctas: its tokens' rows rotated and stored.  KV: there are k and v jobs.
// The table's entries and the page of a token serve all its heads.
template <typename T, bool ROTATE, bool KV>
__device__ __forceinline__ void append_rows(const AppendParams& P, const Spread& S, int64_t cta, int thread) {
    constexpr int N = Vec<T>::N;
    const int half = P.c.d >> 1;
    const int c = thread & ((1 << S.chunks_log2) - 1);
    const int slot = thread >> S.chunks_log2;
    const int ti = slot & ((1 << S.tokens_log2) - 1), lane = slot >> S.tokens_log2;
    uint32_t x = static_cast<uint32_t>(cta);  // ctas < 2^31
    const int tb = x % S.blocks;
    x /= S.blocks;
    const int s = x % P.q.n_seq;
    x /= P.q.n_seq;
    const int group = x % S.groups, l = x / S.groups;
    const c8::SeqView sv = c8::seq_view(P.q, s, P.err);
    const int i = (tb << S.tokens_log2) + ti;
    if (i >= sv.n) return;
    const int pos = sv.pos + i;  // seq_view: no overflow
    const int64_t tok = static_cast<int64_t>(sv.tok0) + i;
    if (!KVB_IN_BOUNDS(P.err, tok, 1, P.q.T) || !KVB_IN_BOUNDS(P.err, l, 1, P.c.n_layers)) return;
    const int e0 = c * N;  // elements e0 .. e0 + N - 1 and the same of the high half

    int pid = -1;
    const int logical = pos >> P.c.page_log2;
    if constexpr (KV)
        if (pos >= 0 && logical < P.q.max_pages && c8::table_in_bounds(P.q, P.err, s, logical))
            pid = __ldg(P.q.page_table + static_cast<int64_t>(s) * P.q.max_pages + logical);
    const bool turned = !ROTATE || (pos >= 0 && pos < P.max_pos);
    Turn<N> turn;
    if (ROTATE && turned && KVB_IN_BOUNDS(P.err, static_cast<int64_t>(pos) * half + e0, N, static_cast<int64_t>(P.max_pos) * half))
        turn.load(P.tab, static_cast<int64_t>(pos) * half + e0);

    const int step = S.lanes * S.groups;
    struct Job {
        uint4 a, b, c, d;  // k and v, or two query heads: low and high halves
    };
    auto row = [&](const Rows& r, int h) -> T* {
        return static_cast<T*>(r.data) + (l * r.l + h * r.h + tok * r.t + e0);
    };
    auto load = [&](int j, Job& w) {
        if (KV && j < S.kv_jobs) {
            const T *k = row(P.src[0], j), *v = row(P.src[1], j);
            w.a = load16(k);
            w.b = load16(k + half);
            w.c = load16(v);
            w.d = load16(v + half);
        } else if (ROTATE) {
            const int h = 2 * (j - S.kv_jobs);
            const T* q = row(P.qs, h);
            w.a = load16(q);
            w.b = load16(q + half);
            if (h + 1 < P.Hq) {
                const T* q1 = row(P.qs, h + 1);
                w.c = load16(q1);
                w.d = load16(q1 + half);
            }
        }
    };
    auto rotate = [&](uint4& u, uint4& v) {
        float lo[N], hi[N];
        Vec<T>::get(u, lo);
        Vec<T>::get(v, hi);
        turn.apply(lo, hi);
        u = Vec<T>::put(lo);
        v = Vec<T>::put(hi);
        if (!turned) u = v = make_uint4(0, 0, 0, 0);
    };
    const int64_t layer = static_cast<int64_t>(P.c.l_begin) + l;
    auto store = [&](int j, Job& w) {
        if (ROTATE) rotate(w.a, w.b);
        if (KV && j < S.kv_jobs) {
            if (!turned) w.c = w.d = make_uint4(0, 0, 0, 0);
            if (pid < 0) return;
            const int64_t blk = (layer * P.c.n_pages + pid) * P.c.H + j;
            if (!KVB_IN_BOUNDS(P.err, blk, 1, (static_cast<int64_t>(P.c.l_begin) + P.c.n_layers) * P.c.n_pages * P.c.H)) return;
            const int64_t at = (((blk << P.c.page_log2) + (pos & (P.c.page - 1))) << P.c.d_log2) + e0;
            T *k = static_cast<T*>(P.c.kv[0]) + at, *v = static_cast<T*>(P.c.kv[1]) + at;
            *reinterpret_cast<uint4*>(k) = w.a;
            *reinterpret_cast<uint4*>(k + half) = w.b;
            *reinterpret_cast<uint4*>(v) = w.c;
            *reinterpret_cast<uint4*>(v + half) = w.d;
        } else if (ROTATE) {
            const int h = 2 * (j - S.kv_jobs);
            T* q = row(P.qo, h);
            *reinterpret_cast<uint4*>(q) = w.a;
            *reinterpret_cast<uint4*>(q + half) = w.b;
            if (h + 1 < P.Hq) {
                rotate(w.c, w.d);
                T* q1 = row(P.qo, h + 1);
                *reinterpret_cast<uint4*>(q1) = w.c;
                *reinterpret_cast<uint4*>(q1 + half) = w.d;
            }
        }
    };
    int j = lane * S.groups + group;
    if (j >= S.jobs) return;
    Job w0, w1;
    load(j, w0);
    if (j + step < S.jobs) load(j + step, w1);
    if (c == 0 && j == 0 && !turned) c8::err_set(P.err, DEV_ERR_BAD_POS);
    if constexpr (KV)
        if (pid < 0 || pid >= P.c.n_pages) {
            if (c == 0 && j == 0) c8::err_set(P.err, DEV_ERR_BAD_SEQ);
            pid = -1;
        }
    for (;;) {
        store(j, w0);
        if (j + 2 * step < S.jobs) load(j + 2 * step, w0);
        if (j + step >= S.jobs) return;
        store(j + step, w1);
        if (j + 3 * step < S.jobs) load(j + 3 * step, w1);
        j += 2 * step;
        if (j >= S.jobs) return;
    }
}

template <typename T, bool ROTATE>
__global__ void __launch_bounds__(NT, 3) append_kernel(const __grid_constant__ RowArgs A) {
    append_rows<T, ROTATE, true>(A.P, A.S, blockIdx.x, threadIdx.x);
}

int log2_up(int64_t x) {  // the smallest n with 2^n >= x
    int n = 0;
    while ((int64_t{1} << n) < x) ++n;
    return n;
}

// As many tokens a CTA as a sequence has, so that the table's entries serve all heads of a long
// call, and jobs over the lanes that are left; then over more CTAs where there would be few.
Spread spread(const AppendParams& P, size_t element, bool kv, int num_sms) {
    Spread S{};
    const int chunks = P.c.d / (32 / static_cast<int>(element));
    S.chunks_log2 = log2_up(chunks);
    const int slots = NT / chunks;
    const int most = log2_up(P.q.max_tokens), cap = log2_up(slots);
    S.tokens_log2 = most < cap ? most : cap;
    S.lanes = slots >> S.tokens_log2;
    S.kv_jobs = kv ? P.c.H : 0;
    S.jobs = S.kv_jobs + (P.Hq + 1) / 2;
    S.blocks = static_cast<int>((static_cast<int64_t>(P.q.max_tokens) + (1 << S.tokens_log2) - 1) >> S.tokens_log2);
    const double one = static_cast<double>(S.blocks) * P.q.n_seq * P.c.n_layers;
    S.groups = 1;
    while (one * S.groups < CTAS_AN_SM * num_sms && S.groups * S.lanes * 2 < S.jobs) S.groups *= 2;
    S.ctas = one * S.groups > 2147483647.0 ? -1 : static_cast<int64_t>(S.blocks) * P.q.n_seq * P.c.n_layers * S.groups;
    return S;
}

template <typename T>
cudaError_t launch_append_t(const AppendParams& P, int num_sms, cudaStream_t s) {
    const RowArgs A{P, spread(P, sizeof(T), true, num_sms)};
    if (P.rotate)
        append_kernel<T, true><<<static_cast<unsigned>(A.S.ctas), NT, 0, s>>>(A);
    else
        append_kernel<T, false><<<static_cast<unsigned>(A.S.ctas), NT, 0, s>>>(A);
    return cudaGetLastError();
}

// ------------------------------------------------------------------ into the 8-bit cache

struct Append8Args {
    AppendParams P;
    c8::Cache c;
    Spread S;       // the queries' CTAs, after those of the blocks
    int items;      // pages that one sequence can touch
    int heads;      // that a group of threads takes one after another
    int shares;     // of the heads: H / heads, rounded up
    int64_t total;  // items * n_seq * shares * n_layers
    unsigned block_ctas;
};

constexpr int INF_BITS = 0x7f800000;
__device__ __forceinline__ int magnitude(float x) { return __float_as_int(x) & 0x7fffffff; }
// The largest magnitude of three, NaN if there is one.
__device__ __forceinline__ float top3(float a, float b, float c) {
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float top8(float m, const float (&x)[8]) {
    return top3(top3(top3(m, x[0], x[1]), x[2], x[3]), top3(0.f, x[4], x[5]), top3(0.f, x[6], x[7]));
}

__device__ __forceinline__ uint2 codes8(const float (&x)[8], float inv) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 y = mul2(make_float2(x[2 * i], x[2 * i + 1]), make_float2(inv, inv));
        w[i] = c8::e4m3x2(y.x, y.y);
    }
    return make_uint2(__byte_perm(w[0], w[1], 0x5410), __byte_perm(w[2], w[3], 0x5410));
}

// A thread's rows on their way: 16-byte pieces of its K and V chunks, in shared memory, one head a stage.
// It reads what it copied itself, so that no thread waits for another's.
template <typename T, int GS, int PAIRS>
struct Stages {
    static constexpr int THREADS = GS > NT ? GS : NT;
    static constexpr int N16 = sizeof(T) / 2;            // pieces of 8 elements
    static constexpr int PIECES = PAIRS * 4 * N16;       // of a thread: low and high of k, of v
    static constexpr int DEPTH = PIECES * THREADS * 32 <= 131072 ? 2 : 1;
    static constexpr int BYTES = DEPTH * PIECES * THREADS * 16;
};

// One page's K and V blocks of one head after another per group of GS threads, as write_kernel of the
// 8-bit cache does it, of rows with strides and rotated keys: a thread's keys are the low and high chunk
// of a pair, held in fp32 after the rotation, between the block's maximum and the rounding.  The table's
// entries serve all heads, and the next heads' rows are on their way while a block is rounded: with a
// block a group, read into registers, none were (32 layers of 8192 tokens, 8 heads of 128, bf16: 504 us; one
// head ahead in registers 352).  Then the instructions bound it, 17.7 an element: addresses taken once for
// all heads, maxima of three numbers, a warp's look at the other warps' maxima made 274 us of 319, 5.9 TB/s.
// 64 registers a thread and 1024 threads an SM; with 80 and 768 it takes 311.
// The CTAs after the blocks' rotate the queries.
// PAIRS: pairs of a thread, 1 but for pages of 128 tokens of 128.
template <typename T, int GS, int PAIRS>
__global__ void __launch_bounds__(Stages<T, GS, PAIRS>::THREADS, PAIRS == 2 ? 1 : GS > NT ? 2 : 4)
    append8_kernel(const __grid_constant__ Append8Args A) {
    using R = Stages<T, GS, PAIRS>;
    constexpr int PER = GS > NT ? 1 : NT / GS, N16 = R::N16, DEPTH = R::DEPTH;
    const AppendParams& P = A.P;
    const c8::Cache& C = A.c;
    if (blockIdx.x >= A.block_ctas) {
        const int64_t cta = static_cast<int64_t>(blockIdx.x - A.block_ctas) * (R::THREADS / NT) + threadIdx.x / NT;
        if (cta < A.S.ctas) append_rows<T, true, false>(P, A.S, cta, threadIdx.x % NT);
        return;
    }
    extern __shared__ uint4 ring[];  // [DEPTH][PIECES][THREADS]
    const int64_t idx = static_cast<int64_t>(blockIdx.x) * PER + threadIdx.x / GS;
    const int t = threadIdx.x % GS;
    if (idx >= A.total) return;  // whole groups leave together, here and below
    uint32_t x = static_cast<uint32_t>(idx);
    const int item = x % A.items;
    x /= A.items;
    const int s = x % P.q.n_seq;
    x /= P.q.n_seq;
    const int h0 = x % A.shares * A.heads, l = x / A.shares;

    const c8::SeqView sv = c8::seq_view(P.q, s, P.err);
    if (sv.n == 0) return;
    const int pos = max(sv.pos, 0);  // pos < 0 counts as a bad page
    const int64_t logical = (pos >> C.page_log2) + item;
    const int64_t p0 = logical << C.page_log2;
    const int lo = item == 0 ? pos - static_cast<int>(p0) : 0;
    const int m = static_cast<int>(min(static_cast<int64_t>(pos) + sv.n - p0, static_cast<int64_t>(C.page))) - lo;
    if (m <= 0) return;
    const int64_t tok0 = sv.tok0 + (p0 + lo - pos);
    const int pid = logical < P.q.max_pages && c8::table_in_bounds(P.q, P.err, s, logical)
                        ? __ldg(P.q.page_table + static_cast<int64_t>(s) * P.q.max_pages + logical) : -1;

    const int half = C.d >> 1, row_log2 = C.d_log2 - 4;  // pairs of chunks in a row: d / 16
    const int n = m << row_log2;
    const int first = static_cast<int>(p0) + lo;  // position of the item's first token
    if (!KVB_IN_BOUNDS(P.err, tok0, m, P.q.T)) return;
    const int heads = min(A.heads, C.H - h0);
    // this thread's chunks of head h0: where they lie, and where their codes go in a block
    const T* from[PAIRS][2];
    int to[PAIRS];
    bool mine[PAIRS];
#pragma unroll
    for (int c = 0; c < PAIRS; ++c) {
        const int y = c * GS + t, i = y >> row_log2, e0 = (y & ((1 << row_log2) - 1)) * 8;
        mine[c] = y < n;
        to[c] = ((lo + i) << C.d_log2) + e0;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv)
            from[c][kv] = static_cast<const T*>(P.src[kv].data) + (l * P.src[kv].l + h0 * P.src[kv].h + (tok0 + i) * P.src[kv].t + e0);
    }
    uint4* const my_ring = ring + threadIdx.x;
    auto piece = [&](int stage, int i) { return my_ring + (stage * R::PIECES + i) * R::THREADS; };
    // asks for the rows of head h0 + i, i = 0, 1, ..: one group of copies, empty past the last head
    auto ask = [&](int i, int stage) {
        if (i < heads)
#pragma unroll
            for (int c = 0; c < PAIRS; ++c)
                if (mine[c])
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        const T* p = from[c][kv] + i * P.src[kv].h;
#pragma unroll
                        for (int u = 0; u < 2; ++u)
#pragma unroll
                            for (int x = 0; x < N16; ++x)
                                copy16(smem_u32(piece(stage, ((c * 2 + kv) * 2 + u) * N16 + x)), p + u * half + x * Vec<T>::N);
                    }
        copies_commit();
    };
    auto get = [&](int stage, int c, int kv, int u, float (&x)[8]) {
        const int i = ((c * 2 + kv) * 2 + u) * N16;
        if constexpr (N16 == 1) {
            Vec<T>::get(*piece(stage, i), x);
        } else {
            float a[4], b[4];
            Vec<T>::get(*piece(stage, i), a);
            Vec<T>::get(*piece(stage, i + 1), b);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[j] = a[j];
                x[4 + j] = b[j];
            }
        }
    };
#pragma unroll
    for (int i = 0; i < DEPTH; ++i) ask(i, i);
    Turn<8> turn[PAIRS];
    bool outside = false;  // some position is not in the table: keys and values of it count as 0
#pragma unroll
    for (int c = 0; c < PAIRS; ++c) {
        const int y = c * GS + t, at = first + (y >> row_log2), e0 = (y & ((1 << row_log2) - 1)) * 8;
        if (P.rotate && mine[c]) {
            if (at >= P.max_pos) outside = true;
            else if (KVB_IN_BOUNDS(P.err, static_cast<int64_t>(at) * half + e0, 8, static_cast<int64_t>(P.max_pos) * half))
                turn[c].load(P.tab, static_cast<int64_t>(at) * half + e0);
        }
    }
    if (outside) c8::err_set(P.err, DEV_ERR_BAD_POS);
    auto in_table = [&](int c) { return !outside || first + ((c * GS + t) >> row_log2) < P.max_pos; };
    const int64_t block0 = ((static_cast<int64_t>(C.l_begin) + l) * C.n_pages + pid) * C.H + h0;
    const bool bad_page = pid < 0 || pid >= C.n_pages || sv.pos < 0;
    if (bad_page && t == 0) c8::err_set(P.err, DEV_ERR_BAD_SEQ);
    if (bad_page || !KVB_IN_BOUNDS(P.err, block0, heads, c8::blocks_of(C)) || !KVB_IN_BOUNDS(P.err, lo, m, C.page)) {
        copies_wait<0>();
        return;
    }

    // The group's largest magnitudes, as the bits of fp32 numbers; the barrier also lets every thread read
    // the old scales.  Heads take turns at two places for them, and a head that is looked at twice has a third.
    constexpr int W = GS > 32 ? GS / 32 : 1;
    __shared__ int tops[3][PER][2 * W];
    auto over_group = [&](int (&top)[2], int place) {
        top[0] = __reduce_max_sync(0xffffffffu, top[0]);
        top[1] = __reduce_max_sync(0xffffffffu, top[1]);
        if constexpr (GS > 32) {
            const int group = threadIdx.x / GS, lane = t & 31;
            if (lane < 2) tops[place][group][lane * W + (t >> 5)] = top[lane];
            named_bar_sync(1 + group, GS);
            const int x = lane < 2 * W ? tops[place][group][lane] : 0;  // K's, then V's
            top[0] = __reduce_max_sync(0xffffffffu, lane < W ? x : 0);
            top[1] = __reduce_max_sync(0xffffffffu, lane < W ? 0 : x);
        } else {
            __syncwarp();
        }
    };
    for (int i = 0; i < heads; ++i) {
        const int64_t block = block0 + i;
        const int stage = DEPTH == 1 ? 0 : i % DEPTH;
        int e_old[2] = {c8::E_MIN, c8::E_MIN};
        if (lo > 0)
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) e_old[kv] = min(max(c8::exponent_of(C.scale[kv][block]), c8::E_MIN), c8::E_MAX);
        copies_wait<DEPTH - 1>();
        float k[PAIRS][2][8];
        float tk = 0.f, tv = 0.f;
        auto value = [&](int c, int u, float (&y)[8]) {
            get(stage, c, 1, u, y);
            if (!in_table(c))
#pragma unroll
                for (int x = 0; x < 8; ++x) y[x] = 0.f;
        };
#pragma unroll
        for (int c = 0; c < PAIRS; ++c)
            if (mine[c]) {
#pragma unroll
                for (int u = 0; u < 2; ++u) get(stage, c, 0, u, k[c][u]);
                if (P.rotate) turn[c].apply(k[c][0], k[c][1]);
                if (!in_table(c))
#pragma unroll
                    for (int x = 0; x < 8; ++x) k[c][0][x] = k[c][1][x] = 0.f;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    float y[8];
                    value(c, u, y);
                    tk = top8(tk, k[c][u]);
                    tv = top8(tv, y);
                }
            }
        int top[2] = {magnitude(tk), magnitude(tv)};
        over_group(top, i & 1);
        const bool odd = max(top[0], top[1]) >= INF_BITS;  // the group's: some value is not finite
        if (odd) {
            bool bad = false;
            tk = tv = 0.f;
#pragma unroll
            for (int c = 0; c < PAIRS; ++c)
                if (mine[c])
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        float y[8];
                        value(c, u, y);
#pragma unroll
                        for (int x = 0; x < 8; ++x) {
                            bad |= magnitude(k[c][u][x]) >= INF_BITS || magnitude(y[x]) >= INF_BITS;
                            if (magnitude(k[c][u][x]) >= INF_BITS) k[c][u][x] = 0.f;
                            if (magnitude(y[x]) >= INF_BITS) y[x] = 0.f;
                        }
                        tk = top8(tk, k[c][u]);
                        tv = top8(tv, y);
                    }
            if (bad) c8::err_set(P.err, DEV_ERR_NONFINITE);
            top[0] = magnitude(tk);
            top[1] = magnitude(tv);
            over_group(top, 2);
            if constexpr (GS > 32) named_bar_sync(1 + threadIdx.x / GS, GS);  // the third place is free again
        }
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            uint8_t* codes = C.code[kv] + ((block << C.page_log2) << C.d_log2);
            const int e = max(e_old[kv], c8::exponent_for(__int_as_float(top[kv])));
            if (t == 0) C.scale[kv][block] = c8::pow2(e);
            const float inv = c8::pow2(-e);
#pragma unroll
            for (int c = 0; c < PAIRS; ++c)
                if (mine[c])
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        float y[8];  // values are read again: in registers they would cost a CTA on the SM
                        if (kv) {
                            value(c, u, y);
                            if (odd)
#pragma unroll
                                for (int x = 0; x < 8; ++x)
                                    if (magnitude(y[x]) >= INF_BITS) y[x] = 0.f;
                        }
                        *reinterpret_cast<uint2*>(codes + to[c] + u * half) = codes8(kv ? y : k[c][u], inv);
                    }
            if (lo > 0 && e > e_old[kv]) c8::lower_codes(codes, (lo << C.d_log2) >> 3, e_old[kv] - e, t, GS);
        }
        ask(i + DEPTH, stage);  // in this head's place
    }
    copies_wait<0>();
}

template <typename T, int GS, int PAIRS = 1>
cudaError_t launch_append8_gs(Append8Args& A, cudaStream_t s) {
    using R = Stages<T, GS, PAIRS>;
    constexpr int PER = GS > NT ? 1 : NT / GS, ROWS = R::THREADS / NT;
    A.block_ctas = static_cast<unsigned>((A.total + PER - 1) / PER);
    const cudaError_t e = cudaFuncSetAttribute(append8_kernel<T, GS, PAIRS>, cudaFuncAttributeMaxDynamicSharedMemorySize, R::BYTES);
    if (e != cudaSuccess) return e;
    append8_kernel<T, GS, PAIRS><<<static_cast<unsigned>(A.block_ctas + (A.S.ctas + ROWS - 1) / ROWS), R::THREADS, R::BYTES, s>>>(A);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_append8_t(const AppendParams& P, const c8::Cache& c, int num_sms, cudaStream_t s) {
    Append8Args A{};
    A.P = P;
    A.c = c;
    A.items = c8::items_of(c, P.q);
    // threads enough to hold the most new values that a block can get, and heads one after another
    // where that leaves threads enough for every SM
    const int values = (P.q.max_tokens < c.page ? P.q.max_tokens : c.page) * c.d;
    int gs = 32;
    while (gs * 16 < values && gs < 512) gs *= 2;
    const double threads = static_cast<double>(A.items) * P.q.n_seq * c.n_layers * c.H * gs;
    A.heads = 1;
    while (A.heads < c.H && threads / (2 * A.heads) >= 512.0 * num_sms) A.heads *= 2;
    A.shares = (c.H + A.heads - 1) / A.heads;
    A.total = static_cast<int64_t>(A.items) * P.q.n_seq * A.shares * c.n_layers;
    if (P.Hq) A.S = spread(P, sizeof(T), false, num_sms);
    switch (gs) {
        case 32: return launch_append8_gs<T, 32>(A, s);
        case 64: return launch_append8_gs<T, 64>(A, s);
        case 128: return launch_append8_gs<T, 128>(A, s);
        case 256: return launch_append8_gs<T, 256>(A, s);
        default: return values <= 512 * 16 ? launch_append8_gs<T, 512>(A, s) : launch_append8_gs<T, 512, 2>(A, s);
    }
}

}  // namespace

double append_ctas(const AppendParams& P, kvb_dtype dtype, int num_sms) {
    const Spread S = spread(P, dtype == KVB_BF16 ? 2 : 4, P.c.kv[0] != nullptr, num_sms);
    const double rows = static_cast<double>(S.blocks) * P.q.n_seq * P.c.n_layers * S.groups;
    if (P.c.kv[0]) return rows;
    return (P.Hq ? rows : 0.0) + ((static_cast<double>(P.q.max_tokens) + P.c.page - 2) / P.c.page + 1) * P.q.n_seq * P.c.H * P.c.n_layers;
}

cudaError_t launch_append(const AppendParams& P, kvb_dtype dtype, int num_sms, cudaStream_t s) {
    return dtype == KVB_BF16 ? launch_append_t<__nv_bfloat16>(P, num_sms, s) : launch_append_t<float>(P, num_sms, s);
}

cudaError_t launch_append8(const AppendParams& P, const c8::Cache& c, kvb_dtype dtype, int num_sms, cudaStream_t s) {
    return dtype == KVB_BF16 ? launch_append8_t<__nv_bfloat16>(P, c, num_sms, s) : launch_append8_t<float>(P, c, num_sms, s);
}

}  // namespace paged
}  // namespace kvb
