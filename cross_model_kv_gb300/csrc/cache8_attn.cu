// Attention over the paged 8-bit cache: few query rows over many keys.
//
// For the g * n query rows of a (layer, sequence, KV head):
//     s_rj = scale * q_r . k_j,  p_rj = 2^(s_rj log2(e) - m_r),
//     o_r = sum_j p_rj v_j / sum_j p_rj.
// Decoding reads every code once for 4 d g flops per 2 d bytes (16 flop/byte
// at g = 8), far below the machine's ratio, so HBM bounds it and the layout
// serves the loads: a warp takes 16 keys at a time straight from global memory
// to registers, in the fragment order of mma.m16n8k16, with the keys as the
// M rows.  Both contractions let their index be permuted freely:
//   S^T = K Q^T  M = 16 keys, K = 16 dims, N = 8 query rows.  Lane (r, c) =
//                (lane / 4, lane % 4) holds d/4 consecutive codes of keys r and
//                r + 8; k step t takes its bytes 4t .. 4t+3, and Q is laid out to match.
//   O^T = V^T P^T  M = 16 dims, K = 16 keys.  Lane (r, c) holds d/8 consecutive
//                codes of keys 2c, 2c+1, 2c+8, 2c+9; a byte permute pairs two
//                keys' codes of one dim, which is an A register after the
//                conversion.  P^T comes from S^T by an 8 x 8 transpose in registers.
// e4m3 converts to fp16 exactly.  A query row is scaled by a power of two to
// at most 2^14 and enters as fp16 (bf16 rows: exact to 2^-28 of the row's
// largest) or as an fp16 pair (fp32 rows); products and sums are fp32.
//
// Numerators carry the values' scale in the exponent: w_rj = 2^(s_rj log2(e) +
// e_v(j) - mv_r) is what multiplies the codes, and the denominator sums
// 2^(s_rj log2(e) - m_r); each has its own reference, so a page's scale, large
// or small, costs neither range nor bits.  References are raised only when a
// tile exceeds them by 2^8 (one vote per tile); weights are biased by 2^7, so fp16
// holds them from 2^15 down to 2^-24 (2^-31 of the reference).
//
// The keys of all units (layer, sequence, row block, head) form one line of 64-key
// tiles, which the CTAs that fit the GPU share evenly: unequal lengths cost
// nothing, and a CTA pays its set-up once for each unit that it meets.  (Chunks of
// 512 / 2048 keys as CTAs of their own took 588 / 402 us for 32 sequences of 32768
// keys: about 4.6 us a CTA.)  The last CTA to arrive at a unit that several share
// joins its pieces in order, so results do not depend on timing.
// 32 sequences of 32768 keys, one token each, 64 query and 8 KV heads: 338 us a call, 336
// replayed from a graph, 6.4 TB/s (0.94 of the copy rate).
#include <cfloat>

#include "cache8_attn.cuh"

namespace kvb {
namespace c8 {

namespace {

constexpr int WARPS = 4;        // of a CTA; 16 keys each make its step, a tile of the line
constexpr int WARPS_FEW = 8;    // where there are few keys: one CTA an SM, its step 128 keys
constexpr int FEW_TILES = 4;
constexpr int LIST_PAGES = 256;         // pages listed in shared memory at a time

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// W consecutive 32-bit words (B bytes), read once: not kept in L1.  WHOLE: 32 bytes are 32-byte
// aligned and come in one load, else (16-byte aligned) in two.
template <int B, bool WHOLE = true>
__device__ __forceinline__ void load_codes(const uint8_t* p, uint32_t* w) {
    if constexpr (B == 32 && !WHOLE) {
        load_codes<16>(p, w);
        load_codes<16>(p + 16, w + 4);
    } else if constexpr (B == 32) {
        asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                     : "l"(p));
    } else if constexpr (B == 16) {
        asm volatile("ld.global.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "l"(p));
    } else if constexpr (B == 8) {
        asm volatile("ld.global.L1::no_allocate.v2.b32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
    } else if constexpr (B == 4) {
        asm volatile("ld.global.b32 %0, [%1];" : "=r"(w[0]) : "l"(p));
    } else {
        uint16_t h;
        asm volatile("ld.global.b16 %0, [%1];" : "=h"(h) : "l"(p));
        w[0] = h;
    }
}

// n consecutive query elements as fp32.
__device__ __forceinline__ float2 load2(const __nv_bfloat16* p) {
    const uint32_t u = __ldg(reinterpret_cast<const uint32_t*>(p));
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ float2 load2(const float* p) { return __ldg(reinterpret_cast<const float2*>(p)); }
// CTAs to keep on an SM: what the accumulators (D/4 registers a row block) and the
// 64 bytes of codes in flight leave.  What spills for that: bf16, D 128, 8 rows: set-up only
// (counted: 0.1 reloads for each 16 keys of a warp); 16 rows: about 10 of the 447 instructions
// for each 16 keys are reloads, which a third CTA on the SM outweighs.
constexpr int resident_ctas(size_t element, int D, int NB) {
    return D < 64 ? 4 : (NB == 1 ? 4 : 3) - (D == 128 && element == 4 ? 1 : 0);
}

template <typename T, int D, int NB, int NWARPS>
struct Shape8 {
    static constexpr int PARTS = sizeof(T) == 4 ? 2 : 1;  // fp16 parts of a query element and of a weight
    static constexpr int ROWS = 8 * NB;
    static constexpr int KS = D / 16;                     // k steps of S, and M tiles of O
    // per warp: its outputs, references and sums; then the page list of the chunk
    static constexpr int Q_WORDS = PARTS * NB * KS * 2 * 32;
    static constexpr size_t smem() {
        return sizeof(float) * (NWARPS * ROWS * D + NWARPS * ROWS * 4) + 4 * Q_WORDS + (LIST_PAGES + 1) * 12;
    }
};

// WHOLE: key rows can be read 32 bytes at a time (see whole_rows).
template <typename T, int D, int NB, int NWARPS, bool WHOLE>
__global__ void __launch_bounds__(NWARPS * 32, NWARPS == WARPS ? resident_ctas(sizeof(T), D, NB) : 1)
    decode_kernel(const __grid_constant__ AttnParams P) {
    constexpr int NT = NWARPS * 32, TILE_KEYS = 16 * NWARPS;
    constexpr int DEPTH = D <= 64 ? 2 : 1;  // 16-key steps of a warp in flight: 4 KB at d 128 and 64
    using S8 = Shape8<T, D, NB, NWARPS>;
    constexpr int PARTS = S8::PARTS, ROWS = S8::ROWS, KS = S8::KS;
    constexpr int KB = D / 4, VB = D / 8;                    // bytes of a lane: of a key row, of a value row
    constexpr int KW = KB / 4, VW = VB >= 4 ? VB / 4 : 1;    // words
    extern __shared__ float4 sm4[];
    float* so = reinterpret_cast<float*>(sm4);               // [NWARPS][ROWS][D]
    float4* stat = reinterpret_cast<float4*>(so + NWARPS * ROWS * D);  // [NWARPS][ROWS] references and sum
    float* sqs = reinterpret_cast<float*>(stat);             // [ROWS] factors of the query rows, before that
    uint32_t* sq = reinterpret_cast<uint32_t*>(stat + NWARPS * ROWS);  // query fragments
    int* s_page = reinterpret_cast<int*>(sq + S8::Q_WORDS);
    float* s_ks = reinterpret_cast<float*>(s_page + LIST_PAGES + 1);  // key scale
    float* s_ev = s_ks + LIST_PAGES + 1;                              // exponent of the value scale
    __shared__ int s_last;
    __shared__ LineStart s_start;
    __shared__ int s_scan[NWARPS];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = lane >> 2, c = lane & 3;

    int at, stop, share;
    int l, e, h, first;
    if (!line_start<ROWS, TILE_KEYS, NT>(P, s_scan, &s_start, at, stop, share, l, e, h, first)) return;
    const int entries = P.q.n_seq * P.row_blocks;
    auto entry = [&](int e) { return row_block(P, e / P.row_blocks, e % P.row_blocks, ROWS); };
    RowBlock B = entry(e);
    int tiles = unit_tiles<TILE_KEYS>(B);

    // one unit, or a piece of one, after another
    for (;;) {
    const int s = e / P.row_blocks;
    const int last = min(tiles, first + (stop - at));  // tiles [first, last)
    const int k0 = first * TILE_KEYS, k1 = min(B.kv_end, last * TILE_KEYS);
    const int nrows = B.nrows;
    const int row0 = B.row0;
    const int64_t unit = (static_cast<int64_t>(l) * entries + e) * P.c.H + h;
    const int64_t layer = static_cast<int64_t>(P.c.l_begin) + l;

    // pages and scales of the keys from k on, up to LIST_PAGES pages' worth
    int page0 = 0;
    auto list_pages = [&](int k) {
        page0 = k >> P.c.page_log2;
        const int span = LIST_PAGES << P.c.page_log2;
        const int end = k1 - k > span ? k + span : k1;  // k + span may pass 2^31
        const int npages = end > k ? ((end - 1) >> P.c.page_log2) - page0 + 1 : 0;
        for (int i = threadIdx.x; i < npages; i += NT) {
            int pid = table_in_bounds(P.q, P.err, s, page0 + i) ? __ldg(P.q.page_table + static_cast<int64_t>(s) * P.q.max_pages + page0 + i) : -1;
            if (pid < 0 || pid >= P.c.n_pages) {
                err_set(P.err, DEV_ERR_BAD_SEQ);
                pid = -1;
            }
            const int64_t b = (layer * P.c.n_pages + pid) * P.c.H + h;
            if (pid >= 0 && !KVB_IN_BOUNDS(P.err, b, 1, blocks_of(P.c))) pid = -1;
            s_page[i] = pid;
            s_ks[i] = pid < 0 ? 1.f : __ldg(P.c.scale[0] + b);
            s_ev[i] = pid < 0 ? 0.f : static_cast<float>(exponent_of(__ldg(P.c.scale[1] + b)));
        }
        return end;
    };
    // the rows' elements are asked for first, then the pages; the first codes come while the
    // rows are laid out (row block b by warp b % NWARPS; every warp needs all of them)
    const T* query = static_cast<const T*>(P.query);
    const int64_t hq0 = (static_cast<int64_t>(l) * P.c.H + h) * P.g;
    constexpr int QB = (NB + NWARPS - 1) / NWARPS;
    float q[QB][KB];
#pragma unroll
    for (int i = 0; i < QB; ++i) {
        const int row = 8 * (warp + i * NWARPS) + r;
        if (row < nrows && KVB_IN_BOUNDS(P.err, B.row_of(P, hq0, row), 1, rows_of(P))) {
            const T* p = query + B.row_of(P, hq0, row) * D + c * KB;
#pragma unroll
            for (int x = 0; x < KB; x += 2) {
                const float2 y = load2(p + x);
                q[i][x] = y.x;
                q[i][x + 1] = y.y;
            }
        } else {
#pragma unroll
            for (int x = 0; x < KB; ++x) q[i][x] = 0.f;
        }
    }
    int listed = list_pages(k0);
    __syncthreads();
    const int64_t slab = layer * P.c.n_pages * P.c.H + h;  // block of page 0
    uint32_t kr[DEPTH][2][KW], vr[DEPTH][4][VW];
    auto load_k = [&](int j, uint32_t (&kw)[2][KW]) {
        const int pi = (j >> P.c.page_log2) - page0;
        if (s_page[pi] < 0) {  // every key of the page is masked
#pragma unroll
            for (int x = 0; x < KW; ++x) kw[0][x] = kw[1][x] = 0;
            return;
        }
        const int64_t blk = slab + static_cast<int64_t>(s_page[pi]) * P.c.H;
        const uint8_t* p = P.c.code[0] + ((blk << P.c.page_log2) + (j & (P.c.page - 1))) * D;
        load_codes<KB, WHOLE>(p + r * D + c * KB, kw[0]);
        load_codes<KB, WHOLE>(p + (r + 8) * D + c * KB, kw[1]);
    };
    auto load_v = [&](int j, uint32_t (&vw)[4][VW]) {
        const int pi = (j >> P.c.page_log2) - page0;
        if (s_page[pi] < 0) {
#pragma unroll
            for (int x = 0; x < VW; ++x) vw[0][x] = vw[1][x] = vw[2][x] = vw[3][x] = 0;
            return;
        }
        const int64_t blk = slab + static_cast<int64_t>(s_page[pi]) * P.c.H;
        const uint8_t* p = P.c.code[1] + ((blk << P.c.page_log2) + (j & (P.c.page - 1))) * D + r * VB;
        load_codes<VB>(p + (2 * c) * D, vw[0]);
        load_codes<VB>(p + (2 * c + 1) * D, vw[1]);
        load_codes<VB>(p + (2 * c + 8) * D, vw[2]);
        load_codes<VB>(p + (2 * c + 9) * D, vw[3]);
    };
    auto first_codes = [&](int kc, int listed) {
#pragma unroll
        for (int i = 0; i < DEPTH; ++i) {
            const int j = kc + (warp + i * NWARPS) * 16;
            if (j < listed) {
                load_k(j, kr[i]);
                load_v(j, vr[i]);
            }
        }
    };
    first_codes(k0, listed);
#pragma unroll
    for (int i = 0; i < QB; ++i) {
        const int b = warp + i * NWARPS;
        if (b >= NB) break;
        float amax = 0.f;
#pragma unroll
        for (int x = 0; x < KB; ++x) amax = fmaxf(amax, fabsf(q[i][x]));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const int eq = max((__float_as_int(amax) >> 23) - 127, -100) - 13;  // amax 2^-eq in [2^13, 2^14)
        const float inv = pow2(-eq);
        if (c == 0) sqs[8 * b + r] = pow2(eq) * P.scale_log2;
#pragma unroll
        for (int t = 0; t < KS; ++t)
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const float a = q[i][4 * t + 2 * w] * inv, z = q[i][4 * t + 2 * w + 1] * inv;
                const uint32_t hi = pack_half2(a, z);
                sq[((b * KS + t) * 2 + w) * 32 + lane] = hi;
                if constexpr (PARTS == 2) {
                    const float2 f = float2_of(hi);
                    sq[NB * KS * 64 + ((b * KS + t) * 2 + w) * 32 + lane] = pack_half2(a - f.x, z - f.y);
                }
            }
    }
    __syncthreads();
    float qs[NB][2];  // log2(e) * scale * 2^eq of query rows 2c, 2c+1
    int qpos[NB][2];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int row = 8 * b + 2 * c + j;
            qs[b][j] = sqs[row];
            qpos[b][j] = row < nrows ? B.pos + (row0 + row) / P.g : INT32_MIN;
        }
    // keys up to whole_to need no look at their scores, unless a row's factor could pass fp32
    bool wide = false;
#pragma unroll
    for (int b = 0; b < NB; ++b) wide |= fmaxf(qs[b][0], qs[b][1]) > WIDE_QUERY;
    const int whole_to = __any_sync(0xffffffffu, wide) ? INT32_MIN : B.pos_lo;
    uint32_t qf[NB * PARTS == 1 ? KS : 1][2];  // in registers where one fragment set serves
    if constexpr (NB * PARTS == 1) {
#pragma unroll
        for (int t = 0; t < KS; ++t)
#pragma unroll
            for (int w = 0; w < 2; ++w) qf[t][w] = sq[(t * 2 + w) * 32 + lane];
    }
    __syncthreads();  // sqs is free

    float o[NB][KS][4];
    float m[NB][2], mv[NB][2], sum[NB][2];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
#pragma unroll
        for (int i = 0; i < KS; ++i) o[b][i][0] = o[b][i][1] = o[b][i][2] = o[b][i][3] = 0.f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            m[b][j] = mv[b][j] = NO_REF;
            sum[b][j] = 0.f;
        }
    }

    // the codes of 16 keys a step further ahead on their way to L2, by one lane for K and one for
    // V: more in flight than the registers hold.  32 sequences of 32768 keys (graph): 348 us without, 334 with
    // one step, 347 and 498 with four and eight; head_dim 64, two steps in registers, gains nothing
    auto ahead = [&](int j, int listed) {
        if (j < listed && lane < 2) {
            const int pi = (j >> P.c.page_log2) - page0;
            if (s_page[pi] >= 0) {
                const int64_t blk = slab + static_cast<int64_t>(s_page[pi]) * P.c.H;
                prefetch_l2(P.c.code[lane] + ((blk << P.c.page_log2) + (j & (P.c.page - 1))) * D, 16 * D);
            }
        }
    };
    // 16 keys from j on, whose codes are in kw and vw; those of jn are asked for instead
    auto step = [&](int j, int jn, int listed, uint32_t (&kw)[2][KW], uint32_t (&vw)[4][VW]) {
        const int pi = (j >> P.c.page_log2) - page0;
        const bool bad = s_page[pi] < 0;
        const float ks = s_ks[pi], ev = s_ev[pi];
        // S^T = K Q^T
        float sc[NB][4];
#pragma unroll
        for (int b = 0; b < NB; ++b) sc[b][0] = sc[b][1] = sc[b][2] = sc[b][3] = 0.f;
#pragma unroll
        for (int t = 0; t < KS; ++t) {
            const uint32_t a0 = half2_of_lo(kw[0][t]), a2 = half2_of_hi(kw[0][t]);
            const uint32_t a1 = half2_of_lo(kw[1][t]), a3 = half2_of_hi(kw[1][t]);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                if constexpr (NB * PARTS == 1) {
                    mma16816(sc[b], a0, a1, a2, a3, qf[t][0], qf[t][1]);
                } else {
#pragma unroll
                    for (int p = 0; p < PARTS; ++p) {
                        const uint32_t* f = sq + ((p * NB + b) * KS + t) * 64 + lane;
                        mma16816(sc[b], a0, a1, a2, a3, f[0], f[32]);
                    }
                }
            }
        }
        if (jn < listed) load_k(jn, kw);
        if (D == 128) ahead(jn + TILE_KEYS, listed);
        // scores in base 2, masked; keys r, r + 8 and query rows 2c, 2c + 1 of each row block
        const bool whole = !bad && j + 16 <= k1 && j + 15 <= whole_to;
        bool raise = false;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                float f = ks * qs[b][u & 1];
                if (!whole) f = fminf(f, FLT_MAX);  // a score of 0 stays 0
                float x = sc[b][u] * f;
                if (!whole) {
                    const int key = j + r + 8 * (u >> 1);
                    if (bad || key >= k1 || key > qpos[b][u & 1]) x = -INFINITY;
                }
                sc[b][u] = x;
                raise |= x > m[b][u & 1] + MARGIN || x + ev > mv[b][u & 1] + MARGIN;
            }
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    float top = fmaxf(sc[b][q], sc[b][q + 2]);
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                    const float mn = fmaxf(m[b][q], top), mvn = fmaxf(mv[b][q], top + ev);
                    sum[b][q] *= ex2(m[b][q] - mn);
                    const float f = ex2(mv[b][q] - mvn);
                    m[b][q] = mn;
                    mv[b][q] = mvn;
#pragma unroll
                    for (int i = 0; i < KS; ++i) {
                        o[b][i][q] *= f;
                        o[b][i][q + 2] *= f;
                    }
                }
        }
        uint32_t pt[NB][PARTS][2];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                float w[2];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const float x = sc[b][2 * hf + q];
                    sum[b][q] += ex2(x - (m[b][q] - BIAS));
                    w[q] = ex2(x + ev - (mv[b][q] - BIAS));
                }
                const uint32_t hi = pack_half2(w[0], w[1]);
                pt[b][0][hf] = transpose8x8(hi);
                if constexpr (PARTS == 2) {
                    const float2 f = float2_of(hi);
                    pt[b][PARTS - 1][hf] = transpose8x8(pack_half2(w[0] - f.x, w[1] - f.y));
                }
            }
        if (j + 16 > k1) {  // slots past the last visible key may hold anything
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (j + 2 * c + (u & 1) + 8 * (u >> 1) >= k1) {
#pragma unroll
                    for (int x = 0; x < VW; ++x) vw[u][x] = 0;
                }
        }
        // O^T += V^T P^T; M tile i: dims r * d/8 + 2i and + 2i + 1
#pragma unroll
        for (int x = 0; x < VW; ++x) {
            const uint32_t e0 = __byte_perm(vw[0][x], vw[1][x], 0x5140), e1 = __byte_perm(vw[0][x], vw[1][x], 0x7362);
            const uint32_t f0 = __byte_perm(vw[2][x], vw[3][x], 0x5140), f1 = __byte_perm(vw[2][x], vw[3][x], 0x7362);
#pragma unroll
            for (int y = 0; y < (VB >= 4 ? 2 : 1); ++y) {
                const uint32_t e = y ? e1 : e0, f = y ? f1 : f0;
                const uint32_t a0 = half2_of_lo(e), a1 = half2_of_hi(e), a2 = half2_of_lo(f), a3 = half2_of_hi(f);
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int p = 0; p < PARTS; ++p) mma16816(o[b][2 * x + y], a0, a1, a2, a3, pt[b][p][0], pt[b][p][1]);
            }
        }
        if (jn < listed) load_v(jn, vw);
    };
    for (int kc = k0;;) {  // keys [kc, listed) are listed, and the first codes asked for
        int j = kc + 16 * warp;
        for (; j < listed; j += DEPTH * TILE_KEYS)
#pragma unroll
            for (int i = 0; i < DEPTH; ++i)
                if (j + i * TILE_KEYS < listed) step(j + i * TILE_KEYS, j + (i + DEPTH) * TILE_KEYS, listed, kr[i], vr[i]);
        if (listed >= k1) break;
        __syncthreads();  // every warp is done with the list
        kc = listed;
        listed = list_pages(kc);
        __syncthreads();
        first_codes(kc, listed);
    }

    // join the warps: outputs in units of 2^mv, sums in units of 2^m (both with the bias)
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            float t = sum[b][q];
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) t += __shfl_xor_sync(0xffffffffu, t, x);
            const int row = 8 * b + 2 * c + q;
            if (r == 0) stat[warp * ROWS + row] = make_float4(m[b][q], mv[b][q], t, 0.f);
            float* dst = so + (warp * ROWS + row) * D + r * VB;
#pragma unroll
            for (int i = 0; i < KS; ++i) *reinterpret_cast<float2*>(dst + 2 * i) = make_float2(o[b][i][q], o[b][i][q + 2]);
        }
    __syncthreads();

    T* out = static_cast<T*>(P.out);
    auto row_of = [&](int row) { return B.row_of(P, hq0, row); };
    // the CTAs that share this unit, and this one's slot
    const int u0 = at - first, c0 = u0 / share;
    const int pieces = (u0 + tiles - 1) / share - c0 + 1;
    const int64_t part0 = (2 * static_cast<int64_t>(blockIdx.x) + (first == 0)) * ROWS;
    for (int i = threadIdx.x; i < nrows * (D / 4); i += NT) {
        const int row = i / (D / 4), d4 = i % (D / 4);
        if (!KVB_IN_BOUNDS(P.err, row_of(row), 1, rows_of(P))) continue;
        Joined z;
#pragma unroll 4
        for (int w = 0; w < NWARPS; ++w) z.reference(stat[w * ROWS + row]);
#pragma unroll 4
        for (int w = 0; w < NWARPS; ++w)
            z.add(stat[w * ROWS + row], reinterpret_cast<const float4*>(so + (w * ROWS + row) * D)[d4]);
        if (pieces == 1) {
            store_out(out + row_of(row) * D + 4 * d4, z.output());
            if (d4 == 0 && P.lse) P.lse[row_of(row)] = z.lse();
        } else if (KVB_IN_BOUNDS(P.err, part0 + row, 1, P.slots * ROWS)) {
            reinterpret_cast<float4*>(P.partial + (part0 + row) * D)[d4] = z.acc;
            if (d4 == 0) P.part_stat[part0 + row] = make_float4(z.m, z.mv, z.sum, 0.f);
        }
    }
    if (pieces > 1)
        join_splits<T, D, ROWS, NT>(P, B, Pieces{pieces, c0}, unit, hq0, &s_last, so, NWARPS * ROWS * D);

    at += last - first;
    if (at >= stop) return;
    first = 0;
    if (++h == P.c.H) {
        h = 0;
        do {
            if (++e == entries) {
                e = 0;
                if (++l == P.c.n_layers) return;  // likewise not reached
            }
            B = entry(e);
            tiles = unit_tiles<TILE_KEYS>(B);
        } while (tiles == 0);
    }
    __syncthreads();  // shared memory is free for the next unit
    }
}

// A lane takes 32 bytes of a key row at head_dim 128.  Rows and pages are multiples of 128
// bytes, so all of them lie as the buffer does, which is 16-byte aligned: where it is not
// 32-byte aligned, instances of their own read halves.  32 sequences of 32768 keys: 335 us, in
// halves 353; both in one kernel under a predicate cost every call 1.3 %.
bool whole_rows(const Cache& c) { return (reinterpret_cast<uintptr_t>(c.code[0]) & 31u) == 0; }

// One instance: CTAs of it that fit an SM (P null), or its launch.
template <typename T, int D, int NB, int NWARPS, bool WHOLE>
cudaError_t instance(const AttnParams* P, int ctas, cudaStream_t s, int* fit) {
    constexpr size_t smem = Shape8<T, D, NB, NWARPS>::smem();
    const auto kernel = decode_kernel<T, D, NB, NWARPS, WHOLE>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    if (!P) {
        static const int resident = [&] {
            int n = 0;
            return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, NWARPS * 32, smem) == cudaSuccess ? n : 0;
        }();
        *fit = resident;
        return cudaSuccess;
    }
    kernel<<<ctas, NWARPS * 32, smem, s>>>(*P);
    return cudaGetLastError();
}

template <typename T, int D, bool WHOLE = true>
cudaError_t instance_rows(int rows, bool few, const AttnParams* P, int ctas, cudaStream_t s, int* fit) {
    switch (rows) {
        case 8:
            if constexpr (D >= 64)
                if (few) return instance<T, D, 1, WARPS_FEW, WHOLE>(P, ctas, s, fit);
            return instance<T, D, 1, WARPS, WHOLE>(P, ctas, s, fit);
        default: return instance<T, D, 2, WARPS, WHOLE>(P, ctas, s, fit);
    }
}

template <typename T>
cudaError_t instance_dim(const Cache& c, int rows, bool few, const AttnParams* P, int ctas, cudaStream_t s, int* fit) {
    switch (c.d) {
        case 16: return instance_rows<T, 16>(rows, few, P, ctas, s, fit);
        case 32: return instance_rows<T, 32>(rows, few, P, ctas, s, fit);
        case 64: return instance_rows<T, 64>(rows, few, P, ctas, s, fit);
        default:
            return whole_rows(c) ? instance_rows<T, 128>(rows, few, P, ctas, s, fit)
                                 : instance_rows<T, 128, false>(rows, few, P, ctas, s, fit);
    }
}

cudaError_t pick(kvb_dtype dtype, const Cache& c, int rows, bool few, const AttnParams* P, int ctas, cudaStream_t s, int* fit) {
    return dtype == KVB_BF16 ? instance_dim<__nv_bfloat16>(c, rows, few, P, ctas, s, fit)
                             : instance_dim<float>(c, rows, few, P, ctas, s, fit);
}

}  // namespace

AttnPlan plan_attention(const Cache& c, const Seqs& q, kvb_dtype dtype, int g, int num_sms) {
    AttnPlan p{};
    const int64_t most = static_cast<int64_t>(q.max_tokens) * g;  // rows of one sequence and head
    const double max_kv = q.max_kv > 0 ? q.max_kv : 1;
    // bf16 rows go to the tensor-core kernel where more than two blocks of 16 would read the keys
    // again, three at head_dim 64.  8 heads, rows 24 / 32 / 40 / 64 / 128, us:
    //   d 128  8 x 4096 keys    here  48 /  49 /  61 /  75 / 128   there  50 /  50 /  52 /  52 /  49
    //          16 x 16384            237 / 239 / 342 / 450 / 882         248 / 249 / 249 / 250 / 202
    //          1 x 4096               22 /  22 /  24 /  33 /  34          25 /  27 /  27 /  28 /  28
    //   d 64   8 x 4096               32 /  32 /  41 /  48 /  81          43 /  44 /  45 /  45 /  41
    //          16 x 16384            176 / 176 / 254 / 336 / 658         214 / 214 / 215 / 214 / 175
    //          1 x 4096               16 /  16 /  17 /  23 /  24          23 /  25 /  26 /  25 /  25
    // Else blocks of 8 or 16 rows; of 32 (fewer warps, spilled registers) they took 55 / 61 us at
    // 24 / 32 rows, d 128, 8 x 4096, and gained 8 % only for fp32 rows in the hundreds; four warps
    // with 16 rows each over the same keys took 82 us at 40 rows.
    p.tensor = dtype == KVB_BF16 && c.d >= 64 && most > (c.d == 128 ? 32 : 48);
    p.rows = p.tensor ? PREFILL_ROWS : most <= 8 ? 8 : 16;
    p.row_blocks = static_cast<int>((most + p.rows - 1) / p.rows);
    p.units = static_cast<int64_t>(c.n_layers) * q.n_seq * c.H * p.row_blocks;
    auto tiles = [&](int keys) { return static_cast<double>(p.units) * ((static_cast<int64_t>(max_kv) + keys - 1) / keys); };
    // up to eight rows over few keys (less than FEW_TILES of 64 for each of four CTAs an SM):
    // 8 warps a CTA take 128 keys in one step and the unit has few pieces to join (one token
    // over 4096 keys: 11.5 us; with 4 warps and 4 tiles each 14.9, with 16 warps 13.0)
    p.few = !p.tensor && p.rows == 8 && c.d >= 64 && tiles(16 * WARPS) < static_cast<double>(FEW_TILES) * 4 * num_sms;
    int fit = 1;
    if (!p.tensor) pick(dtype, c, p.rows, p.few, nullptr, 0, nullptr, &fit);
    // the CTAs that fit the GPU, no more than the keys give the least share to
    p.min_tiles = p.few ? 1 : MIN_TILES;
    const double need = (tiles(p.tensor ? 128 : 16 * (p.few ? WARPS_FEW : WARPS)) + p.min_tiles - 1) / p.min_tiles;
    p.ctas = num_sms * (fit > 0 ? fit : 1);
    if (need < p.ctas) p.ctas = static_cast<int>(need) < 1 ? 1 : static_cast<int>(need);
    p.tiles = tiles(p.tensor ? 128 : 64);
    p.slots = 2 * static_cast<int64_t>(p.ctas);
    p.counter_bytes = p.tensor ? 0 : (static_cast<size_t>(p.units) * sizeof(int) + 255) / 256 * 256;
    p.unit_bytes = p.tensor ? static_cast<size_t>(p.units) * sizeof(int2) : 0;
    p.partial_bytes = static_cast<size_t>(p.slots) * p.rows * (c.d + 4) * sizeof(float);
    return p;
}

cudaError_t launch_decode(const AttnParams& P, kvb_dtype dtype, const AttnPlan& p, cudaStream_t s) {
    return pick(dtype, P.c, p.rows, p.few, &P, p.ctas, s, nullptr);
}

}  // namespace c8
}  // namespace kvb
