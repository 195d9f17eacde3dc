// Attention over the paged 8-bit cache on the 5th-generation tensor cores: many
// query rows (prompts over a cached prefix, several drafted tokens), bf16, head_dim 64 and 128.
//
// The mathematics and the references are those of cache8_attn.cu; here the
// products are large enough to be bound by the SM itself.  One CTA an SM takes 256
// rows of a unit (layer, sequence, row block, head) as two tiles of 128 and walks
// its keys 128 at a time; the 128-key tiles of all units form one line that the CTAs
// share evenly.
//   warps 0..3, 4..7  softmax of tile 0, 1, a row a thread, 64 keys a step: scores
//                 from TMEM to registers, P as fp16 over them, the sum in fp32; O is
//                 rescaled in TMEM on the rare raise;
//   warps 8..15   read the codes, four warps of K and four of V (prefetched into
//                 registers a tile ahead), convert them to fp16 (exact) and lay them
//                 out as operands, keys and values alike: 128-byte swizzle, key rows,
//                 K-major for S and MN-major for O;
//                 also the scales of the tile's 16-key groups and the CTA's next piece;
//   warps 16, 17  one lane of each issues S_x = Q_x K^T for tile x;
//   warps 18, 19  and O_x += P_x V (P from TMEM): four warps, so that no product
//                 waits behind a wait of another kind.
// TMEM: score buffer b of tile x at 128 x + 64 b, O_x at 256 + 128 x.  P takes its
// scores' columns, so a buffer's next scores are issued when O_x += P V has
// completed; meanwhile the softmax works on the other buffer (one buffer of 128
// keys left it waiting 2500 of 5800 cycles for each 128 keys).
// What 128 keys of 256 rows cost an SM, cycles: products 2048; shared memory 3072
// (192 KB of S operands, 64 of V, 64 + 64 of the conversion, at 128 bytes a cycle);
// exponentials about 1000, maxima, masks and conversions on the ALU about 2000.
// The weights carry the value scale, w = 2^(s + e_v - mv); a 16-key group's sum goes
// into the denominator with the factor 2^(mv - m - e_v), or is taken from
// exponentials of its own where that factor could leave fp32's range.
// 1024 tokens over 16K, 64 query and 8 KV heads: 503 us a call, 497 replayed from a graph (the
// steps' figures here are graph replays), 1.13 PF/s, about 4200 cycles for each 128 keys of 256 rows.  No unit is full; the two tiles' chains S -> softmax -> P V
// hide most of each other's waits, not all.
// Every wait is bounded; after one gives up, its role runs through the rest without
// touching TMEM, meeting the others at every barrier.
#include <cfloat>

#include "cache8_attn.cuh"

namespace kvb {
namespace c8 {

namespace {

constexpr int TR = 128;              // rows of a tile, TMEM lanes
constexpr int ROWS = PREFILL_ROWS;   // 256: two tiles
constexpr int TK = 128;              // keys of an operand tile
constexpr int SK = 64;               // keys of a step (two score buffers a tile in TMEM)
constexpr int ATOM = 128 * 128;  // bytes of 128 rows x 64 fp16
constexpr int tile_bytes(int HD) { return HD / 64 * ATOM; }  // 128 rows
constexpr int STAGES = 2;  // operand tiles of K, and of V
constexpr int SOFT = 256, CONV = 256;
constexpr int NUM_THREADS = SOFT + CONV + 128;
// Registers a thread: 96 at launch, then by role.  256 * 144 + 256 * 72 + 128 * 40 = 60416 of
// the launch's 640 * 96 = 61440.
constexpr int REGS_SOFTMAX = 144, REGS_CONVERT = 72, REGS_MMA = 40;
constexpr int INFO_RING = 8;  // scales are written at most seven tiles before the softmax is done with them
constexpr int smem_bytes(int HD) { return (2 + 2 * STAGES) * tile_bytes(HD) + 1024 + 2048; }
constexpr uint32_t TM_S = 0, TM_O = 256;  // TMEM columns, 128 more for tile 1
constexpr float FACTOR_LOG2 = 60.f;  // a group's factor is used within 2^-60 .. 2^60
constexpr uint64_t DRAIN_NS = 200ull * 1000 * 1000;

__device__ __forceinline__ uint32_t sw_off(int r, int c) {  // 16-byte chunk c (0..15) of row r
    return static_cast<uint32_t>((c >> 3) * ATOM + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}
// Operand descriptors of a tile (step 0) and the distance to step kk, in the
// descriptor's 16-byte units: the issuing thread adds a constant for each product.
__device__ __forceinline__ uint64_t desc_k(const uint8_t* tile) { return sdesc_k_sw128(smem_u32(tile)); }
__device__ __forceinline__ uint64_t desc_v(const uint8_t* tile) { return sdesc_mn_sw128(smem_u32(tile), ATOM); }
constexpr uint32_t step_k(int kk) { return ((kk >> 2) * ATOM + (kk & 3) * 32) >> 4; }
constexpr uint32_t step_v(int kk) { return (kk * 16 * 128) >> 4; }
constexpr uint32_t idesc_f16_f32(uint32_t M, uint32_t N) {
    return (1u << 4) | ((N >> 3) << 17) | ((M >> 4) << 24);
}
// The issuing warps run converged and elect the lane at the products only: under `lane == 0` eight
// of them and their commit took 840 to 1160 cycles to issue, so 400 to 600 (1024 tokens over 16K: 526
// -> 503 us).  Row maxima are taken of three numbers an instruction (by fmaxf: 503 us, not 495).

// 16 bytes, or zeros where !pred: a predicated load, so that a thread's loads are
// all in flight together (behind branches they went one by one: 940 us, not 590, at
// 1024 tokens over 16K with the conversion left out).
__device__ __forceinline__ uint4 load16_if(const void* p, bool pred) {
    uint4 v;
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %5, 0;\n\t"
        "mov.u32 %0, 0;\n\tmov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\tmov.u32 %3, 0;\n\t"
        "@q ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
        : "l"(p), "r"(static_cast<uint32_t>(pred)));
    return v;
}

__device__ __forceinline__ float load4_if(const float* p, bool pred) {
    float v;
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %2, 0;\n\tmov.f32 %0, 0f00000000;\n\t@q ld.global.f32 %0, [%1];\n\t}"
        : "=&f"(v)
        : "l"(p), "r"(static_cast<uint32_t>(pred)));
    return v;
}

struct TileInfo {
    float ks[8], ev[8];  // key scale (0: the page is bad, nothing of it is seen) and value exponent, 16 keys each
};

// A piece of a unit, as the roles read it.
struct Segment {
    RowBlock B;
    int s, l, h;
    int k0, k1;   // keys [k0, k1)
    int whole;    // the unit's only piece
    int64_t unit, slot;
    Pieces pieces;
};

// The CTA's place in the line of tiles.
struct Walk {
    int at, stop, share;
    int e, h, l, first;
};

struct Smem {
    uint64_t k_full[STAGES], k_empty[STAGES], v_full[STAGES], v_empty[STAGES];
    uint64_t s_full[2][2], p_full[2][2], pv_done[2][2];  // [tile][buffer]
    uint64_t q_full[2], drain[4], info_full[INFO_RING];
    uint32_t tmem;
    int abort;
    int more[2];        // a segment follows (by parity of its number)
    Segment seg[2];
    int scan[NUM_THREADS / 32];
    LineStart start;
    Walk walk;
    alignas(16) TileInfo info[INFO_RING];
};

template <int HD>
__global__ void __launch_bounds__(NUM_THREADS, 1) prefill_kernel(const __grid_constant__ AttnParams P) {
    constexpr int TILE = tile_bytes(HD);
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* sQ = smem;
    uint8_t* sK = smem + 2 * TILE;
    uint8_t* sV = sK + STAGES * TILE;
    Smem& M = *reinterpret_cast<Smem*>(sV + STAGES * TILE);
    static_assert(sizeof(Smem) <= 2048, "layout");
    volatile int* abort_flag = &M.abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const DevErr derr{P.err.word, P.err.timeout_ns};

    {
        Walk w;
        if (!line_start<ROWS, TK, NUM_THREADS>(P, M.scan, &M.start, w.at, w.stop, w.share, w.l, w.e, w.h, w.first)) return;
        if (threadIdx.x == SOFT) M.walk = w;
    }

    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&M.k_full[i], CONV / 2);
            mbar_init(&M.k_empty[i], 2);
            mbar_init(&M.v_full[i], CONV / 2);
            mbar_init(&M.v_empty[i], 2);
        }
        for (int x = 0; x < 2; ++x) {
            for (int i = 0; i < 2; ++i) {
                mbar_init(&M.s_full[x][i], 1);
                mbar_init(&M.p_full[x][i], TR);
                mbar_init(&M.pv_done[x][i], 1);
                mbar_init(&M.drain[2 * x + i], 1);
            }
            mbar_init(&M.q_full[x], TR);
        }
        for (int i = 0; i < INFO_RING; ++i) mbar_init(&M.info_full[i], 8);
        M.abort = 0;
        fence_mbar_init();
    }
    // the segment at W, into slot i; W moves past it
    auto walk = [&](int i) {
        Walk W = M.walk;
        const int entries = P.q.n_seq * P.row_blocks;
        Segment& g = M.seg[i];
        RowBlock B = row_block(P, W.e / P.row_blocks, W.e % P.row_blocks, ROWS);
        int tiles = unit_tiles<TK>(B);
        if (W.at >= W.stop || W.l >= P.c.n_layers || tiles == 0) {
            M.more[i] = 0;
            return;
        }
        const int last = min(tiles, W.first + (W.stop - W.at));
        const int u0 = W.at - W.first, c0 = u0 / W.share;
        g.B = B;
        g.s = W.e / P.row_blocks;
        g.l = W.l;
        g.h = W.h;
        g.k0 = W.first * TK;
        g.k1 = min(B.kv_end, last * TK);
        g.unit = (static_cast<int64_t>(W.l) * entries + W.e) * P.c.H + W.h;
        g.pieces = Pieces{(u0 + tiles - 1) / W.share - c0 + 1, c0};
        g.whole = g.pieces.n == 1;
        if (KVB_IN_BOUNDS(P.err, g.unit, 1, P.units)) P.shared_by[g.unit] = make_int2(g.pieces.n, g.pieces.c0);  // every CTA of the unit the same
        g.slot = 2 * static_cast<int64_t>(blockIdx.x) + (W.first == 0);
        M.more[i] = 1;
        W.at += last - W.first;
        W.first = 0;
        if (++W.h == P.c.H) {
            W.h = 0;
            do {
                if (++W.e == entries) {
                    W.e = 0;
                    ++W.l;
                }
                if (W.at >= W.stop || W.l >= P.c.n_layers) break;
                tiles = unit_tiles<TK>(row_block(P, W.e / P.row_blocks, W.e % P.row_blocks, ROWS));
            } while (tiles == 0);
        }
        M.walk = W;
    };
    if (threadIdx.x == SOFT) walk(0);
    if (warp == 16) {
        tmem_alloc(&M.tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = M.tmem;
    auto wait_all = [&](uint64_t* b, uint32_t parity) {  // warp-uniform outcome
        return __all_sync(0xffffffffu, mbar_wait(b, parity, derr, abort_flag)) != 0;
    };
    // Every role goes through the CTA's segments; `base` counts the operand tiles before the
    // segment, so that stages and phases run on over the segments.  A segment of at most 128 rows leaves the second tile idle.
    uint32_t base = 0;

    if (warp < SOFT / 32) {
        // ------------------------------------------------------- softmax
        regs_up<REGS_SOFTMAX>();
        const int x = warp >> 2;                 // tile
        const int row = 32 * (warp & 3) + lane;  // row of the tile, and TMEM lane
        const uint32_t tl = tmem_base + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
        const uint32_t tS = tl + TM_S + 128u * x, tO = tl + TM_O + 128u * x;
        bool ok = true;
        uint32_t even = 0, odd = 0;  // uses of the tile's score buffers before this segment
        for (int n = 0; M.more[n & 1]; ++n) {
            const Segment& G = M.seg[n & 1];
            const int k0 = G.k0, k1 = G.k1;
            const int nsteps = TR * x < G.B.nrows ? (k1 - k0 + SK - 1) / SK : 0;
            const int brow = TR * x + row;
            const bool valid = brow < G.B.nrows && KVB_IN_BOUNDS(P.err, G.B.row_of(P, (static_cast<int64_t>(G.l) * P.c.H + G.h) * P.g, brow), 1, rows_of(P));
            // worked out where it is used: kept, it would cost the score loop's registers
            auto row_index = [&] { return valid ? G.B.row_of(P, (static_cast<int64_t>(G.l) * P.c.H + G.h) * P.g, brow) : 0; };  // in [n_layers][Hq][T]
            float m = NO_REF, mv = NO_REF, sum = 0.f;
            // the row as fp16 under a power of two: largest element in [2^13, 2^14)
            float qs;
            {
                const uint4* q = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(P.query) + row_index() * HD);
                uint4 u[HD / 8];
#pragma unroll
                for (int c = 0; c < HD / 8; ++c) u[c] = valid ? __ldg(q + c) : make_uint4(0, 0, 0, 0);
                float amax = 0.f;
#pragma unroll
                for (int c = 0; c < HD / 8; ++c) {
                    const uint32_t w[4] = {u[c].x, u[c].y, u[c].z, u[c].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xffff0000u))));
                }
                const int eq = max((__float_as_int(amax) >> 23) - 127, -100) - 13;
                const float inv = pow2(-eq);
                qs = fminf(pow2(eq) * P.scale_log2, FLT_MAX);
#pragma unroll
                for (int c = 0; c < HD / 8; ++c) {
                    const uint32_t w[4] = {u[c].x, u[c].y, u[c].z, u[c].w};
                    uint32_t o[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        o[i] = pack_half2(__uint_as_float(w[i] << 16) * inv, __uint_as_float(w[i] & 0xffff0000u) * inv);
                    *reinterpret_cast<uint4*>(sQ + x * TILE + sw_off(row, c)) = make_uint4(o[0], o[1], o[2], o[3]);
                }
                fence_proxy_async_smem();
                mbar_arrive(&M.q_full[x]);
            }
            // keys below `see` are visible to this row
            const int see = valid ? min(k1, G.B.pos + (G.B.row0 + brow) / P.g + 1) : 0;
            // a step's visible keys that need no look at their scores: none where a factor could pass fp32
            const int full = qs > WIDE_QUERY ? INT32_MAX : SK;
            for (int u = 0; u < nsteps; ++u) {
                const uint32_t gt = base + (u >> 1), ring = gt & (INFO_RING - 1);
                const int hf = u & 1;
                if (hf == 0) ok = ok && wait_all(&M.info_full[ring], (gt / INFO_RING) & 1);
                const uint32_t use = (hf ? odd : even) + (u >> 1);
                ok = ok && wait_all(&M.s_full[x][hf], use & 1);
                if (!ok) break;
                tc_fence_after();
                const uint32_t cS = tS + SK * hf;
                uint32_t sv[SK];
                tmem_ld32(cS, sv);
                tmem_ld32(cS + 32, sv + 32);
                const TileInfo& I = M.info[ring];
                const float4 ks4 = *reinterpret_cast<const float4*>(I.ks + 4 * hf);
                const float4 ev4 = *reinterpret_cast<const float4*>(I.ev + 4 * hf);
                const float ev[4] = {ev4.x, ev4.y, ev4.z, ev4.w};
                float k[4] = {ks4.x * qs, ks4.y * qs, ks4.z * qs, ks4.w * qs};
                // visible keys of this row are a prefix of the step's
                const int nvis = min(see - (k0 + u * SK), SK);
                const bool whole = nvis == full && ks4.x != 0.f && ks4.y != 0.f && ks4.z != 0.f && ks4.w != 0.f;
                tmem_ld_wait();
                if (!__all_sync(0xffffffffu, whole)) {
                    const float seen[4] = {ks4.x, ks4.y, ks4.z, ks4.w};
#pragma unroll
                    for (int gq = 0; gq < 4; ++gq) k[gq] = fminf(fmaxf(k[gq], FLT_MIN), FLT_MAX);  // of 0 and -inf: no NaN
#pragma unroll
                    for (int j = 0; j < SK; ++j)
                        if (j >= nvis || seen[j >> 4] == 0.f) sv[j] = 0xff800000u;  // -inf
                }
                // maxima of s and of s + e_v (factors are positive)
                float ms = -INFINITY, mvs = -INFINITY;
#pragma unroll
                for (int gq = 0; gq < 4; ++gq) {
                    float top[5];
#pragma unroll
                    for (int j = 0; j < 5; ++j)
                        top[j] = max3(__uint_as_float(sv[16 * gq + 3 * j]), __uint_as_float(sv[16 * gq + 3 * j + 1]),
                                      __uint_as_float(sv[16 * gq + 3 * j + 2]));
                    const float best = fmaxf(max3(top[0], top[1], top[2]), max3(top[3], top[4], __uint_as_float(sv[16 * gq + 15]))) * k[gq];
                    ms = fmaxf(ms, best);
                    mvs = fmaxf(mvs, best + ev[gq]);
                }
                const bool raise = ms > m + MARGIN || mvs > mv + MARGIN;
                if (__any_sync(0xffffffffu, raise)) {
                    float f = 1.f;
                    if (raise) {
                        const float mn = fmaxf(m, ms), mvn = fmaxf(mv, mvs);
                        sum *= ex2(m - mn);
                        f = ex2(mv - mvn);
                        m = mn;
                        mv = mvn;
                    }
                    __syncwarp();
                    if (u > 0) {
                        // O is complete up to the step before
                        ok = wait_all(&M.pv_done[x][hf ^ 1], (hf ? even + (u >> 1) : odd + (u >> 1) - 1) & 1);
                        if (ok) {
                            tc_fence_after();
#pragma unroll 1
                            for (int c0 = 0; c0 < HD; c0 += 16) {
                                uint32_t o[16];
                                tmem_ld16(tO + c0, o);
                                tmem_ld_wait();
#pragma unroll
                                for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                                tmem_st16(tO + c0, o);
                            }
                            tmem_st_wait();
                        }
                    }
                }
                // the weights; P takes the columns of the scores.  No branch lies between them: one
                // a 16-key group cost 72 us of 556.
                float far = 0.f;  // the largest |log2 factor| of a group
#pragma unroll
                for (int g2 = 0; g2 < 2; ++g2) {
                    uint32_t pw[16];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int gq = 2 * g2 + c;
                        const float b = ev[gq] - mv + BIAS, e = mv - m - ev[gq];
                        float2 w[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float2 a = make_float2(__uint_as_float(sv[16 * gq + 2 * j]), __uint_as_float(sv[16 * gq + 2 * j + 1]));
                            w[j] = fma2(a, make_float2(k[gq], k[gq]), make_float2(b, b));
                            w[j] = make_float2(ex2(w[j].x), ex2(w[j].y));
                            pw[8 * c + j] = pack_half2(w[j].x, w[j].y);
                        }
                        const float2 p = add2(add2(add2(w[0], w[1]), add2(w[2], w[3])), add2(add2(w[4], w[5]), add2(w[6], w[7])));
                        far = fmaxf(far, fabsf(e));
                        sum += fabsf(e) < FACTOR_LOG2 ? (p.x + p.y) * ex2(e) : 0.f;
                    }
                    tmem_st16(cS + 16 * g2, pw);
                }
                if (far >= FACTOR_LOG2) {  // the sums of such groups from exponentials of their own
#pragma unroll
                    for (int gq = 0; gq < 4; ++gq)
                        if (fabsf(mv - m - ev[gq]) >= FACTOR_LOG2) {
#pragma unroll
                            for (int j = 0; j < 16; ++j) sum += ex2(fmaf(__uint_as_float(sv[16 * gq + j]), k[gq], BIAS - m));
                        }
                }
                __syncwarp();
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&M.p_full[x][hf]);
            }
            if (nsteps > 0) {
                const int hf = (nsteps - 1) & 1;
                ok = ok && wait_all(&M.pv_done[x][hf], ((hf ? odd : even) + ((nsteps - 1) >> 1)) & 1);
            }
            even += (nsteps + 1) / 2;
            odd += nsteps / 2;
            base += (k1 - k0 + TK - 1) / TK;

            // outputs: from TMEM (units of 2^mv, sums of 2^m, both with the bias)
            const bool have = ok && nsteps > 0;
            if (have) tc_fence_after();
            const int64_t part = G.slot * ROWS + brow, out_row = row_index();
            const float half = ex2(0.5f * (mv - m)), f = sum == 0.f ? 0.f : half / sum;
#pragma unroll 1
            for (int c0 = 0; c0 < HD; c0 += 16) {
                uint32_t o[16];
                if (have) {
                    tmem_ld16(tO + c0, o);
                    tmem_ld_wait();
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j) o[j] = 0u;
                }
                if (valid && G.whole) {
                    uint32_t w[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        w[j] = pack_bf16x2(__uint_as_float(o[2 * j]) * f * half, __uint_as_float(o[2 * j + 1]) * f * half);
                    uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(P.out) + out_row * HD + c0);
                    dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
                    dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
                } else if (valid && KVB_IN_BOUNDS(P.err, part, 1, P.slots * ROWS)) {
                    uint4* dst = reinterpret_cast<uint4*>(P.partial + part * HD + c0);
#pragma unroll
                    for (int j = 0; j < 4; ++j) dst[j] = make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                }
                __syncwarp();
            }
            if (valid) {
                if (!G.whole) {
                    if (KVB_IN_BOUNDS(P.err, part, 1, P.slots * ROWS)) P.part_stat[part] = make_float4(m, mv, sum, 0.f);
                } else if (P.lse) P.lse[out_row] = sum == 0.f ? -INFINITY : (m - BIAS + log2f(sum)) * 0.693147180559945f;
            }
            tc_fence_before();
            __syncthreads();  // the segment is done, the next one worked out
        }
    } else if (warp < (SOFT + CONV) / 32) {
        // ------------------------------------------------------- codes -> fp16 operands
        regs_down<REGS_CONVERT>();
        const int tid = threadIdx.x - SOFT;
        const int kv = tid >> 7;                               // half of the threads for K, half for V
        constexpr int COLS = HD / 16, RP = 128 / COLS, N = TK / RP;  // 16-code columns of a row, rows of a pass, passes
        const int rr = (tid & 127) / COLS, c16 = tid % COLS;   // row of the pass, column
        uint8_t* const operand = kv ? sV : sK;
        uint64_t* const full = kv ? M.v_full : M.k_full;
        uint64_t* const empty = kv ? M.v_empty : M.k_empty;
        const int pm = P.c.page - 1;
        const uint32_t page_bytes = static_cast<uint32_t>(P.c.H << P.c.page_log2) * HD;
        bool go = true;
        for (int n = 0; M.more[n & 1]; ++n) {
            const Segment& G = M.seg[n & 1];
            const int k0 = G.k0, k1 = G.k1, ntiles = (k1 - k0 + TK - 1) / TK, last = max(k1 - 1, 0);
            const int* table = P.q.page_table + static_cast<int64_t>(G.s) * P.q.max_pages;
            const int64_t block0 = (static_cast<int64_t>(P.c.l_begin) + G.l) * P.c.n_pages * P.c.H + G.h;  // of page 0
            // this thread's first code in page 0; page_bytes from one page's block to the next's
            const int64_t first = (block0 << P.c.page_log2) * HD + c16 * 16;
            const uint8_t* from = P.c.code[kv] + first;
            uint4 raw[N];  // of the tile that is converted next
            int pid[N];    // pages of the tile after it
            auto page = [&](int t, int i) {
                int p = -1;
                const int at = min(k0 + t * TK + RP * i + (RP > 16 ? rr : 0), last) >> P.c.page_log2;
                if (table_in_bounds(P.q, P.err, G.s, at)) asm volatile("ld.global.u32 %0, [%1];" : "=r"(p) : "l"(table + at));
                return p;
            };
            auto load = [&](int t, int i, int p) {
                const int j = k0 + t * TK + RP * i + rr;
                // slots past the last visible key may hold anything: not read
                const bool have = j < k1 && p >= 0 && p < P.c.n_pages &&
                                  KVB_IN_BOUNDS(P.err, block0 + static_cast<int64_t>(p) * P.c.H, 1, blocks_of(P.c));
                return load16_if(from + static_cast<uint64_t>(static_cast<uint32_t>(p)) * page_bytes + (j & pm) * HD, have);
            };
            auto store = [&](uint8_t* tile, int i, const uint4& u) {
                // codes 16 c16 .. +15 are chunks 2 c16 and 2 c16 + 1; lanes of the upper 64 dims
                // store theirs in the other order, so that eight lanes hit eight bank groups (of a row
                // of 64 dims: the eight lanes are two rows, which the swizzle sets apart)
                const int flip = c16 >> 2;
                const uint4 a = make_uint4(half2_of_lo(u.x), half2_of_hi(u.x), half2_of_lo(u.y), half2_of_hi(u.y));
                const uint4 b = make_uint4(half2_of_lo(u.z), half2_of_hi(u.z), half2_of_lo(u.w), half2_of_hi(u.w));
                *reinterpret_cast<uint4*>(tile + sw_off(RP * i + rr, 2 * c16 + flip)) = flip ? b : a;
                *reinterpret_cast<uint4*>(tile + sw_off(RP * i + rr, 2 * c16 + 1 - flip)) = flip ? a : b;
            };
            // scales of 16-key group `tid` of a tile, for eight threads: its page is asked for two
            // tiles ahead and its scales one, so that neither is waited for
            float ks = 0.f, vs = 0.f;
            int gp = -1;
            bool in_range = false;
            auto group_page = [&](int t) {
                const int j = k0 + t * TK + 16 * tid;
                in_range = j < k1;
                gp = in_range && table_in_bounds(P.q, P.err, G.s, j >> P.c.page_log2) ? __ldg(table + (j >> P.c.page_log2)) : -1;
            };
            auto scales = [&] {
                const int64_t blk = block0 + static_cast<int64_t>(gp) * P.c.H;
                const bool have = gp >= 0 && gp < P.c.n_pages && KVB_IN_BOUNDS(P.err, blk, 1, blocks_of(P.c));
                if (in_range && !have) err_set(P.err, DEV_ERR_BAD_SEQ);
                ks = load4_if(P.c.scale[0] + blk, have);  // not looked at before the next tile
                vs = load4_if(P.c.scale[1] + blk, have);
            };
            if (tid < 8 && ntiles > 0) {
                group_page(0);
                scales();
                group_page(1);
            }
            if (ntiles > 0) {
#pragma unroll
                for (int i = 0; i < N; ++i) pid[i] = page(0, i);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    raw[i] = load(0, i, pid[i]);
                    pid[i] = page(1, i);
                }
            }
            uint32_t stage = base % STAGES, round = base / STAGES;
            for (int t = 0; go && t < ntiles; ++t) {
                if (!(go = mbar_wait(&empty[stage], (round & 1) ^ 1, derr, abort_flag))) break;
                if (tid < 8) {
                    TileInfo& I = M.info[(base + t) & (INFO_RING - 1)];
                    I.ks[tid] = ks;
                    I.ev[tid] = ks != 0.f ? static_cast<float>(exponent_of(vs)) : 0.f;
                    mbar_arrive(&M.info_full[(base + t) & (INFO_RING - 1)]);
                    scales();
                    group_page(t + 2);
                }
#pragma unroll
                for (int i = 0; i < N; ++i) {  // each chunk's registers ask for the next tile's at once
                    store(operand + stage * TILE, i, raw[i]);
                    raw[i] = load(t + 1, i, pid[i]);
                    pid[i] = page(t + 2, i);
                }
                fence_proxy_async_smem();
                mbar_arrive(&full[stage]);
                if (++stage == STAGES) {
                    stage = 0;
                    ++round;
                }
            }
            if (tid == 0) walk((n + 1) & 1);  // while the softmax is a tile or two behind
            base += ntiles;
            __syncthreads();
        }
    } else {
        // ------------------------------------------------------- products
        regs_down<REGS_MMA>();
        const int who = __shfl_sync(0xffffffffu, warp - 16, 0), x = who & 1;  // tile
        const uint32_t cS = tmem_base + TM_S + 128u * x;
        bool go = true;
        uint32_t even = 0, odd = 0;  // uses of the tile's score buffers before this segment
        for (int n = 0; M.more[n & 1]; ++n) {
            const Segment& G = M.seg[n & 1];
            const int ntiles = (G.k1 - G.k0 + TK - 1) / TK;
            const bool idle = TR * x >= G.B.nrows;
            const int nsteps = (G.k1 - G.k0 + SK - 1) / SK;
            if (who < 2) {
                constexpr uint32_t idesc = idesc_f16_f32(TR, SK);
                const uint64_t q = desc_k(sQ + x * TILE), k0 = desc_k(sK);
                // A limit of 0 leaves no time to wait: the wait for the queries is a timeout, whatever it
                // would have found.  These waits are too short for mbar_wait to look at the clock, and
                // what a look at the barrier finds would depend on which warp is first.
                if (go && ntiles > 0 && derr.timeout_ns == 0) {
                    dev_err_set(derr, DEV_ERR_TIMEOUT);
                    *abort_flag = 1;
                    go = false;
                }
                go = go && (ntiles == 0 || wait_all(&M.q_full[x], n & 1));
                for (int t = 0; go && t < ntiles; ++t) {
                    const uint32_t stage = (base + t) % STAGES;
                    if (!(go = wait_all(&M.k_full[stage], ((base + t) / STAGES) & 1))) break;
                    for (int hf = 0; go && !idle && hf < 2 && 2 * t + hf < nsteps; ++hf) {
                        // P of this buffer's use before lies where these scores go
                        const uint32_t use = (hf ? odd : even) + t;
                        if (use > 0 && !(go = wait_all(&M.pv_done[x][hf], (use - 1) & 1))) break;
                        tc_fence_after();
                        const uint64_t k = k0 + (stage * TILE + hf * SK * 128) / 16;
                        if (elect_one()) {
#pragma unroll
                            for (int kk = 0; kk < HD / 16; ++kk)
                                umma_bf16(cS + SK * hf, q + step_k(kk), k + step_k(kk), idesc, kk != 0);
                            umma_commit(&M.s_full[x][hf]);
                        }
                        __syncwarp();
                    }
                    if (go && elect_one()) umma_commit(&M.k_empty[stage]);
                    __syncwarp();
                }
            } else {
                constexpr uint32_t idesc = idesc_f16_f32(TR, HD) | IDESC_B_MN;
                const uint32_t cO = tmem_base + TM_O + 128u * x;
                const uint64_t v0 = desc_v(sV);
                for (int t = 0; go && t < ntiles; ++t) {
                    const uint32_t stage = (base + t) % STAGES;
                    if (!(go = wait_all(&M.v_full[stage], ((base + t) / STAGES) & 1))) break;
                    for (int hf = 0; go && !idle && hf < 2 && 2 * t + hf < nsteps; ++hf) {
                        if (!(go = wait_all(&M.p_full[x][hf], ((hf ? odd : even) + t) & 1))) break;
                        tc_fence_after();
                        const uint64_t v = v0 + (stage * TILE) / 16 + step_v(4 * hf);
                        if (elect_one()) {
#pragma unroll
                            for (int kk = 0; kk < SK / 16; ++kk)
                                umma_f16_ts(cO, cS + SK * hf + 8u * kk, v + step_v(kk), idesc, (t | hf | kk) != 0);
                            umma_commit(&M.pv_done[x][hf]);
                        }
                        __syncwarp();
                    }
                    if (go && elect_one()) umma_commit(&M.v_empty[stage]);
                    __syncwarp();
                }
            }
            __syncwarp();
            base += ntiles;
            if (!idle) {
                even += (nsteps + 1) / 2;
                odd += nsteps / 2;
            }
            __syncthreads();
        }
        if (elect_one()) {
            umma_commit(&M.drain[who]);  // every MMA issued here completes before TMEM is released
            mbar_wait_drain(&M.drain[who], 0, DRAIN_NS);
        }
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 16) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem_base, 512);
    }
    if (threadIdx.x == 0 && *abort_flag) *reinterpret_cast<volatile int*>(P.err.mirror) = DEV_ERR_TIMEOUT;
}

// Joins the pieces of the units that several CTAs shared, in the order of their keys,
// a warp a row: 256 rows of a unit are too many for its last CTA, which was 20 to
// 30 us behind the others (1024 tokens over 16K: 570 us with that, 527 without).
constexpr int JOIN_ROWS = 32;  // of a CTA
template <int HD>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ AttnParams P) {
    constexpr int PER = ROWS / JOIN_ROWS;
    const int unit = blockIdx.x / PER, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int entries = P.q.n_seq * P.row_blocks;
    const int h = unit % P.c.H, e = unit / P.c.H % entries, l = unit / P.c.H / entries;
    const RowBlock B = row_block(P, e / P.row_blocks, e % P.row_blocks, ROWS);
    const int row0 = (blockIdx.x % PER) * JOIN_ROWS;
    if (row0 >= B.nrows) return;
    if (!KVB_IN_BOUNDS(P.err, unit, 1, P.units)) return;
    const int2 by = P.shared_by[unit];
    if (by.x <= 1) return;
    const Pieces pieces{by.x, by.y};
    if (!pieces_in_bounds(P, pieces)) return;
    for (int row = row0 + warp; row < min(row0 + JOIN_ROWS, B.nrows); row += 8) {
        auto stat = [&](int i) { return P.part_stat[pieces.slot(i) * ROWS + row]; };
        Joined z;
        for (int i = lane; i < pieces.n; i += 32) z.reference(stat(i));
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) {
            z.m = fmaxf(z.m, __shfl_xor_sync(0xffffffffu, z.m, x));
            z.mv = fmaxf(z.mv, __shfl_xor_sync(0xffffffffu, z.mv, x));
        }
#pragma unroll 4
        for (int i = 0; i < pieces.n; ++i)
            z.add(stat(i), reinterpret_cast<const float4*>(P.partial + (pieces.slot(i) * ROWS + row) * HD)[lane % (HD / 4)]);
        const int64_t o = B.row_of(P, (static_cast<int64_t>(l) * P.c.H + h) * P.g, row);
        if (!KVB_IN_BOUNDS(P.err, o, 1, rows_of(P))) continue;
        if (lane < HD / 4) store_out(static_cast<__nv_bfloat16*>(P.out) + o * HD + 4 * lane, z.output());
        if (lane == 0 && P.lse) P.lse[o] = z.lse();
    }
}

template <int HD>
cudaError_t launch(const AttnParams& P, const AttnPlan& p, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(prefill_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes(HD));
    if (e != cudaSuccess) return e;
    prefill_kernel<HD><<<p.ctas, NUM_THREADS, smem_bytes(HD), s>>>(P);
    if ((e = cudaGetLastError()) != cudaSuccess || p.ctas == 1) return e;
    join_kernel<HD><<<static_cast<unsigned>(p.units * (ROWS / JOIN_ROWS)), 256, 0, s>>>(P);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prefill(const AttnParams& P, const AttnPlan& p, cudaStream_t s) {
    return P.c.d == 64 ? launch<64>(P, p, s) : launch<128>(P, p, s);
}

}  // namespace c8
}  // namespace kvb
