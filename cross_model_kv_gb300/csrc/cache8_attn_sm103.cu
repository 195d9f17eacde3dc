// Attention over the paged 8-bit cache on the 5th-generation tensor cores: many
// query rows (prompts over a cached prefix), bf16, head_dim 128.
//
// The mathematics and the references are those of cache8_attn.cu; here the
// product of the rows (tokens x query heads of a KV head) with the keys is large
// enough to be bound by the tensor cores.  One CTA takes 256 rows as two tiles
// of 128 and walks the keys 128 at a time:
//   warps 8..15   read the codes (prefetched into registers a tile ahead),
//                 convert them to fp16 (exact) and lay them out as operands, keys
//                 and values alike: 128-byte swizzle, key rows, K-major for S and
//                 MN-major for O; also the scales of the tile's 16-key groups;
//   warps 16, 17  one thread each issues S_x = Q_x K^T (SS) for tile x;
//   warps 18, 19  and O_x += P_x V (P from TMEM): four threads, so that no product
//                 waits behind a wait of another kind;
//   warps 0..3, 4..7  softmax of tile 0, 1, a row a thread, 64 keys a step: scores
//                 from TMEM to registers, P as fp16 over them, the sum in fp32; O is
//                 rescaled in TMEM on the rare raise.
// TMEM: score buffer b of tile x at 128 x + 64 b, O_x at 256 + 128 x.  P takes its
// scores' columns, so a buffer's next scores are issued when O_x += P V has
// completed; meanwhile the softmax works on the other buffer (one buffer of 128
// keys left it waiting 2500 of 5800 cycles for each 128 keys).
// The weights carry the value scale, w = 2^(s + e_v - mv); a 16-key group's sum goes
// into the denominator with the factor 2^(mv - m - e_v), or is taken from
// exponentials of its own where that factor could leave fp32's range.
// Every wait is bounded.
#include <cfloat>

#include "cache8_attn.cuh"

namespace kvb {
namespace c8 {

namespace {

constexpr int TR = 128;  // rows of a tile
constexpr int TK = 128;  // keys of an operand tile
constexpr int SK = 64;   // keys of a step (two score buffers a tile in TMEM)
constexpr int HD = 128;
constexpr int ATOM = 128 * 128;  // bytes of 128 rows x 64 fp16
constexpr int TILE = 2 * ATOM;
constexpr int NUM_THREADS = 640;
constexpr int CONV = 256;  // threads that convert
// Registers a thread: 96 at launch, then by role.  256 * 144 + 256 * 72 + 128 * 40 = 60416 of
// the launch's 640 * 96 = 61440.
constexpr int REGS_SOFTMAX = 144, REGS_CONVERT = 72, REGS_MMA = 40;
constexpr int INFO_RING = 4;  // scales are written at most three tiles before the slowest softmax reads them
constexpr int SMEM_BYTES = 6 * TILE + 1024 + 1024;
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
// A from TMEM (lane = row, two fp16 a column)
__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

template <int N>
__device__ __forceinline__ void regs_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// 32 lanes x 32 bits, 32 consecutive columns per thread (no wait).
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,"
        "%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z, w;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, w;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

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

struct TileInfo {
    float ks[8], ev[8];  // key scale (0: the page is bad, nothing of it is seen) and value exponent, 16 keys each
};

__global__ void __launch_bounds__(NUM_THREADS, 1) prefill_kernel(const __grid_constant__ AttnParams P) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* sQ = smem;
    uint8_t* sK = smem + 2 * TILE;
    uint8_t* sV = smem + 4 * TILE;
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem + 6 * TILE);
    uint64_t* k_full = bar;        // [2]
    uint64_t* k_empty = bar + 2;   // [2]
    uint64_t* v_full = bar + 4;    // [2]
    uint64_t* v_empty = bar + 6;   // [2]
    uint64_t* s_full = bar + 8;    // [tile x][buffer]
    uint64_t* p_full = bar + 12;   // [tile x][buffer]
    uint64_t* pv_done = bar + 16;  // [tile x][buffer]
    uint64_t* drain = bar + 20;    // [issuer]
    uint64_t* q_full = bar + 24;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar + 25);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* s_last = reinterpret_cast<int*>(tmem_slot + 2);
    uint64_t* info_full = bar + 28;  // [INFO_RING]
    TileInfo* info = reinterpret_cast<TileInfo*>(bar + 28 + INFO_RING);

    const int split = blockIdx.x;
    const int64_t unit = blockIdx.y + static_cast<int64_t>(blockIdx.z) * gridDim.y;
    const int h = blockIdx.y % P.c.H;
    const int rb = blockIdx.y / P.c.H;
    const int s = blockIdx.z % P.q.n_seq;
    const int l = blockIdx.z / P.q.n_seq;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    const RowBlock B = row_block(P, s, rb, 2 * TR);
    const int active = max(1, (B.kv_end + P.chunk - 1) / P.chunk);  // chunks that have keys
    if (B.nrows == 0 || split >= active) return;
    const int k0 = split * P.chunk, k1 = min(B.kv_end, k0 + P.chunk);
    const int ntiles = (k1 - k0 + TK - 1) / TK, nsteps = (k1 - k0 + SK - 1) / SK;
    const int tiles = B.nrows > TR ? 2 : 1;  // the second tile's warps have nothing to do where there is one
    const int64_t layer = static_cast<int64_t>(P.c.l_begin) + l;
    const int64_t hq0 = (static_cast<int64_t>(l) * P.c.H + h) * P.g;
    const DevErr derr{P.err.word, P.err.timeout_ns};

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&k_full[i], CONV);
            mbar_init(&k_empty[i], tiles);
            mbar_init(&v_full[i], CONV);
            mbar_init(&v_empty[i], tiles);
            mbar_init(&s_full[2 * i], 1);
            mbar_init(&s_full[2 * i + 1], 1);
            mbar_init(&p_full[2 * i], 128);
            mbar_init(&p_full[2 * i + 1], 128);
            mbar_init(&pv_done[2 * i], 1);
            mbar_init(&pv_done[2 * i + 1], 1);
            mbar_init(&drain[2 * i], 1);
            mbar_init(&drain[2 * i + 1], 1);
        }
        for (int i = 0; i < INFO_RING; ++i) mbar_init(&info_full[i], 8);
        mbar_init(q_full, TR * tiles);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 16) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    auto wait_all = [&](uint64_t* b, uint32_t parity) {  // warp-uniform outcome
        return __all_sync(0xffffffffu, mbar_wait(b, parity, derr, abort_flag)) != 0;
    };

    // softmax warps: this thread's row
    const int x = warp >> 2;                 // tile
    const int row = threadIdx.x & 127;       // row of the tile
    const int brow = threadIdx.x;            // row of the block
    const bool valid = warp < 8 && brow < B.nrows;
    float m = NO_REF, mv = NO_REF, sum = 0.f;
    bool ok = true;
    const int64_t gr = B.row0 + (valid ? brow : 0);
    const int64_t tok = gr / P.g;
    const int64_t out_row = (hq0 + (gr - tok * P.g)) * P.q.T + B.tok0 + tok;  // in [n_layers][Hq][T]
    const uint32_t tl = tmem_base + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    const uint32_t tS = tl + 128u * x, tO = tl + 256u + 128u * x;

    if (warp < 8) {
        regs_up<REGS_SOFTMAX>();
        // the row as fp16 under a power of two: largest element in [2^13, 2^14)
        float qs = 1.f;
        if (x < tiles) {
            const uint4* q = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(P.query) + out_row * HD);
            uint4 u[16];
#pragma unroll
            for (int c = 0; c < 16; ++c) u[c] = valid ? __ldg(q + c) : make_uint4(0, 0, 0, 0);
            float amax = 0.f;
#pragma unroll
            for (int c = 0; c < 16; ++c) {
                const uint32_t w[4] = {u[c].x, u[c].y, u[c].z, u[c].w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xffff0000u))));
            }
            const int eq = max((__float_as_int(amax) >> 23) - 127, -100) - 13;
            const float inv = pow2(-eq);
            qs = pow2(eq) * P.scale_log2;
#pragma unroll
            for (int c = 0; c < 16; ++c) {
                const uint32_t w[4] = {u[c].x, u[c].y, u[c].z, u[c].w};
                uint32_t o[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o[i] = pack_half2(__uint_as_float(w[i] << 16) * inv, __uint_as_float(w[i] & 0xffff0000u) * inv);
                *reinterpret_cast<uint4*>(sQ + x * TILE + sw_off(row, c)) = make_uint4(o[0], o[1], o[2], o[3]);
            }
            fence_proxy_async_smem();
            mbar_arrive(q_full);
        }
        // keys below `see` are visible to this row
        const int see = valid ? min(k1, B.pos + static_cast<int>(tok) + 1) : 0;
        for (int u = 0; x < tiles && u < nsteps; ++u) {
            const int t = u >> 1, hf = u & 1;
            if (hf == 0) ok = wait_all(&info_full[t & (INFO_RING - 1)], (t / INFO_RING) & 1);
            ok = ok && wait_all(&s_full[2 * x + hf], t & 1);
            if (!ok) break;
            tc_fence_after();
            const uint32_t cS = tS + SK * hf;
            uint32_t sv[SK];
            tmem_ld32(cS, sv);
            tmem_ld32(cS + 32, sv + 32);
            const TileInfo& I = info[t & (INFO_RING - 1)];
            const float4 ks4 = *reinterpret_cast<const float4*>(I.ks + 4 * hf), ev4 = *reinterpret_cast<const float4*>(I.ev + 4 * hf);
            const float ev[4] = {ev4.x, ev4.y, ev4.z, ev4.w};
            const float k[4] = {fmaxf(ks4.x * qs, FLT_MIN), fmaxf(ks4.y * qs, FLT_MIN), fmaxf(ks4.z * qs, FLT_MIN),
                                fmaxf(ks4.w * qs, FLT_MIN)};
            // visible keys of this row are a prefix of the step's
            const int nvis = min(see - (k0 + u * SK), SK);
            const bool whole = nvis == SK && ks4.x != 0.f && ks4.y != 0.f && ks4.z != 0.f && ks4.w != 0.f;
            tmem_ld_wait();
            if (!__all_sync(0xffffffffu, whole)) {
                const float seen[4] = {ks4.x, ks4.y, ks4.z, ks4.w};
#pragma unroll
                for (int j = 0; j < SK; ++j)
                    if (j >= nvis || seen[j >> 4] == 0.f) sv[j] = 0xff800000u;  // -inf
            }
            // maxima of s and of s + e_v (factors are positive)
            float ms = -INFINITY, mvs = -INFINITY;
#pragma unroll
            for (int gq = 0; gq < 4; ++gq) {
                float top[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    top[j] = fmaxf(fmaxf(__uint_as_float(sv[16 * gq + 4 * j]), __uint_as_float(sv[16 * gq + 4 * j + 1])),
                                   fmaxf(__uint_as_float(sv[16 * gq + 4 * j + 2]), __uint_as_float(sv[16 * gq + 4 * j + 3])));
                const float best = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * k[gq];
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
                    ok = wait_all(&pv_done[2 * x + (hf ^ 1)], ((u - 1) >> 1) & 1);  // O is complete up to the step before
                    if (!ok) break;
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
            // the weights; P takes the columns of the scores
            float factor = 0.f;
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
                    if (gq == 0 || ev[gq] != ev[gq - 1]) factor = ex2(e);
                    float2 p = add2(add2(add2(w[0], w[1]), add2(w[2], w[3])), add2(add2(w[4], w[5]), add2(w[6], w[7])));
                    float p1 = (p.x + p.y) * factor;
                    if (fabsf(e) > 60.f) {
                        p1 = 0.f;
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            p1 += ex2(fmaf(__uint_as_float(sv[16 * gq + j]), k[gq], BIAS - m));
                    }
                    sum += p1;
                }
                __syncwarp();  // the warp-wide store, after branches that lanes may take apart
                tmem_st16(cS + 16 * g2, pw);
            }
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&p_full[2 * x + hf]);
        }
        if (x < tiles && nsteps > 0) ok = ok && wait_all(&pv_done[2 * x + ((nsteps - 1) & 1)], ((nsteps - 1) >> 1) & 1);

        // outputs: from TMEM (units of 2^mv, sums of 2^m, both with the bias)
        const bool have = x < tiles && ok && nsteps > 0;
        if (have) tc_fence_after();
        const int64_t part = (unit * P.splits + split) * (2 * TR) + brow;
        const float half = ex2(0.5f * (mv - m)), f = sum == 0.f ? 0.f : half / sum;
#pragma unroll 1
        for (int c0 = 0; c0 < HD; c0 += 16) {
            uint32_t o[16];
            if (have) {
                tmem_ld16(tO + c0, o);
                tmem_ld_wait();
            } else {
#pragma unroll
                for (int u = 0; u < 16; ++u) o[u] = 0u;
            }
            if (valid && active == 1) {
                uint32_t w[8];
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    w[u] = pack_bf16x2(__uint_as_float(o[2 * u]) * f * half, __uint_as_float(o[2 * u + 1]) * f * half);
                uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(P.out) + out_row * HD + c0);
                dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
                dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
            } else if (valid) {
                uint4* dst = reinterpret_cast<uint4*>(P.partial + part * HD + c0);
#pragma unroll
                for (int u = 0; u < 4; ++u) dst[u] = make_uint4(o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]);
            }
            __syncwarp();
        }
        if (valid) {
            if (active > 1) P.part_stat[part] = make_float4(m, mv, sum, 0.f);
            else if (P.lse) P.lse[out_row] = sum == 0.f ? -INFINITY : (m - BIAS + log2f(sum)) * 0.693147180559945f;
        }
        if (active > 1) join_splits<__nv_bfloat16, HD, 2 * TR, 256, true>(P, B, Pieces{active, unit * P.splits, unit * P.splits + 1, 1}, unit, hq0, s_last, reinterpret_cast<float*>(sQ), 2 * TILE / 4);
    } else if (warp < 16) {
        // ------------------------------------------------------- codes -> fp16 operands
        regs_down<REGS_CONVERT>();
        const int tid = threadIdx.x - 256;
        const int r32 = tid >> 3, c16 = tid & 7;  // row within 32 keys, 16-code column
        const int* table = P.q.page_table + static_cast<int64_t>(s) * P.q.max_pages;
        const int pm = P.c.page - 1;
        const int last = max(k1 - 1, 0);
        // this thread's first code in page 0, and bytes from one page's block to the next's
        const int64_t first = (((layer * P.c.n_pages) * P.c.H + h) << P.c.page_log2) * HD + c16 * 16;
        const uint8_t* base[2] = {P.c.code[0] + first, P.c.code[1] + first};
        const uint32_t page_bytes = static_cast<uint32_t>(P.c.H << P.c.page_log2) * HD;
        uint4 kr[4], vr[4];
        int pid[4], pid_next[4];  // pages of the tile being loaded and of the one after it
        auto pages = [&](int t, int (&p)[4]) {
#pragma unroll
            for (int i = 0; i < 4; ++i) p[i] = __ldg(table + (min(k0 + t * TK + 32 * i + r32, last) >> P.c.page_log2));
        };
        auto load = [&](int kv, int t, uint4 (&u)[4]) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = k0 + t * TK + 32 * i + r32;
                // slots past the last visible key may hold anything: not read
                const bool have = j < k1 && pid[i] >= 0 && pid[i] < P.c.n_pages;
                u[i] = load16_if(base[kv] + static_cast<uint64_t>(static_cast<uint32_t>(pid[i])) * page_bytes + (j & pm) * HD, have);
            }
        };
        auto store = [&](uint8_t* tile, const uint4 (&u)[4]) {
            // codes 16 c16 .. +15 are chunks 2 c16 and 2 c16 + 1; lanes of the upper 64 dims
            // store theirs in the other order, so that eight lanes hit eight bank groups
            const int flip = c16 >> 2;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 a = make_uint4(half2_of_lo(u[i].x), half2_of_hi(u[i].x), half2_of_lo(u[i].y), half2_of_hi(u[i].y));
                const uint4 b = make_uint4(half2_of_lo(u[i].z), half2_of_hi(u[i].z), half2_of_lo(u[i].w), half2_of_hi(u[i].w));
                *reinterpret_cast<uint4*>(tile + sw_off(32 * i + r32, 2 * c16 + flip)) = flip ? b : a;
                *reinterpret_cast<uint4*>(tile + sw_off(32 * i + r32, 2 * c16 + 1 - flip)) = flip ? a : b;
            }
        };
        if (ntiles > 0) {
            pages(0, pid);
            pages(1, pid_next);
            load(0, 0, kr);
            load(1, 0, vr);
        }
        for (int t = 0; t < ntiles; ++t) {
            const int b = t & 1;
            float ks = 0.f, ev = 0.f;
            if (tid < 8) {
                const int j = k0 + t * TK + 16 * tid;
                if (j < k1) {
                    const int pid = __ldg(table + (j >> P.c.page_log2));
                    if (pid >= 0 && pid < P.c.n_pages) {
                        const int64_t blk = (layer * P.c.n_pages + pid) * P.c.H + h;
                        ks = __ldg(P.c.scale[0] + blk);
                        ev = static_cast<float>(exponent_of(__ldg(P.c.scale[1] + blk)));
                    } else {
                        err_set(P.err, DEV_ERR_BAD_SEQ);
                    }
                }
            }
            if (!mbar_wait(&k_empty[b], ((t >> 1) & 1) ^ 1, derr, abort_flag)) break;
            if (tid < 8) {
                TileInfo& I = info[t & (INFO_RING - 1)];
                I.ks[tid] = ks;
                I.ev[tid] = ev;
                mbar_arrive(&info_full[t & (INFO_RING - 1)]);
            }
            store(sK + b * TILE, kr);
            fence_proxy_async_smem();
            mbar_arrive(&k_full[b]);
#pragma unroll
            for (int i = 0; i < 4; ++i) pid[i] = pid_next[i];
            if (t + 1 < ntiles) load(0, t + 1, kr);
            if (t + 2 < ntiles) pages(t + 2, pid_next);
            if (!mbar_wait(&v_empty[b], ((t >> 1) & 1) ^ 1, derr, abort_flag)) break;
            store(sV + b * TILE, vr);
            fence_proxy_async_smem();
            mbar_arrive(&v_full[b]);
            if (t + 1 < ntiles) load(1, t + 1, vr);
        }
    } else {
        // ------------------------------------------------------- MMA issuer
        regs_down<REGS_MMA>();
        const int xx = warp & 1;
        if (lane == 0 && nsteps > 0 && xx < tiles) {
            const uint32_t cS = tmem_base + 128u * xx;
            if (warp < 18) {
                constexpr uint32_t idesc = idesc_f16_f32(TR, SK);
                const uint64_t q = desc_k(sQ + xx * TILE), k0 = desc_k(sK);
                bool go = mbar_wait(q_full, 0, derr, abort_flag);
                for (int u = 0; go && u < nsteps; ++u) {
                    const int t = u >> 1, hf = u & 1;
                    if (hf == 0 && !(go = mbar_wait(&k_full[t & 1], (t >> 1) & 1, derr, abort_flag))) break;
                    // P of step u - 2 lies where these scores go
                    if (u > 1 && !(go = mbar_wait(&pv_done[2 * xx + hf], (t - 1) & 1, derr, abort_flag))) break;
                    tc_fence_after();
                    const uint64_t k = k0 + ((t & 1) * TILE + hf * 64 * 128) / 16;
#pragma unroll
                    for (int kk = 0; kk < HD / 16; ++kk) umma_bf16(cS + SK * hf, q + step_k(kk), k + step_k(kk), idesc, kk != 0);
                    umma_commit(&s_full[2 * xx + hf]);
                    if (hf == 1 || u + 1 == nsteps) umma_commit(&k_empty[t & 1]);
                }
            } else {
                constexpr uint32_t idesc = idesc_f16_f32(TR, HD) | IDESC_B_MN;
                const uint32_t cO = tmem_base + 256u + 128u * xx;
                const uint64_t v0 = desc_v(sV);
                for (int u = 0; u < nsteps; ++u) {
                    const int t = u >> 1, hf = u & 1;
                    if (hf == 0 && !mbar_wait(&v_full[t & 1], (t >> 1) & 1, derr, abort_flag)) break;
                    if (!mbar_wait(&p_full[2 * xx + hf], t & 1, derr, abort_flag)) break;
                    tc_fence_after();
                    const uint64_t v = v0 + ((t & 1) * TILE) / 16 + step_v(4 * hf);
#pragma unroll
                    for (int kk = 0; kk < SK / 16; ++kk)
                        umma_f16_ts(cO, cS + SK * hf + 8u * kk, v + step_v(kk), idesc, (u | kk) != 0);
                    umma_commit(&pv_done[2 * xx + hf]);
                    if (hf == 1) umma_commit(&v_empty[t & 1]);
                }
            }
            umma_commit(&drain[warp - 16]);  // every MMA issued here completes before TMEM is released
            mbar_wait_drain(&drain[warp - 16], 0, DRAIN_NS);
        }
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

}  // namespace

cudaError_t launch_prefill(const AttnParams& P, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(prefill_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
    if (e != cudaSuccess) return e;
    dim3 grid(P.splits, P.c.H * P.row_blocks, P.q.n_seq * P.c.n_layers);
    prefill_kernel<<<grid, NUM_THREADS, SMEM_BYTES, s>>>(P);
    return cudaGetLastError();
}

}  // namespace c8
}  // namespace kvb
