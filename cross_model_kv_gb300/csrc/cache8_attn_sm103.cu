// Attention over the paged 8-bit cache on the 5th-generation tensor cores: many
// query rows (prompts over a cached prefix), bf16, head_dim 128.
//
// The mathematics and the references are those of cache8_attn.cu; here the
// product of the rows (tokens x query heads of a KV head) with the keys is large
// enough to be bound by the tensor cores.  One CTA takes 256 rows as two tiles
// of 128 and walks the keys 128 at a time:
//   warps 8..11   read the codes (prefetched into registers a tile ahead),
//                 convert them to fp16 (exact) and lay them out as operands, keys
//                 and values alike: 128-byte swizzle, key rows, K-major for S and
//                 MN-major for O; also the scales of the tile's 16-key groups;
//   warp 12       one thread issues S_x = Q_x K^T (SS) and O_x += P_x V (P from TMEM)
//                 for the tiles x = 0, 1 in turn, so that one tile's softmax runs
//                 under the other's products;
//   warps 0..3, 4..7  softmax of tile 0, 1, a row a thread: S from TMEM twice (the
//                 maximum, then the weights), P as fp16 over the S just read, the
//                 sum in fp32; O is rescaled in TMEM on the rare raise.
// TMEM: S_x at 128 x, O_x at 256 + 128 x.  P_x lies in S_x's columns, so S_x of
// the next tile is issued when O_x += P_x V has completed.
// The weights carry the value scale, w = 2^(s + e_v - mv); a 16-key group's sum goes
// into the denominator with the factor 2^(mv - m - e_v), or is taken from
// exponentials of its own where that factor could leave fp32's range.
// Every wait is bounded.
#include "cache8_attn.cuh"

namespace kvb {
namespace c8 {

namespace {

constexpr int TR = 128;  // rows of a tile
constexpr int TK = 128;  // keys of a step
constexpr int HD = 128;
constexpr int ATOM = 128 * 128;  // bytes of 128 rows x 64 fp16
constexpr int TILE = 2 * ATOM;
constexpr int NUM_THREADS = 416;
constexpr int INFO_RING = 4;  // scales are written at most three tiles before the slowest softmax reads them
constexpr int SMEM_BYTES = 6 * TILE + 1024 + 1024;
constexpr uint64_t DRAIN_NS = 200ull * 1000 * 1000;

__device__ __forceinline__ uint32_t sw_off(int r, int c) {  // 16-byte chunk c (0..15) of row r
    return static_cast<uint32_t>((c >> 3) * ATOM + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}
__device__ __forceinline__ uint64_t desc_k(const uint8_t* tile, int kk) {
    return sdesc_k_sw128(smem_u32(tile) + (kk >> 2) * ATOM + (kk & 3) * 32);
}
__device__ __forceinline__ uint64_t desc_v(const uint8_t* tile, int kk) {
    return sdesc_mn_sw128(smem_u32(tile) + kk * 16 * 128, ATOM);
}
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
    uint64_t* s_full = bar + 8;    // [2] tile x
    uint64_t* p_full = bar + 10;   // [2]
    uint64_t* pv_done = bar + 12;  // [2]
    uint64_t* q_full = bar + 14;
    uint64_t* drain = bar + 15;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar + 16);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* s_last = reinterpret_cast<int*>(tmem_slot + 2);
    uint64_t* info_full = bar + 18;  // [INFO_RING]
    TileInfo* info = reinterpret_cast<TileInfo*>(bar + 18 + INFO_RING);

    const int split = blockIdx.x;
    const int64_t unit = blockIdx.y + static_cast<int64_t>(blockIdx.z) * gridDim.y;
    const int h = blockIdx.y % P.c.H;
    const int rb = blockIdx.y / P.c.H;
    const int s = blockIdx.z % P.q.n_seq;
    const int l = blockIdx.z / P.q.n_seq;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    RowBlock B;
    if (!row_block(P, s, rb, 2 * TR, split, B)) return;
    const int ntiles = (B.k1 - B.k0 + TK - 1) / TK;
    const int64_t layer = static_cast<int64_t>(P.c.l_begin) + l;
    const int64_t hq0 = (static_cast<int64_t>(l) * P.c.H + h) * P.g;
    const DevErr derr{P.err.word, P.err.timeout_ns};

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&k_full[i], 128);
            mbar_init(&k_empty[i], 1);
            mbar_init(&v_full[i], 128);
            mbar_init(&v_empty[i], 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 128);
            mbar_init(&pv_done[i], 1);
        }
        for (int i = 0; i < INFO_RING; ++i) mbar_init(&info_full[i], 8);
        mbar_init(q_full, 256);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 12) {
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
        // the row as fp16 under a power of two: largest element in [2^13, 2^14)
        float qs;
        {
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
        const int qpos = valid ? B.pos + static_cast<int>(tok) : INT32_MIN;
        for (int t = 0; t < ntiles; ++t) {
            ok = wait_all(&info_full[t & (INFO_RING - 1)], (t / INFO_RING) & 1) && wait_all(&s_full[x], t & 1);
            if (!ok) break;
            tc_fence_after();
            const TileInfo& I = info[t & (INFO_RING - 1)];
            // visible keys of this row are a prefix of the tile
            const int j0 = B.k0 + t * TK;
            const int nvis = static_cast<int>(min(static_cast<int64_t>(min(B.k1, qpos == INT32_MAX ? B.k1 : qpos + 1)) - j0,
                                                  static_cast<int64_t>(TK)));
            bool whole = nvis == TK;
#pragma unroll
            for (int gq = 0; gq < 8; ++gq) whole &= I.ks[gq] != 0.f;
            whole = __all_sync(0xffffffffu, whole);
            // pass 1: the maxima of s and of s + e_v
            float ms = -INFINITY, mvs = -INFINITY;
#pragma unroll 1
            for (int c0 = 0; c0 < TK; c0 += 32) {
                uint32_t sv[2][16];
                tmem_ld16(tS + c0, sv[0]);
                tmem_ld16(tS + c0 + 16, sv[1]);
                tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int gq = (c0 >> 4) + c;
                    float top = -INFINITY;
                    if (whole) {
#pragma unroll
                        for (int u = 0; u < 16; ++u) top = fmaxf(top, __uint_as_float(sv[c][u]));
                    } else {
#pragma unroll
                        for (int u = 0; u < 16; ++u)
                            if (16 * gq + u < nvis && I.ks[gq] != 0.f) top = fmaxf(top, __uint_as_float(sv[c][u]));
                    }
                    if (top > -INFINITY) {
                        top *= I.ks[gq] * qs;
                        ms = fmaxf(ms, top);
                        mvs = fmaxf(mvs, top + I.ev[gq]);
                    }
                }
            }
            __syncwarp();
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
                if (t > 0) {
#pragma unroll 1
                    for (int c0 = 0; c0 < HD; c0 += 16) {
                        uint32_t o[16];
                        tmem_ld16(tO + c0, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int u = 0; u < 16; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * f);
                        tmem_st16(tO + c0, o);
                    }
                    tmem_st_wait();
                }
            }
            // pass 2: the weights, over the scores just read
#pragma unroll 1
            for (int c0 = 0; c0 < TK; c0 += 32) {
                uint32_t sv[2][16];
                tmem_ld16(tS + c0, sv[0]);
                tmem_ld16(tS + c0 + 16, sv[1]);
                tmem_ld_wait();
                uint32_t pw[16];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int gq = (c0 >> 4) + c;
                    const float k = I.ks[gq] * qs, ev = I.ev[gq], b = ev - mv + BIAS;
                    float w[16];
                    if (whole) {
#pragma unroll
                        for (int u = 0; u < 16; ++u) w[u] = ex2(fmaf(__uint_as_float(sv[c][u]), k, b));
                    } else {
#pragma unroll
                        for (int u = 0; u < 16; ++u)
                            w[u] = 16 * gq + u < nvis && k != 0.f ? ex2(fmaf(__uint_as_float(sv[c][u]), k, b)) : 0.f;
                    }
                    float p = 0.f;
                    const float e = mv - m - ev;
                    if (fabsf(e) < 60.f) {
#pragma unroll
                        for (int u = 0; u < 16; ++u) p += w[u];
                        p *= ex2(e);
                    } else {
#pragma unroll
                        for (int u = 0; u < 16; ++u)
                            if (16 * gq + u < nvis && k != 0.f) p += ex2(fmaf(__uint_as_float(sv[c][u]), k, BIAS - m));
                    }
                    sum += p;
#pragma unroll
                    for (int u = 0; u < 8; ++u) pw[8 * c + u] = pack_half2(w[2 * u], w[2 * u + 1]);
                }
                __syncwarp();  // the warp-wide store, after branches that lanes take apart
                tmem_st16(tS + (c0 >> 1), pw);
            }
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&p_full[x]);
        }
        ok = ok && (ntiles == 0 || wait_all(&pv_done[x], (ntiles - 1) & 1));
    } else if (warp < 12) {
        // ------------------------------------------------------- codes -> fp16 operands
        const int tid = threadIdx.x - 256;
        const int r8 = tid >> 3, c16 = tid & 7;  // row within a 16-key group, 16-code column
        const int* table = P.q.page_table + static_cast<int64_t>(s) * P.q.max_pages;
        const int pm = P.c.page - 1;
        uint4 kr[8], vr[8];
        auto load = [&](int kv, int t, uint4 (&u)[8]) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int j = B.k0 + t * TK + 16 * i;
                u[i] = make_uint4(0, 0, 0, 0);
                if (j + r8 < B.k1) {  // slots past the last visible key may hold anything
                    const int pid = __ldg(table + (j >> P.c.page_log2));
                    if (pid >= 0 && pid < P.c.n_pages) {
                        const int64_t blk = (layer * P.c.n_pages + pid) * P.c.H + h;
                        u[i] = __ldg(reinterpret_cast<const uint4*>(P.c.code[kv] + ((blk << P.c.page_log2) + (j & pm) + r8) * HD) + c16);
                    }
                }
            }
        };
        auto store = [&](uint8_t* tile, const uint4 (&u)[8]) {
            // codes 16 c16 .. +15 are chunks 2 c16 and 2 c16 + 1; lanes of the upper 64 dims
            // store theirs in the other order, so that eight lanes hit eight bank groups
            const int flip = c16 >> 2;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint4 a = make_uint4(half2_of_lo(u[i].x), half2_of_hi(u[i].x), half2_of_lo(u[i].y), half2_of_hi(u[i].y));
                const uint4 b = make_uint4(half2_of_lo(u[i].z), half2_of_hi(u[i].z), half2_of_lo(u[i].w), half2_of_hi(u[i].w));
                *reinterpret_cast<uint4*>(tile + sw_off(16 * i + r8, 2 * c16 + flip)) = flip ? b : a;
                *reinterpret_cast<uint4*>(tile + sw_off(16 * i + r8, 2 * c16 + 1 - flip)) = flip ? a : b;
            }
        };
        if (ntiles > 0) {
            load(0, 0, kr);
            load(1, 0, vr);
        }
        for (int t = 0; t < ntiles; ++t) {
            const int b = t & 1;
            float ks = 0.f, ev = 0.f;
            if (tid < 8) {
                const int j = B.k0 + t * TK + 16 * tid;
                if (j < B.k1) {
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
            if (t + 1 < ntiles) load(0, t + 1, kr);
            if (!mbar_wait(&v_empty[b], ((t >> 1) & 1) ^ 1, derr, abort_flag)) break;
            store(sV + b * TILE, vr);
            fence_proxy_async_smem();
            mbar_arrive(&v_full[b]);
            if (t + 1 < ntiles) load(1, t + 1, vr);
        }
    } else if (lane == 0 && ntiles > 0) {
        // ------------------------------------------------------- MMA issuer
        constexpr uint32_t idesc_s = idesc_f16_f32(TR, TK);
        constexpr uint32_t idesc_o = idesc_f16_f32(TR, HD) | IDESC_B_MN;
        auto scores = [&](int xx, int b) {
#pragma unroll
            for (int kk = 0; kk < HD / 16; ++kk)
                umma_bf16(tmem_base + 128u * xx, desc_k(sQ + xx * TILE, kk), desc_k(sK + b * TILE, kk), idesc_s, kk != 0);
            umma_commit(&s_full[xx]);
        };
        bool go = mbar_wait(q_full, 0, derr, abort_flag) && mbar_wait(&k_full[0], 0, derr, abort_flag);
        if (go) {
            tc_fence_after();
            scores(0, 0);
            scores(1, 0);
            umma_commit(&k_empty[0]);
        }
        for (int t = 0; go && t < ntiles; ++t) {
            const int b = t & 1, nb = (t + 1) & 1;
            go = mbar_wait(&v_full[b], (t >> 1) & 1, derr, abort_flag);
            if (go && t + 1 < ntiles) go = mbar_wait(&k_full[nb], ((t + 1) >> 1) & 1, derr, abort_flag);
            for (int xx = 0; go && xx < 2; ++xx) {
                go = mbar_wait(&p_full[xx], t & 1, derr, abort_flag);
                if (!go) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < TK / 16; ++kk)
                    umma_f16_ts(tmem_base + 256u + 128u * xx, tmem_base + 128u * xx + 8u * kk, desc_v(sV + b * TILE, kk),
                                idesc_o, (t | kk) != 0);
                umma_commit(&pv_done[xx]);
                if (t + 1 < ntiles) {
                    go = mbar_wait(&pv_done[xx], t & 1, derr, abort_flag);
                    if (go) scores(xx, nb);
                }
            }
            if (go) {
                umma_commit(&v_empty[b]);
                if (t + 1 < ntiles) umma_commit(&k_empty[nb]);
            }
        }
        umma_commit(drain);  // every MMA issued here completes before TMEM is released
        mbar_wait_drain(drain, 0, DRAIN_NS);
    }

    // outputs: from TMEM (units of 2^mv, sums of 2^m, both with the bias)
    if (warp < 8) {
        const bool have = ok && ntiles > 0;
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
            if (valid && B.active == 1) {
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
            if (B.active > 1) P.part_stat[part] = make_float4(m, mv, sum, 0.f);
            else if (P.lse) P.lse[out_row] = sum == 0.f ? -INFINITY : (m - BIAS + log2f(sum)) * 0.693147180559945f;
        }
    }
    tc_fence_before();
    __threadfence();
    __syncthreads();
    if (warp == 12) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem_base, 512);
    }
    if (threadIdx.x == 0 && *abort_flag) *reinterpret_cast<volatile int*>(P.err.mirror) = DEV_ERR_TIMEOUT;
    if (B.active > 1) join_splits<__nv_bfloat16, HD, 2 * TR, NUM_THREADS>(P, B, unit, hq0, s_last);
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
