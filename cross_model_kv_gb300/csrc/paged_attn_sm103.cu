// Attention over the paged cache on the 5th-generation tensor cores: more query rows than
// mma.sync keeps up with (drafted tokens being checked), bf16, head_dim 64 and 128.
//
// The mathematics and the references are those of paged_attn.cu.  One CTA an SM takes up to 128 rows
// of a unit (layer, sequence, row block, head) and walks its keys 64 at a time; the 64-key tiles
// of all units form one line that the CTAs share evenly.
//   warps 0..3  softmax, a row a thread: scores from TMEM to registers, P over them as a bf16
//               pair (16 bits of a weight), the sum in fp32; O is rescaled in TMEM on the rare raise.
//               They load the rows, write the outputs and join the pieces of shared units;
//   warp 4      page numbers, and TMA loads of K and V into a ring of tiles, 128-byte swizzle, key
//               rows: K-major for S, MN-major for O, as they lie in the pages;
//   warp 5      one lane issues S = Q K^T;
//   warp 6      and O += P V, the high parts and the low ones (P from TMEM).
// TMEM: score buffer b at 64 b, O at 128.  P takes its scores' columns.
// HBM bounds it (128 rows a key are 128 flop/byte, the machine has 280); a warp of the softmax whose rows
// do not exist only passes the barriers.  Every role finds the CTA's pieces by itself, so that
// the ring is filled (4 us of loads) while the softmax goes from one unit to the next.
// Every wait is bounded; after one gives up, the softmax still arrives at the units that it shares,
// so that their counters are left as the next call needs them, the loads and products that
// were issued are waited for, and TMEM is freed.
#include "kvb_host.h"
#include "paged_attn.cuh"

namespace kvb {
namespace paged {

namespace {

constexpr int TR = TENSOR_ROWS;  // rows of a unit, TMEM lanes
constexpr int TK = 64;           // keys of a tile
constexpr int SOFT = 128;        // threads of the softmax
constexpr int NUM_THREADS = SOFT + 96;
constexpr int GROUPS = TK / 16;  // 16 keys lie in one page
constexpr uint32_t TM_S = 0, TM_O = 128, TM_COLUMNS = 256;
constexpr uint64_t DRAIN_NS = 200ull * 1000 * 1000;

template <int HD>
struct Layout {
    static constexpr int Q_HALF = TR * 128, Q = HD / 64 * Q_HALF;      // 64 dims of all rows
    static constexpr int HALF = TK * 128, TILE = HD / 64 * HALF;       // of K, and of V
    static constexpr int STAGES = HD == 128 ? 5 : 8;
    static constexpr int BYTES = 1024 + Q + STAGES * 2 * TILE + 2048;
};

// A piece of a unit.
struct Segment {
    RowBlock B;
    int s, l, h;
    int k0, k1;  // keys [k0, k1)
    int64_t unit, slot;
    Pieces pieces;
    __device__ __forceinline__ int tiles() const { return (k1 - k0 + TK - 1) / TK; }
};

// The CTA's place in the line of tiles.
struct Walk {
    int at, stop, share, l, e, h, first;
    RowBlock B;
    int tiles;  // of unit (l, e, h); 0 before the first

    __device__ __forceinline__ RowBlock entry(const AttnParams& P) const {
        return c8::row_block(P, e / P.row_blocks, e % P.row_blocks, TR);
    }
    // The next piece, if there is one.
    __device__ __forceinline__ bool next(const AttnParams& P, Segment& g) {
        if (at >= stop) return false;
        const int entries = P.q.n_seq * P.row_blocks;
        if (tiles == 0) {
            B = entry(P);
            tiles = c8::unit_tiles<TK>(B);
            if (tiles == 0) return false;  // not reached while the call's arrays stay as they are, here and below
        } else {
            first = 0;
            if (++h == P.c.H) {
                h = 0;
                do {
                    if (++e == entries) {
                        e = 0;
                        if (++l == P.c.n_layers) return false;
                    }
                    B = entry(P);
                    tiles = c8::unit_tiles<TK>(B);
                } while (tiles == 0);
            }
        }
        const int last = min(tiles, first + (stop - at));
        const int u0 = at - first, c0 = u0 / share;
        g.B = B;
        g.s = e / P.row_blocks;
        g.l = l;
        g.h = h;
        g.k0 = first * TK;
        g.k1 = max(g.k0, min(B.kv_end, last * TK));
        g.unit = (static_cast<int64_t>(l) * entries + e) * P.c.H + h;
        g.pieces = Pieces{(u0 + tiles - 1) / share - c0 + 1, c0};
        g.slot = 2 * static_cast<int64_t>(blockIdx.x) + (first == 0);
        at += last - first;
        return true;
    }
};

struct Smem {
    uint64_t k_full[8], k_empty[8], v_full[8], v_empty[8];
    uint64_t s_full[2], p_full[2], pv_done[2], q_full, drain[2];
    uint32_t tmem;
    int abort;
    uint32_t present[8];  // of a stage: bit of a 16-key group whose page is there
    int scan[NUM_THREADS / 32];
    LineStart start;
    int last;
    alignas(16) float join[2 * TR];
};
static_assert(sizeof(Smem) <= 2048, "layout");

struct Maps {
    CUtensorMap kv[2];
};

template <int HD>
__global__ void __launch_bounds__(NUM_THREADS, 1) rows_kernel(const __grid_constant__ Maps maps, const __grid_constant__ AttnParams P) {
    using L = Layout<HD>;
    constexpr int STAGES = L::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* sQ = smem;
    uint8_t* sK = sQ + L::Q;
    uint8_t* sV = sK + STAGES * L::TILE;
    Smem& M = *reinterpret_cast<Smem*>(sV + STAGES * L::TILE);
    volatile int* abort_flag = &M.abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const DevErr derr{P.err.word, P.err.timeout_ns};

    Walk W;
    W.tiles = 0;
    if (!c8::line_start<TR, TK, NUM_THREADS>(P, M.scan, &M.start, W.at, W.stop, W.share, W.l, W.e, W.h, W.first)) return;
    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&M.k_full[i], 1);
            mbar_init(&M.k_empty[i], 1);
            mbar_init(&M.v_full[i], 1);
            mbar_init(&M.v_empty[i], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&M.s_full[b], 1);
            mbar_init(&M.p_full[b], SOFT);
            mbar_init(&M.pv_done[b], 1);
            mbar_init(&M.drain[b], 1);
        }
        mbar_init(&M.q_full, SOFT);
        M.abort = 0;
        fence_mbar_init();
    }
    if (warp == 5) {
        tmem_alloc(&M.tmem, TM_COLUMNS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = M.tmem;
    auto wait_all = [&](uint64_t* b, uint32_t parity) {  // warp-uniform outcome
        return __all_sync(0xffffffffu, mbar_wait(b, parity, derr, abort_flag)) != 0;
    };
    // t counts the tiles of all of the CTA's pieces: stage t % STAGES, score buffer t & 1
    uint32_t t = 0;
    Segment G;

    if (warp < 4) {
        // ------------------------------------------------------- softmax
        const int row = threadIdx.x;  // of the unit, and TMEM lane
        const uint32_t tl = tmem_base + (static_cast<uint32_t>(32 * warp) << 16);
        const float f = P.scale_log2;
        bool ok = true;
        while (W.next(P, G)) {
            const int ntiles = G.tiles();
            const bool valid = row < G.B.nrows, active = 32 * warp < G.B.nrows;
            const RowPlace at = place_of(P, G.B, G.h, valid ? row : 0);
            {
                const uint4* q = reinterpret_cast<const uint4*>(address<__nv_bfloat16>(P.query, G.l, at));
                uint4 u[HD / 8];
#pragma unroll
                for (int c = 0; c < HD / 8; ++c) u[c] = valid ? __ldg(q + c) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int c = 0; c < HD / 8; ++c)
                    *reinterpret_cast<uint4*>(sQ + (c >> 3) * L::Q_HALF + row * 128 + (((c & 7) ^ (row & 7)) << 4)) = u[c];
                fence_proxy_async_smem();
                mbar_arrive(&M.q_full);
            }
            const int see = valid ? min(G.k1, G.B.pos + (G.B.row0 + row) / P.g + 1) : 0;  // keys below are visible
            float m = LOWEST, sum = 0.f;
            for (int i = 0; i < ntiles; ++i, ++t) {
                const uint32_t b = t & 1, stage = t % STAGES;
                // V's barrier too: its stage, with what is noted of its pages, is not given away before P is there
                ok = ok && wait_all(&M.v_full[stage], (t / STAGES) & 1);
                ok = ok && wait_all(&M.s_full[b], (t >> 1) & 1);
                if (!ok) break;
                tc_fence_after();
                const int j0 = G.k0 + i * TK;
                const uint32_t present = M.present[stage];
                const bool ragged = present != (1u << GROUPS) - 1 || j0 + TK > G.k1;  // the same for all
                if (active) {
                    const uint32_t cS = tl + TM_S + TK * b;
                    uint32_t sv[TK];
                    tmem_ld32(cS, sv);
                    tmem_ld32(cS + 32, sv + 32);
                    const int nvis = see - j0;
                    tmem_ld_wait();
                    if (!__all_sync(0xffffffffu, !ragged && nvis >= TK)) {
#pragma unroll
                        for (int j = 0; j < TK; ++j)
                            if (j >= nvis || !((present >> (j / 16)) & 1u)) sv[j] = 0xff800000u;  // -inf
                    }
                    float top[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const uint32_t* v = sv + 16 * x;
                        float y[5];
#pragma unroll
                        for (int j = 0; j < 5; ++j)
                            y[j] = max3(__uint_as_float(v[3 * j]), __uint_as_float(v[3 * j + 1]), __uint_as_float(v[3 * j + 2]));
                        top[x] = fmaxf(max3(y[0], y[1], y[2]), max3(y[3], y[4], __uint_as_float(v[15])));
                    }
                    const float best = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * f;
                    const bool raise = best > m + MARGIN;
                    if (__any_sync(0xffffffffu, raise)) {
                        float lower = 1.f;
                        if (raise) {
                            lower = ex2(m - best);
                            sum *= lower;
                            m = best;
                        }
                        __syncwarp();
                        if (i > 0) {  // O is complete up to the tile before
                            ok = wait_all(&M.pv_done[b ^ 1], ((t - 1) >> 1) & 1);
                            if (ok) {
                                tc_fence_after();
#pragma unroll 1
                                for (int c0 = 0; c0 < HD; c0 += 16) {
                                    uint32_t o[16];
                                    tmem_ld16(tl + TM_O + c0, o);
                                    tmem_ld_wait();
#pragma unroll
                                    for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * lower);
                                    tmem_st16(tl + TM_O + c0, o);
                                }
                                tmem_st_wait();
                            }
                        }
                    }
                    // the weights, 32 keys at a time: high parts to columns 0 .. 31 of the buffer, low ones to 32 .. 63
                    const float2 f2 = make_float2(f, f), m2 = make_float2(-m, -m);
                    float2 part = make_float2(0.f, 0.f);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        uint32_t hi[16], lo[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            float2 w = fma2(make_float2(__uint_as_float(sv[32 * x + 2 * j]), __uint_as_float(sv[32 * x + 2 * j + 1])), f2, m2);
                            w = make_float2(ex2(w.x), ex2(w.y));
                            part = add2(part, w);
                            hi[j] = pack_bf16x2(w.x, w.y);
                            lo[j] = pack_bf16x2(w.x - __uint_as_float(hi[j] << 16), w.y - __uint_as_float(hi[j] & 0xffff0000u));
                        }
                        tmem_st16(cS + 16 * x, hi);
                        tmem_st16(cS + 32 + 16 * x, lo);
                    }
                    sum += part.x + part.y;
                    __syncwarp();
                    tmem_st_wait();
                    tc_fence_before();
                }
                if (ragged) {  // slots that nothing sees may hold anything: their value rows are zeros
                    for (int y = threadIdx.x; y < L::TILE / 16; y += SOFT) {
                        const int key = (y >> 3) % TK;
                        if (j0 + key >= G.k1 || !((present >> (key / 16)) & 1u))
                            *reinterpret_cast<uint4*>(sV + stage * L::TILE + 16 * y) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                }
                mbar_arrive(&M.p_full[b]);
            }
            if (ok && ntiles > 0) ok = wait_all(&M.pv_done[(t - 1) & 1], ((t - 1) >> 1) & 1);
            const bool have = ok && ntiles > 0 && active;
            if (have) tc_fence_after();
            const int64_t part0 = G.slot * TR + row;
            const float by = sum == 0.f ? 0.f : 1.f / sum;
            const int64_t lse_row = (static_cast<int64_t>(G.l) * P.c.H * P.g + at.head) * P.q.T + at.token;
            const bool write = valid && KVB_IN_BOUNDS(P.err, lse_row, 1, c8::rows_of(P));
            if (active) {
#pragma unroll 1
                for (int c0 = 0; c0 < HD; c0 += 16) {
                    uint32_t o[16];
                    if (have) {
                        tmem_ld16(tl + TM_O + c0, o);
                        tmem_ld_wait();
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j) o[j] = 0u;
                    }
                    if (write && G.pieces.n == 1) {
                        uint32_t w[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) w[j] = pack_bf16x2(__uint_as_float(o[2 * j]) * by, __uint_as_float(o[2 * j + 1]) * by);
                        uint4* dst = reinterpret_cast<uint4*>(address<__nv_bfloat16>(P.out, G.l, at) + c0);
                        dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
                        dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
                    } else if (write && KVB_IN_BOUNDS(P.err, part0, 1, P.slots * TR)) {
                        uint4* dst = reinterpret_cast<uint4*>(P.partial + part0 * HD + c0);
#pragma unroll
                        for (int j = 0; j < 4; ++j) dst[j] = make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                    }
                    __syncwarp();
                }
                if (write && G.pieces.n == 1) {
                    if (P.lse) P.lse[lse_row] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.693147180559945f;
                } else if (write && KVB_IN_BOUNDS(P.err, part0, 1, P.slots * TR)) {
                    P.part_stat[part0] = make_float2(m, sum);
                }
                tc_fence_before();
            }
            if (G.pieces.n > 1)
                join_pieces<__nv_bfloat16, HD, TR, SOFT>(P, G.B, G.pieces, G.unit, G.l, G.h, &M.last, M.join, 2 * TR,
                                                         [] { named_bar_sync(1, SOFT); });
        }
    } else if (warp == 4) {
        // ------------------------------------------------------- pages and loads
        const int rows = min(P.c.page, TK), per = TK / rows;  // keys of a load; loads of a tile
        bool go = true;
        while (go && W.next(P, G)) {
            const int ntiles = G.tiles();
            const int64_t block0 = (static_cast<int64_t>(P.c.l_begin) + G.l) * P.c.n_pages * P.c.H + G.h;
            const int loads = (G.k1 - G.k0 + rows - 1) / rows;
            auto page_of = [&](int x0) {  // of load x0 + lane
                const int x = x0 + lane;
                if (x >= loads) return -1;
                const int p = (G.k0 + x * rows) >> P.c.page_log2;
                int pid = p < P.q.max_pages && c8::table_in_bounds(P.q, P.err, G.s, p)
                              ? __ldg(P.q.page_table + static_cast<int64_t>(G.s) * P.q.max_pages + p) : -1;
                if (pid < 0 || pid >= P.c.n_pages) {
                    c8::err_set(P.err, DEV_ERR_BAD_SEQ);
                    pid = -1;
                }
                const int64_t blocks = (static_cast<int64_t>(P.c.l_begin) + P.c.n_layers) * P.c.n_pages * P.c.H;
                if (pid >= 0 && !KVB_IN_BOUNDS(P.err, block0 + static_cast<int64_t>(pid) * P.c.H, 1, blocks)) pid = -1;
                return pid;
            };
            int now = page_of(0), next = page_of(32);
            for (int i = 0; i < ntiles; ++i, ++t) {
                const uint32_t stage = t % STAGES, round = t / STAGES;
                const int x0 = i * per;
                if (x0 > 0 && (x0 & 31) == 0) {
                    now = next;
                    next = page_of(x0 + 32);
                }
                int z[GROUPS];  // blocks of the tile's loads, -1: none
                uint32_t present = 0;
#pragma unroll
                for (int x = 0; x < GROUPS; ++x) {
                    const int pid = __shfl_sync(0xffffffffu, now, (x0 + x) & 31);
                    z[x] = x < per && pid >= 0 ? static_cast<int>(block0 + static_cast<int64_t>(pid) * P.c.H) : -1;
                    if (z[x] >= 0) present |= ((1u << (rows / 16)) - 1) << (x * (rows / 16));
                }
                const uint32_t bytes = static_cast<uint32_t>(__popc(present)) * 16 * HD * 2;
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    uint64_t* full = kv ? &M.v_full[stage] : &M.k_full[stage];
                    if (go) go = wait_all(kv ? &M.v_empty[stage] : &M.k_empty[stage], (round & 1) ^ 1);
                    if (!go) break;
                    if (lane == 0) {
                        if (kv) M.present[stage] = present;
                        if (bytes) mbar_arrive_expect_tx(full, bytes);
                        else mbar_arrive(full);
                        uint8_t* tile = (kv ? sV : sK) + stage * L::TILE;
#pragma unroll
                        for (int x = 0; x < GROUPS; ++x)
                            if (z[x] >= 0)
#pragma unroll
                                for (int hf = 0; hf < HD / 64; ++hf)
                                    tma_load_3d(tile + hf * L::HALF + x * rows * 128, &maps.kv[kv], full, 64 * hf,
                                                (G.k0 + (x0 + x) * rows) & (P.c.page - 1), z[x]);
                    }
                    __syncwarp();
                }
                if (!go) break;
            }
        }
        if (!go) {  // what was asked for arrives before the CTA ends (k of tile t may have been)
            for (uint32_t u = t >= STAGES ? t - STAGES : 0; u <= t; ++u) {
                const uint32_t stage = u % STAGES, parity = (u / STAGES) & 1;
                mbar_wait_drain(&M.k_full[stage], parity, DRAIN_NS / 16);
                mbar_wait_drain(&M.v_full[stage], parity, DRAIN_NS / 16);
            }
        }
    } else {
        // ------------------------------------------------------- products
        const bool scores = warp == 5;
        bool go = true;
        const uint64_t q0 = sdesc_k_sw128(smem_u32(sQ)), k0 = sdesc_k_sw128(smem_u32(sK));
        const uint64_t v0 = sdesc_mn_sw128(smem_u32(sV), L::HALF);
        for (int n = 0; go && W.next(P, G); ++n) {
            const int ntiles = G.tiles();
            if (scores && ntiles > 0) {
                // A limit of 0 leaves no time to wait: a timeout, whatever the wait would have found.
                if (derr.timeout_ns == 0) {
                    dev_err_set(derr, DEV_ERR_TIMEOUT);
                    *abort_flag = 1;
                    go = false;
                }
                go = go && wait_all(&M.q_full, n & 1);
            }
            for (int i = 0; go && i < ntiles; ++i, ++t) {
                const uint32_t b = t & 1, stage = t % STAGES, parity = (t / STAGES) & 1;
                const uint32_t cS = tmem_base + TM_S + TK * b;
                if (scores) {
                    constexpr uint32_t idesc = idesc_bf16_f32(TR, TK);
                    go = wait_all(&M.k_full[stage], parity);
                    if (go && t >= 2) go = wait_all(&M.pv_done[b], ((t >> 1) - 1) & 1);  // P lies where these scores go
                    if (!go) break;
                    tc_fence_after();
                    const uint64_t k = k0 + stage * L::TILE / 16;
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < HD / 16; ++kk)
                            umma_bf16(cS, q0 + ((kk >> 2) * L::Q_HALF + (kk & 3) * 32) / 16, k + ((kk >> 2) * L::HALF + (kk & 3) * 32) / 16,
                                      idesc, kk != 0);
                        umma_commit(&M.s_full[b]);
                        umma_commit(&M.k_empty[stage]);
                    }
                } else {
                    constexpr uint32_t idesc = idesc_bf16_f32(TR, HD) | IDESC_B_MN;
                    go = wait_all(&M.v_full[stage], parity);
                    go = go && wait_all(&M.p_full[b], (t >> 1) & 1);
                    if (!go) break;
                    tc_fence_after();
                    const uint64_t v = v0 + stage * L::TILE / 16;
                    if (elect_one()) {
#pragma unroll
                        for (int part = 0; part < 2; ++part)
#pragma unroll
                            for (int kk = 0; kk < TK / 16; ++kk)
                                umma_f16_ts(tmem_base + TM_O, cS + 32u * part + 8u * kk, v + kk * 16 * 128 / 16, idesc, (i | part | kk) != 0);
                        umma_commit(&M.v_empty[stage]);
                        umma_commit(&M.pv_done[b]);
                    }
                }
                __syncwarp();
            }
            __syncwarp();
        }
        if (elect_one()) {
            umma_commit(&M.drain[scores ? 0 : 1]);  // every product issued here completes before TMEM is released
            mbar_wait_drain(&M.drain[scores ? 0 : 1], 0, DRAIN_NS);
        }
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 5) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem_base, TM_COLUMNS);
    }
    if (threadIdx.x == 0 && *abort_flag) *reinterpret_cast<volatile int*>(P.err.mirror) = DEV_ERR_TIMEOUT;
}

template <int HD>
cudaError_t launch(const AttnParams& P, const AttnPlan& p, cudaStream_t s, std::string* why) {
    EncodeTiledFn enc = get_encode_tiled();
    if (!enc) {
        *why = "cuTensorMapEncodeTiled unavailable from the driver";
        return cudaErrorInvalidValue;
    }
    Maps maps;
    const cuuint64_t page = static_cast<cuuint64_t>(P.c.page);
    // the layers up to the call's last are named, and a call reads no other
    const cuuint64_t dims[3] = {HD, page, (static_cast<cuuint64_t>(P.c.l_begin) + P.c.n_layers) * P.c.n_pages * P.c.H};
    const cuuint64_t strides[2] = {HD * 2, page * HD * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(P.c.page < TK ? P.c.page : TK), 1}, ones[3] = {1, 1, 1};
    for (int kv = 0; kv < 2; ++kv) {
        const CUresult r = enc(&maps.kv[kv], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, P.c.kv[kv], dims, strides, box, ones,
                               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
        if (r != CUDA_SUCCESS) {
            *why = "cuTensorMapEncodeTiled failed with code " + std::to_string(static_cast<int>(r));
            return cudaErrorInvalidValue;
        }
    }
    cudaError_t e = cudaFuncSetAttribute(rows_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<HD>::BYTES);
    if (e != cudaSuccess) return e;
    rows_kernel<HD><<<p.ctas, NUM_THREADS, Layout<HD>::BYTES, s>>>(maps, P);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attention_rows(const AttnParams& P, const AttnPlan& p, cudaStream_t s, std::string* why) {
    return P.c.d == 64 ? launch<64>(P, p, s, why) : launch<128>(P, p, s, why);
}

}  // namespace paged
}  // namespace kvb
