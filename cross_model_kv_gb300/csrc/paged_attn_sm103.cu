// Attention over the paged cache on the 5th-generation tensor cores: more query rows than
// mma.sync keeps up with (drafted tokens being checked), bf16, head_dim 64 and 128.
//
// The mathematics and the references are those of paged_attn.cu.  A CTA an SM takes NR (up to 64)
// rows of a unit (layer, sequence, row block, head) and walks its keys 128 at a time; the 128-key
// tiles of all units form one line that the CTAs share evenly.  The keys are the M rows of the
// products and the query rows N, so that few rows cost little:
//   S^T = K Q^T     M = 128 keys, N = NR rows;
//   O^T += V^T P^T  M = the dims, K = 128 keys, N = NR rows twice: P as a bf16 pair (hi, lo), the two
//                   parts' outputs side by side, added at the end.
// (Query rows as M, 128 of them whatever their number, 64 keys a tile: 122 us for 16 sequences of
// 8192 keys, 8 heads, 32 rows each, 1860 cycles a tile, of which HBM takes 1400; the products' warps
// took 900 to 1000 cycles to issue eight of 128 x 64 x 16 or 128 x 128 x 16.)
//   warps 0..3, 4..7  softmax of every other piece of a unit (64 rows: one set, of every piece), a key a
//               thread: scores from TMEM to registers, the weights of its key to shared memory, every row's sum in registers until the
//               piece ends.  No thread knows a row's maximum: they vote whether some score passes its
//               reference by 2^8, and only then reduce, and rescale O in TMEM.  They load the rows and write
//               the outputs while the other four warps are in the next piece;
//   warp 8      page numbers, and TMA loads of K and V into rings of tiles, 128-byte swizzle, key
//               rows: K-major for S, MN-major for O, as they lie in the pages;
//   warp 9      one lane issues S^T = K Q^T;
//   warp 10     and O^T += V^T P^T.
// At head_dim 64 O^T has 64 rows and M is 128 all the same: the upper 64 are the lower ones again.
// TMEM: score buffer b at 64 b, O's high part at 128 (and 256, odd pieces), its low part NR columns on.
// HBM bounds it where keys are many (16 sequences of 1024 to 8192 keys, 8 heads, 40 rows: 63 us, 0.66 of the copy rate; of
// 8192 each 97 us, 0.82); a unit's chain of hand-overs, 5 to 12 us of which two units overlap, where they are few.
// Every role finds the CTA's pieces by itself, so that the rings are filled while the softmax goes from one
// unit to the next.  A second kernel joins the units that several CTAs share.
// Every wait is bounded; after one gives up, the loads and products that were issued are waited for, TMEM is
// freed, and what the call still writes is marked as wrong by its status.
#include "kvb_host.h"
#include "paged_attn.cuh"

namespace kvb {
namespace paged {

namespace {

constexpr int TK = 128;          // keys of a tile, TMEM lanes
constexpr int SOFT = 128;        // threads of the softmax of a piece
// Two sets of softmax warps where their registers suffice: 64 rows take more than 200 a thread (16 x 8192 keys:
// 99 us with one set, 121 with two; 40 rows, 16 x 1024..8192 keys: 73 and 63.5).
constexpr int sets_of(int NR) { return NR <= 48 ? 2 : 1; }
constexpr int threads_of(int NR) { return sets_of(NR) * SOFT + 128; }  // the last warp only makes up a warpgroup
// Registers a thread: 168 at launch, then by role.  256 * 192 + 128 * 96 = 61440 of the launch's 384 * 168 = 64512.
constexpr int REGS_SOFTMAX = 192, REGS_OTHERS = 96;
constexpr int GROUPS = TK / 16;  // 16 keys lie in one page
constexpr int ATOM = TK * 128;   // 64 dims of a tile's keys, or 64 rows' weights of them
constexpr uint32_t TM_S = 0, TM_O = 128, TM_COLUMNS = 512;
constexpr uint64_t DRAIN_NS = 200ull * 1000 * 1000;
constexpr uint32_t IDESC_A_MN = 1u << 15;  // A operand MN-major

// What the softmax of even, or of odd, pieces notes.
struct Rows {
    alignas(16) float ref[64];       // of every row
    alignas(16) float by[64];        // factors of a raise; 1 / sum of a piece
    alignas(16) float part[4][64];   // of a warp
    int pos[64];                     // positions of the rows
    int odd;                         // values that are not finite have been taken out of the products
    int64_t to[64];                  // element of P.out that their outputs begin at
};
struct Smem {
    uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
    uint64_t s_full[2], s_empty[2], p_full[2], pv_done[2], q_full[2], o_full[2], handed[2], drain[2];
    uint32_t tmem;
    int abort;
    // bit of a tile's 16-key group whose page is there; a tile's place is written again 8 tiles later, when
    // at most four tiles are behind the one that is loaded
    uint64_t info_full[8];
    uint32_t present[8];
    int scan[12];
    LineStart start;
    Rows rows[2];
};

template <int HD, int NR>
struct Layout {
    static constexpr int Q_HALF = NR * 128, Q = HD / 64 * Q_HALF;  // 64 dims of all rows
    static constexpr int TILE = HD / 64 * ATOM;                    // of K, and of V
    static constexpr int STAGES = HD == 128 ? 2 : 4;
    static constexpr int WEIGHTS = (2 * NR + 63) / 64 * ATOM;      // a buffer of two
    static constexpr int SETS = sets_of(NR);
    static constexpr int BYTES = 1024 + STAGES * 2 * TILE + 2 * WEIGHTS + SETS * Q + sizeof(Smem);  // rows of every set
    static_assert(Q % 1024 == 0, "layout");
    static_assert(BYTES <= 227 * 1024, "layout");
};

// A piece of a unit.
struct Segment {
    RowBlock B;
    int s, l, h;
    int k0, k1;  // keys [k0, k1)
    int64_t slot;
    Pieces pieces;
    // One at least: of a unit without keys a tile that nothing sees.  Every piece passes every barrier of the
    // roles then, so that none gets two phases ahead of a wait.
    __device__ __forceinline__ int tiles() const { return max(1, (k1 - k0 + TK - 1) / TK); }
};

// The CTA's place in the line of tiles.
template <int NR>
struct Walk {
    static constexpr int UNIT_TILES = unit_tiles_of(NR);
    int at, stop, share, l, e, h, first;
    RowBlock B;
    int tiles;  // of unit (l, e, h), UNIT_TILES without keys first; 0 before the first

    __device__ __forceinline__ RowBlock entry(const AttnParams& P) const {
        return c8::row_block(P, e / P.row_blocks, e % P.row_blocks, NR);
    }
    // The next piece with keys, if there is one.
    __device__ __forceinline__ bool next(const AttnParams& P, Segment& g) {
        const int entries = P.q.n_seq * P.row_blocks;
        for (;;) {
            if (at >= stop) return false;
            if (tiles == 0) {
                B = entry(P);
                tiles = c8::unit_tiles<TK, UNIT_TILES>(B);
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
                        tiles = c8::unit_tiles<TK, UNIT_TILES>(B);
                    } while (tiles == 0);
                }
            }
            const int last = min(tiles, first + (stop - at));
            const int u0 = at - first, c0 = (u0 + UNIT_TILES) / share;  // the CTA of its first keys
            at += last - first;
            if (last <= UNIT_TILES) continue;
            g.B = B;
            g.s = e / P.row_blocks;
            g.l = l;
            g.h = h;
            g.k0 = max(first - UNIT_TILES, 0) * TK;
            g.k1 = max(g.k0, min(B.kv_end, (last - UNIT_TILES) * TK));
            g.pieces = Pieces{(u0 + tiles - 1) / share - c0 + 1, c0};
            g.slot = 2 * static_cast<int64_t>(blockIdx.x) + (first <= UNIT_TILES);
            return true;
        }
    }
};

struct Maps {
    CUtensorMap kv[2];
};

// The 64-dim halves (or single half) of an operand of 128-byte rows, K-major: step kk of 16 dims.
template <int HALF>
__device__ __forceinline__ constexpr uint32_t step_k(int kk) {
    return ((kk >> 2) * HALF + (kk & 3) * 32) / 16;
}

__device__ __forceinline__ float warp_max(float x) {  // NaN loses
    float y;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}

template <int HD, int NR>
__global__ void __launch_bounds__(threads_of(NR), 1) rows_kernel(const __grid_constant__ Maps maps, const __grid_constant__ AttnParams P) {
    using L = Layout<HD, NR>;
    constexpr int STAGES = L::STAGES, SETS = L::SETS, NUM_THREADS = threads_of(NR);
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* sK = smem;
    uint8_t* sV = sK + STAGES * L::TILE;
    uint8_t* sP = sV + STAGES * L::TILE;
    uint8_t* sQ = sP + 2 * L::WEIGHTS;
    Smem& M = *reinterpret_cast<Smem*>(sQ + SETS * L::Q);
    volatile int* abort_flag = &M.abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const DevErr derr{P.err.word, P.err.timeout_ns};

    Walk<NR> W;
    W.tiles = 0;
    if (threadIdx.x == 0 && KVB_IN_BOUNDS(P.err, 2 * static_cast<int64_t>(blockIdx.x), 1, P.slots))
        P.shared[2 * blockIdx.x] = make_int4(0, 0, 0, 0);  // (until it is known, after a barrier)
    if (!c8::line_start<NR, TK, NUM_THREADS, Walk<NR>::UNIT_TILES, 4>(P, M.scan, &M.start, W.at, W.stop, W.share, W.l, W.e, W.h, W.first)) return;
    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&M.k_full[i], 1);
            mbar_init(&M.k_empty[i], 1);
            mbar_init(&M.v_full[i], 1);
            mbar_init(&M.v_empty[i], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&M.s_full[b], 1);
            mbar_init(&M.s_empty[b], SOFT);
            mbar_init(&M.p_full[b], SOFT);
            mbar_init(&M.pv_done[b], 1);
            mbar_init(&M.drain[b], 1);
            mbar_init(&M.q_full[b], SOFT);
            mbar_init(&M.o_full[b], 1);
            mbar_init(&M.handed[b], SOFT);
        }
        for (int i = 0; i < 8; ++i) mbar_init(&M.info_full[i], 1);
        M.abort = 0;
        fence_mbar_init();
    }
    if (warp == 4 * SETS + 1) {
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
    // t counts the tiles of all of the CTA's pieces: stage t % STAGES, scores and weights t & 1
    uint32_t t = 0;
    Segment G;

    if (warp < 4 * SETS) {
        // ------------------------------------------------------- softmax
        if constexpr (SETS == 2) regs_up<REGS_SOFTMAX>();
        const int half = warp / 4, w4 = warp & 3;  // even or odd pieces; warp of the set
        const int key = threadIdx.x % SOFT;        // of the tile, and TMEM lane; the dim of an output
        const uint32_t tl = tmem_base + (static_cast<uint32_t>(32 * w4) << 16);
        const uint32_t tO = tl + TM_O + 128u * half;
        uint8_t* const myQ = sQ + half * L::Q;
        Rows& N = M.rows[half];
        const int id = 1 + half;  // of the barrier
        const float f = P.scale_log2;
        bool ok = true;
        for (int piece = 0; W.next(P, G); ++piece) {
            const int ntiles = G.tiles();
            if (piece % SETS != half) {
                t += ntiles;
                continue;
            }
            named_bar_sync(id, SOFT);  // ref, pos and by are free
            // the rows: 16-byte chunks c of row r, by all threads
            {
                constexpr int MINE = NR * (HD / 8) / SOFT;
                uint4 u[MINE];
#pragma unroll
                for (int i = 0; i < MINE; ++i) {
                    const int r = (i * SOFT + key) / (HD / 8), c = key % (HD / 8);
                    u[i] = r < G.B.nrows ? __ldg(reinterpret_cast<const uint4*>(address<__nv_bfloat16>(P.query, G.l, place_of(P, G.B, G.h, r))) + c)
                                         : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int i = 0; i < MINE; ++i) {
                    const int r = (i * SOFT + key) / (HD / 8), c = key % (HD / 8);
                    *reinterpret_cast<uint4*>(myQ + (c >> 3) * L::Q_HALF + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = u[i];
                }
            }
            if (key == 0) N.odd = 0;
            if (key < NR) {
                N.ref[key] = key < G.B.nrows ? LOWEST : 0.f;  // rows that do not exist: weights of 1, never raised
                N.pos[key] = key < G.B.nrows ? G.B.pos + (G.B.row0 + key) / P.g : INT32_MAX - 1;
            }
            fence_proxy_async_smem();
            mbar_arrive(&M.q_full[half]);
            float sum[NR];
#pragma unroll
            for (int n = 0; n < NR; ++n) sum[n] = 0.f;
            named_bar_sync(id, SOFT);
            // The piece before has its last weights: a wait for a phase of a barrier is only right when the
            // phase before it is over, and those of the tiles are waited for by one set of warps after the other.
            if (SETS == 2 && piece > 0) ok = ok && wait_all(&M.handed[half ^ 1], ((piece - 1) >> 1) & 1);
            for (int i = 0; i < ntiles; ++i, ++t) {
                const uint32_t b = t & 1, use = t >> 1, stage = t % STAGES;
                ok = ok && wait_all(&M.info_full[t % 8], (t / 8) & 1);
                ok = ok && wait_all(&M.s_full[b], use & 1);
                const int j = G.k0 + i * TK + key;
                uint32_t sv[NR];
                bool above = false, special = false;  // special: not every row sees the key
                auto dead = [&] { return j >= G.k1 || !((M.present[t % 8] >> (key / 16)) & 1u); };  // nothing sees it
                if (ok) {
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < NR; c += 16) tmem_ld16(tl + TM_S + 64 * b + c, *reinterpret_cast<uint32_t(*)[16]>(sv + c));
                    special = dead() || j > G.B.pos_lo;
                    tmem_ld_wait();
                    tc_fence_before();
                    mbar_arrive(&M.s_empty[b]);
                    if (__any_sync(0xffffffffu, special)) {
                        const int from = dead() ? INT32_MAX : j;
#pragma unroll
                        for (int n = 0; n < NR; ++n)
                            if (from > N.pos[n]) sv[n] = 0xff800000u;  // -inf
                    }
                    float top = -INFINITY;
#pragma unroll
                    for (int n = 0; n < NR; n += 4) {
                        const float4 r = *reinterpret_cast<const float4*>(N.ref + n);
                        top = max3(top, fmaf(__uint_as_float(sv[n]), f, -r.x), fmaf(__uint_as_float(sv[n + 1]), f, -r.y));
                        top = max3(top, fmaf(__uint_as_float(sv[n + 2]), f, -r.z), fmaf(__uint_as_float(sv[n + 3]), f, -r.w));
                    }
                    above = top > MARGIN;
                }
                if (!named_bar_and(id, SOFT, ok && !above)) {
                    ok = named_bar_and(id, SOFT, ok);
                    if (!ok) break;
                    // some score passes its reference: every row's is raised to the tile's maximum
#pragma unroll
                    for (int n = 0; n < NR; ++n) {
                        const float x = warp_max(__uint_as_float(sv[n]));
                        if (lane == 0) N.part[w4][n] = x;
                    }
                    named_bar_sync(id, SOFT);
                    if (key < NR) {
                        const float x = fmaxf(fmaxf(N.part[0][key], N.part[1][key]), fmaxf(N.part[2][key], N.part[3][key]));
                        const float old = N.ref[key], up = fmaxf(old, x * f);
                        N.by[key] = ex2(old - up);
                        N.ref[key] = up;
                    }
                    named_bar_sync(id, SOFT);
#pragma unroll
                    for (int n = 0; n < NR; ++n) sum[n] *= N.by[n];
                    if (i > 0) {  // O is complete up to the tile before
                        ok = wait_all(&M.pv_done[b ^ 1], ((t - 1) >> 1) & 1);
                        if (ok) {
                            tc_fence_after();
#pragma unroll 1
                            for (int c = 0; c < 2 * NR; c += 16) {
                                uint32_t o[16];
                                tmem_ld16(tO + c, o);
                                tmem_ld_wait();
#pragma unroll
                                for (int n = 0; n < 16; ++n) o[n] = __float_as_uint(__uint_as_float(o[n]) * N.by[(c + n) % NR]);
                                tmem_st16(tO + c, o);
                            }
                            tmem_st_wait();
                            tc_fence_before();
                        }
                    }
                }
                // the weights' buffer is free when its products are done
                if (ok && use > 0) ok = wait_all(&M.pv_done[b], (use - 1) & 1);
                if (ok && __any_sync(0xffffffffu, special)) ok = wait_all(&M.v_full[stage], (t / STAGES) & 1);
                if (!ok) continue;  // to the next vote
                uint8_t* mine = sP + b * L::WEIGHTS + key * 128;
#pragma unroll
                for (int c = 0; c < NR / 8; ++c) {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const int r = 8 * c + 2 * n;
                        const float2 ref = *reinterpret_cast<const float2*>(N.ref + r);
                        const float2 w = make_float2(ex2(fmaf(__uint_as_float(sv[r]), f, -ref.x)), ex2(fmaf(__uint_as_float(sv[r + 1]), f, -ref.y)));
                        sum[r] += w.x;
                        sum[r + 1] += w.y;
                        hi[n] = pack_bf16x2(w.x, w.y);
                        lo[n] = pack_bf16x2(w.x - __uint_as_float(hi[n] << 16), w.y - __uint_as_float(hi[n] & 0xffff0000u));
                    }
                    constexpr int LO = NR / 8;
                    *reinterpret_cast<uint4*>(mine + (c >> 3) * ATOM + (((c & 7) ^ (key & 7)) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4*>(mine + ((LO + c) >> 3) * ATOM + ((((LO + c) & 7) ^ (key & 7)) << 4)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
                if (special) {  // slots that nothing sees may hold anything: their value rows are zeros
                    uint4* row = reinterpret_cast<uint4*>(sV + stage * L::TILE + key * 128);
                    const bool none = dead();
#pragma unroll 4
                    for (int c = 0; c < HD / 8; ++c) {
                        uint4& v = row[(c >> 3) * (ATOM / 16) + (c & 7)];
                        if (none) v = make_uint4(0, 0, 0, 0);
                        else if (make_finite<__nv_bfloat16>(v)) N.odd = 1;
                    }
                }
                fence_proxy_async_smem();
                mbar_arrive(&M.p_full[b]);
            }
            if (SETS == 2) mbar_arrive(&M.handed[half]);
            // (a barrier of its own: those of the tiles go on with the next piece)
            ok = ok && wait_all(&M.o_full[half], (piece / SETS) & 1);
            if (ok) tc_fence_after();
            // the rows' sums, and where their outputs go
#pragma unroll
            for (int n0 = 0; n0 < NR; n0 += 16) {  // 16 rows: a lane keeps half of them at each exchange
                float x[16];
#pragma unroll
                for (int n = 0; n < 16; ++n) x[n] = sum[n0 + n];
#pragma unroll
                for (int z = 8; z > 0; z >>= 1)
#pragma unroll
                    for (int n = 0; n < z; ++n) {
                        const float keep = lane & z ? x[n + z] : x[n], give = lane & z ? x[n] : x[n + z];
                        x[n] = keep + __shfl_xor_sync(0xffffffffu, give, z);
                    }
                x[0] += __shfl_xor_sync(0xffffffffu, x[0], 16);
                if (lane < 16) N.part[w4][n0 + lane] = x[0];
            }
            named_bar_sync(id, SOFT);
            const bool alone = G.pieces.n == 1;
            const int64_t part0 = G.slot * NR;
            if (key < NR && key >= G.B.nrows) N.to[key] = -1;
            if (key < G.B.nrows) {
                const float total = ok ? (N.part[0][key] + N.part[1][key]) + (N.part[2][key] + N.part[3][key]) : 0.f, m = N.ref[key];
                const RowPlace at = place_of(P, G.B, G.h, key);
                const int64_t lse_row = (static_cast<int64_t>(G.l) * P.c.H * P.g + at.head) * P.q.T + at.token;
                const bool inside = KVB_IN_BOUNDS(P.err, lse_row, 1, c8::rows_of(P)) && KVB_IN_BOUNDS(P.err, G.slot, 1, P.slots);
                N.by[key] = total == 0.f ? 0.f : 1.f / total;
                N.to[key] = inside ? G.l * P.out.l + at.head * P.out.h + at.token * P.out.t : -1;
                if (inside && !alone) P.part_stat[part0 + key] = make_float2(m, total);
                if (inside && alone && P.lse) P.lse[lse_row] = total == 0.f ? -INFINITY : (m + log2f(total)) * 0.693147180559945f;
            }
            named_bar_sync(id, SOFT);
            if (key < HD && (alone || KVB_IN_BOUNDS(P.err, G.slot, 1, P.slots))) {  // whole warps; lane = dim
#pragma unroll 1
                for (int c = 0; c < G.B.nrows; c += 16) {
                    uint32_t hi[16], lo[16];
                    if (ok) {
                        tmem_ld16(tO + c, hi);
                        tmem_ld16(tO + NR + c, lo);
                        tmem_ld_wait();
                    } else {
#pragma unroll
                        for (int n = 0; n < 16; ++n) hi[n] = lo[n] = 0u;
                    }
                    float o[16];
#pragma unroll
                    for (int n = 0; n < 16; ++n) o[n] = __uint_as_float(hi[n]) + __uint_as_float(lo[n]);
                    if (ok && N.odd) {
#pragma unroll 1
                        for (int j = max(G.k0, G.B.pos_lo + 1); j < G.k1; ++j) {
                            const float v = value_of<__nv_bfloat16>(P, G.s, G.l, G.h, j, key);
                            if (not_finite(v))
#pragma unroll
                                for (int n = 0; n < 16; ++n)
                                    if (j <= N.pos[c + n]) o[n] += v;
                        }
                    }
                    if (alone) {
                        int64_t to[16];
                        float by[16];
#pragma unroll
                        for (int n = 0; n < 16; ++n) {
                            to[n] = N.to[c + n];
                            by[n] = N.by[c + n];
                        }
#pragma unroll
                        for (int n = 0; n < 16; ++n)
                            if (to[n] >= 0) static_cast<__nv_bfloat16*>(P.out.data)[to[n] + key] = __float2bfloat16_rn(by[n] == 0.f ? 0.f : o[n] * by[n]);
                    } else {
                        float* to = P.partial + (part0 + c) * HD + key;
#pragma unroll
                        for (int n = 0; n < 16; ++n)
                            if (c + n < G.B.nrows) to[n * HD] = o[n];
                    }
                    __syncwarp();
                }
            }
            tc_fence_before();
            if (key == 0 && !alone && G.k0 == 0 && KVB_IN_BOUNDS(P.err, G.slot, 1, P.slots)) {  // at most one of a CTA's pieces
                P.shared[2 * blockIdx.x + 1] = make_int4(G.l, G.h, 0, 0);
                P.shared[2 * blockIdx.x] = make_int4(G.pieces.n, G.B.nrows, G.B.row0, G.B.tok0);
            }
        }
    } else if (warp == 4 * SETS) {
        // ------------------------------------------------------- pages and loads
        if constexpr (SETS == 2) regs_down<REGS_OTHERS>();
        constexpr int HALVES = HD / 64;
        const int rows = min(P.c.page, TK), per = TK / rows;  // keys of a load; loads of a tile, of 64 dims
        bool go = true;
        uint32_t asked[2] = {0, 0};  // tiles of K, and of V, whose barrier has been armed
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
                // lane x * HALVES + hf issues load x of 64 dims: one lane after another took 1300 cycles for K,
                // the whole of a tile's loads 2600 of the 2700 that HBM takes for it
                const int x = lane / HALVES, hf = lane % HALVES;
                const int pid = __shfl_sync(0xffffffffu, now, (x0 + x) & 31), group_pid = __shfl_sync(0xffffffffu, now, (x0 + lane * 16 / rows) & 31);
                const uint32_t present = __ballot_sync(0xffffffffu, lane < GROUPS && group_pid >= 0);
                const bool mine = x < per && pid >= 0;
                const int z = static_cast<int>(block0 + static_cast<int64_t>(max(pid, 0)) * P.c.H), y = (G.k0 + (x0 + x) * rows) & (P.c.page - 1);
                const uint32_t bytes = static_cast<uint32_t>(__popc(present)) * 16 * HD * 2;
                if (elect_one()) {
                    M.present[t % 8] = present;
                    mbar_arrive(&M.info_full[t % 8]);
                }
                __syncwarp();
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    uint64_t* full = kv ? &M.v_full[stage] : &M.k_full[stage];
                    if (go) go = wait_all(kv ? &M.v_empty[stage] : &M.k_empty[stage], (round & 1) ^ 1);
                    if (!go) break;
                    asked[kv] = t + 1;
                    if (elect_one()) {
                        if (bytes) mbar_arrive_expect_tx(full, bytes);
                        else mbar_arrive(full);
                    }
                    __syncwarp();
                    if (mine) tma_load_3d((kv ? sV : sK) + stage * L::TILE + hf * ATOM + x * rows * 128, &maps.kv[kv], full, 64 * hf, y, z);
                    __syncwarp();
                }
                if (!go) break;
            }
        }
        // What was asked for arrives before the CTA ends, also where the other roles gave up before they looked at it
        // and no wait of this warp did: the first STAGES tiles find their places empty.
#pragma unroll
        for (int kv = 0; kv < 2; ++kv)
            for (uint32_t u = asked[kv] > STAGES ? asked[kv] - STAGES : 0; u < asked[kv]; ++u)
                mbar_wait_drain(kv ? &M.v_full[u % STAGES] : &M.k_full[u % STAGES], (u / STAGES) & 1, DRAIN_NS);
    } else if (warp == 4 * SETS + 3) {
        if constexpr (SETS == 2) regs_down<REGS_OTHERS>();
    } else {
        // ------------------------------------------------------- products
        if constexpr (SETS == 2) regs_down<REGS_OTHERS>();
        const bool scores = warp == 4 * SETS + 1;
        bool go = true;
        const uint64_t k0 = sdesc_k_sw128(smem_u32(sK)), q0 = sdesc_k_sw128(smem_u32(sQ));
        const uint64_t v0 = sdesc_mn_sw128(smem_u32(sV), HD == 128 ? ATOM : 0), p0 = sdesc_mn_sw128(smem_u32(sP), ATOM);
        for (int n = 0; go && W.next(P, G); ++n) {
            const int ntiles = G.tiles();
            if (scores) {
                // A limit of 0 leaves no time to wait: a timeout, whatever the wait would have found.
                if (derr.timeout_ns == 0) {
                    dev_err_set(derr, DEV_ERR_TIMEOUT);
                    *abort_flag = 1;
                    go = false;
                }
                go = go && wait_all(&M.q_full[n % SETS], (n / SETS) & 1);
            }
            for (int i = 0; go && i < ntiles; ++i, ++t) {
                const uint32_t b = t & 1, use = t >> 1, stage = t % STAGES, parity = (t / STAGES) & 1;
                if (scores) {
                    constexpr uint32_t idesc = idesc_bf16_f32(TK, NR);
                    go = wait_all(&M.k_full[stage], parity);
                    if (go && use > 0) go = wait_all(&M.s_empty[b], (use - 1) & 1);
                    if (!go) break;
                    tc_fence_after();
                    const uint64_t k = k0 + stage * (L::TILE / 16);
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < HD / 16; ++kk)
                            umma_bf16(tmem_base + TM_S + 64 * b, k + step_k<ATOM>(kk), q0 + (n % SETS) * (L::Q / 16) + step_k<L::Q_HALF>(kk), idesc, kk != 0);
                        umma_commit(&M.s_full[b]);
                        umma_commit(&M.k_empty[stage]);
                    }
                } else {
                    constexpr uint32_t idesc = idesc_bf16_f32(TK, 2 * NR) | IDESC_A_MN | IDESC_B_MN;
                    go = wait_all(&M.v_full[stage], parity);
                    go = go && wait_all(&M.p_full[b], use & 1);
                    if (!go) break;
                    tc_fence_after();
                    const uint64_t v = v0 + stage * (L::TILE / 16), p = p0 + b * (L::WEIGHTS / 16);
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < TK / 16; ++kk)
                            umma_bf16(tmem_base + TM_O + 128 * (n % SETS), v + kk * (16 * 128 / 16), p + kk * (16 * 128 / 16), idesc, (i | kk) != 0);
                        umma_commit(&M.v_empty[stage]);
                        umma_commit(&M.pv_done[b]);
                    }
                }
                __syncwarp();
            }
            if (go && !scores && elect_one()) umma_commit(&M.o_full[n % SETS]);  // the piece's outputs are complete
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
    if (warp == 4 * SETS + 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem_base, TM_COLUMNS);
    }
    if (threadIdx.x == 0 && *abort_flag) *reinterpret_cast<volatile int*>(P.err.mirror) = DEV_ERR_TIMEOUT;
}

// The units that several CTAs share, in the order of their pieces: a thread takes four columns of a row.  A kernel of
// its own: the last CTA to arrive took 1 us for each piece of a unit, and 8 to 19 pieces where there are few units.
constexpr int JOIN_THREADS = 256;
template <int HD, int NR>
__global__ void __launch_bounds__(JOIN_THREADS) join_rows_kernel(const __grid_constant__ AttnParams P) {
    const int4 who = P.shared[2 * blockIdx.x], where = P.shared[2 * blockIdx.x + 1];
    const int row = (blockIdx.y * JOIN_THREADS + threadIdx.x) / (HD / 4), d4 = threadIdx.x % (HD / 4);
    const Pieces pieces{min(who.x, static_cast<int>(gridDim.x - blockIdx.x)), static_cast<int>(blockIdx.x)};
    if (row >= who.y || pieces.n < 2 || !c8::pieces_in_bounds(P, pieces)) return;
    Joined z;
#pragma unroll 8
    for (int i = 0; i < pieces.n; ++i) z.reference(P.part_stat[pieces.slot(i) * NR + row]);
#pragma unroll 8
    for (int i = 0; i < pieces.n; ++i) {
        const int64_t at = pieces.slot(i) * NR + row;
        z.add(P.part_stat[at], reinterpret_cast<const float4*>(P.partial)[at * (HD / 4) + d4]);
    }
    RowBlock B{};
    B.row0 = who.z;
    B.tok0 = who.w;
    write_row<__nv_bfloat16>(P, where.x, place_of(P, B, where.y, row), d4, z);
}

template <int HD, int NR>
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
    cudaError_t e = cudaFuncSetAttribute(rows_kernel<HD, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<HD, NR>::BYTES);
    if (e != cudaSuccess) return e;
    rows_kernel<HD, NR><<<p.ctas, threads_of(NR), Layout<HD, NR>::BYTES, s>>>(maps, P);
    join_rows_kernel<HD, NR><<<dim3(static_cast<unsigned>(p.ctas), NR * (HD / 4) / JOIN_THREADS), JOIN_THREADS, 0, s>>>(P);
    return cudaGetLastError();
}

template <int HD>
cudaError_t launch_rows(const AttnParams& P, const AttnPlan& p, cudaStream_t s, std::string* why) {
    return p.rows == 32 ? launch<HD, 32>(P, p, s, why) : p.rows == 48 ? launch<HD, 48>(P, p, s, why) : launch<HD, 64>(P, p, s, why);
}

}  // namespace

cudaError_t launch_attention_rows(const AttnParams& P, const AttnPlan& p, cudaStream_t s, std::string* why) {
    return P.c.d == 64 ? launch_rows<64>(P, p, s, why) : launch_rows<128>(P, p, s, why);
}

}  // namespace paged
}  // namespace kvb
