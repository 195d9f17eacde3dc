// Attention of new tokens over the paged cache of the model's own type: few query rows, many keys.
//
// For the g * n query rows of a (layer, sequence, KV head):
//     s_rj = scale * q_r . k_j,  p_rj = 2^(s_rj log2(e) - m_r),
//     o_r = sum_j p_rj v_j / sum_j p_rj,  lse_r = (m_r + log2 sum_j p_rj) ln 2
// in one pass over the keys, with a reference m_r that is raised when a score passes it by 2^8.
// One token of 64 query heads over 8 KV heads of 128, bf16: 16 x 32768 keys 299 us (7.2 TB/s, above the copy rate), 64 of
// 1024 to 8192 181 (0.97 of it), one of 4096 9.8.
// Every key is read once for 4 d g flops per 2 d elements (8 flop/byte at g = 8 and bf16), so HBM
// bounds it and what counts is that enough of it is on its way: each warp has a ring of its own
// in shared memory, filled by cp.async some steps of 16 keys ahead, and meets the other warps
// only at the end of a unit.  Slots that hold nothing visible are filled with zeros instead.
//
// bf16: mma.m16n8k16 with the 16 keys as M rows and 8 query rows as N, so that eight rows (one
// token of eight heads) waste nothing:
//   S^T = K Q^T    K by ldmatrix, Q in registers;
//   O^T = V^T P^T  V^T by transposing ldmatrix; P^T from S^T by an 8 x 8 transpose in registers,
//                  as a bf16 pair (hi, lo): 16 bits of a weight, for twice the products.
// fp32: CUDA cores, two products an instruction (f32x2).
//
// Three ways to cut a call: the keys of all units (layer, sequence, row block, head) form one line of
// 64-key tiles that the CTAs which fit the GPU share evenly, and the last CTA to arrive at a unit that
// several share joins its pieces in order; a cluster takes a unit, where units are few and short; a CTA
// takes a unit, where they are many and short.  Results do not depend on timing.
#include "paged_attn.cuh"

namespace kvb {
namespace paged {

namespace {

constexpr int WARPS = 4;              // of a CTA
constexpr int STEP = 16;              // keys of a warp's step
constexpr int TILE = STEP * WARPS;    // a tile
// Tiles that a unit itself counts as in the line.  0 / 4: 64 sequences of up to 4000 keys, 16 rows, 108 / 99 us, 24 of up to 2000, 8
// rows, 24.9 / 23.4; 16 of 8192 each 81 either way.
constexpr int LINE_UNIT_TILES = 4;
constexpr int MIN_TILES = 2;          // 1 and 4 measure the same within 2 %
// bf16 rows up to which mma.sync keeps up (d 64, 128).  16 rows, here / on tcgen05: 14.2 / 23.5 us for one
// sequence of 4096 keys, 8 heads, 58.0 / 59.1 for 16 of 1024 to 8192; 24 rows, 16 of 8192: 126 / 92.
constexpr int MMA_ROWS = 16;
// More rows stay here, in blocks of 16, where keys are few: up to FEW_TILES tiles of a row block an SM, and up to 128 rows over
// SHORT_KEYS / d tiles.  8 heads of 128, here / tcgen05, 40 rows: one sequence of 300, 4096, 8192 keys 10.5, 18.1, 26.5 /
// 15.6, 19.2, 21.9 us, four of 1024, 2048 16.8, 22.4 / 18.5, 20.4; 64 of up to 250, 500, 2000 26, 34, 87 / 39, 45, 70; of 500
// each 65 / 56.  20 rows of d 64: 64 of up to 1000 24 / 39.  The rules see the longest sequence and the most tokens alone, and
// lose where all sequences have as many: 64 of 5 tokens (40 rows) and 250, 500 keys each 48, 68 / 37, 56, and 500 at most
// 54 / 49; of 8 tokens 64, 88 / 55, 75 and 71 / 73 (the first figures are of 2 to 5 tokens each).
constexpr int FEW_TILES = 16, SHORT_KEYS = 1024;
// Two CTAs an SM where more would cut a unit into more pieces than this, all of which one CTA joins: 8 units of 35000, 131072 keys
// 36, 90 us with two and 42, 99 with four; 16 units of 35000 53 and 58.
constexpr int MOST_PIECES = 36;
// A CTA for each unit, if there are more of them than SMs and they are short: up to SHORT tiles, or so many units
// a tile that the last ones to finish do not count.  Against the line, 8 rows of d 128: 256 sequences of up to
// 300 keys, 8 heads, 35 us and 54, 128 of up to 1000 50 and 64, 64 of 1000 each 42 and 48, 256 of up to 4000 327 and 344;
// but 64 of up to 8192 202 and 181.  Only the longest sequence is looked at: 256 of 200 keys 46 and 47, but 255 of them and
// one of 4000 87 and 55 (70 and 54 where that one comes first).
constexpr int SHORT = 16;
// Steps of a warp up to which a cluster takes a unit where there are no more units than SMs.  One row block of 8,
// 8 heads, cluster / line: 4096 keys 10 / 14 us, 32768 34 / 41; 8 sequences of 8192 45 / 53, 16 of 1024 to 8192
// 57.9 / 55.7 (64 steps would take the clusters there).
constexpr int FEW_SHARES = 32;

// A step's K or V rows in shared memory: 16-byte chunks, chunk c of row r at c ^ swizzle(r), so that
// eight rows' chunks of one number, and a row's chunks, lie in different banks.
template <int CH>  // chunks of a row
__device__ __forceinline__ int swizzled(int row, int chunk) {
    if constexpr (CH >= 8) return row * CH + (chunk ^ (row & 7));
    else return row * CH + (chunk ^ ((row / (8 / CH)) & (CH - 1)));
}

// 16 zero bytes unless taken (`any`: an address of the buffer, not read)
__device__ __forceinline__ void copy16_or_zero(uint32_t dst, const void* src, const void* any, bool take) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(take ? src : any), "r"(take ? 16 : 0) : "memory");
}
// Ring of one warp: the K rows of a step and its V rows, in turn, each a part.
template <typename T, int D>
struct Ring {
    static constexpr int CH = D * sizeof(T) / 16;       // 16-byte chunks of a row
    static constexpr int PART = STEP * D * sizeof(T);   // bytes
    // Four warps' rings fit an SM four times in bf16, twice in fp32.  Twice in bf16, 6 parts of d 128: 16 x 32768 keys
    // 313 us against 303, 64 x 1024..8192 185 against 181, one sequence of 32768 31.6 against 34.3.  Registers for four
    // CTAs, 128 a thread, where they suffice (8 rows; three CTAs with 164): 64 of 1000, a CTA each, 42 against 53 us.  The line,
    // which runs three, takes the same time with either (16 x 32768 keys 299, 64 x 8192 312 and 311, 16 x 8192 81).
    static constexpr int FIT = (sizeof(T) == 2 ? 12288 : 24576) / PART;
    static constexpr int DEPTH = FIT > 16 ? 16 : FIT;   // d 128: 3 parts
    static constexpr int BYTES = DEPTH * PART;
};

// What one of NW warps reads in one unit: steps n = 0, 1, .. of keys first + TILE * n up to end.
template <typename T, int D, int NW>
struct Feeder {
    using R = Ring<T, D>;
    static constexpr int TILE = STEP * NW;            // keys between a warp's steps
    static constexpr int AT_ONCE = 32 / R::CH;        // rows that the warp copies at once
    static constexpr int COPIES = STEP / AT_ONCE;     // of a lane, for a part
    int s, first, end, steps;
    int64_t slab;     // block of page 0
    uint32_t ring;    // this warp's
    int now, next;    // pages of 32 steps, one a lane: those in use, and the 32 after them; -1: none
    int stage;        // that the next part is copied to
    int64_t row0;     // first row of the step that is asked for, in the pages; negative: its page is not there
    uint32_t absent;  // bit of a stage: likewise

    __device__ __forceinline__ int page_of(const AttnParams& P, int n0) const {
        const int n = n0 + (threadIdx.x & 31);
        if (n >= steps) return -1;
        const int64_t p = (first + TILE * n) >> P.c.page_log2;
        int pid = p < P.q.max_pages && c8::table_in_bounds(P.q, P.err, s, p)
                      ? __ldg(P.q.page_table + static_cast<int64_t>(s) * P.q.max_pages + p) : -1;
        if (pid < 0 || pid >= P.c.n_pages) {
            c8::err_set(P.err, DEV_ERR_BAD_SEQ);
            pid = -1;
        }
        const int64_t blocks = (static_cast<int64_t>(P.c.l_begin) + P.c.n_layers) * P.c.n_pages * P.c.H;
        if (pid >= 0 && !KVB_IN_BOUNDS(P.err, slab + static_cast<int64_t>(pid) * P.c.H, 1, blocks)) pid = -1;
        return pid;
    }
    __device__ __forceinline__ void begin(const AttnParams& P, int s_, int64_t slab_, int first_, int end_) {
        s = s_;
        slab = slab_;
        first = first_;
        end = end_;
        steps = first < end ? (end - first + TILE - 1) / TILE : 0;
        stage = 0;
        absent = 0;
        next = -1;
        now = page_of(P, 0);
    }
    // Asks for the rows of part m = 0, 1, .. in turn (K of step m / 2, then V): one group of copies, empty
    // past the last step.
    template <int KV>
    __device__ __forceinline__ void ask(const AttnParams& P, int n) {
        if (n < steps) {
            const int j = first + TILE * n;
            if constexpr (KV == 0) {
                if ((n & 31) == 0) {
                    if (n > 0) now = next;
                    if (n + 32 < steps) next = page_of(P, n + 32);
                }
                const int pid = __shfl_sync(0xffffffffu, now, n & 31);
                row0 = pid < 0 ? -1 : ((slab + static_cast<int64_t>(pid) * P.c.H) << P.c.page_log2) + (j & (P.c.page - 1));
                absent = pid < 0 ? absent | (1u << stage) : absent & ~(1u << stage);
            }
            const int lane = threadIdx.x & 31, row = lane / R::CH, chunk = lane % R::CH;
            const uint32_t dst = ring + stage * R::PART;
            const T* from = static_cast<const T*>(P.c.kv[KV]) + (row0 + row) * D + chunk * (16 / static_cast<int>(sizeof(T)));
            if (row0 >= 0 && j + STEP <= end) {
#pragma unroll
                for (int i = 0; i < COPIES; ++i)
                    copy16(dst + 16 * swizzled<R::CH>(row + i * AT_ONCE, chunk), from + i * AT_ONCE * D);
            } else {
#pragma unroll
                for (int i = 0; i < COPIES; ++i)
                    copy16_or_zero(dst + 16 * swizzled<R::CH>(row + i * AT_ONCE, chunk), from + i * AT_ONCE * D, P.c.kv[KV],
                                   row0 >= 0 && j + row + i * AT_ONCE < end);
            }
            stage = stage + 1 == R::DEPTH ? 0 : stage + 1;
        }
        copies_commit();
    }
};

// ------------------------------------------------------------------ bf16: tensor cores

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&a)[4], uint32_t p) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
                 : "r"(p)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&a)[4], uint32_t p) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
                 : "r"(p)
                 : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// The arithmetic of a warp.  Lane (r, c): keys r and r + 8 of a step, query rows 2c and 2c + 1 of
// each block of 8.
template <typename T, int D, int NB, int NW>
struct Math;

template <int D, int NB, int NW>
struct Math<__nv_bfloat16, D, NB, NW> {
    static constexpr int ROWS = 8 * NB, KS = D / 16, SHARED = 0;
    using R = Ring<__nv_bfloat16, D>;
    uint32_t q[NB][KS][2];
    float o[NB][KS][4];
    float m[NB][2], sum[NB][2];
    int qpos[NB][2];
    uint32_t hi[NB][2], lo[NB][2];  // the step's weights

    static __device__ __forceinline__ int r() { return (threadIdx.x & 31) >> 2; }
    static __device__ __forceinline__ int c() { return threadIdx.x & 3; }

    // row(i): address of query row i of the unit; rows from nrows on are zeros
    template <class Row>
    __device__ __forceinline__ void load(float*, int nrows, Row row) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const bool have = 8 * b + r() < nrows;
            const __nv_bfloat16* p = have ? row(8 * b + r()) + 2 * c() : nullptr;
#pragma unroll
            for (int t = 0; t < KS; ++t)
#pragma unroll
                for (int w = 0; w < 2; ++w) q[b][t][w] = have ? __ldg(reinterpret_cast<const uint32_t*>(p + 16 * t + 8 * w)) : 0u;
        }
    }
    __device__ __forceinline__ void reset(const RowBlock& B, int g) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
#pragma unroll
            for (int i = 0; i < KS; ++i) o[b][i][0] = o[b][i][1] = o[b][i][2] = o[b][i][3] = 0.f;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int row = 8 * b + 2 * c() + j;
                m[b][j] = LOWEST;
                sum[b][j] = 0.f;
                qpos[b][j] = row < B.nrows ? B.pos + (B.row0 + row) / g : INT32_MIN;
            }
        }
    }
    // Weights of keys j .. j + 15, whose rows are at `at` in shared memory; f = scale * log2(e).
    // whole: all rows see all keys.
    __device__ __forceinline__ void keys(uint32_t at, float*, int j, int end, bool whole, bool absent, float f) {
        const int lane = threadIdx.x & 31;
        // products in a few chains, so that one need not wait for the last
        constexpr int CHAINS = NB * 4 <= KS ? 4 / NB : 1;
        float sc[NB][4], part[CHAINS][NB][4];
#pragma unroll
        for (int x = 0; x < CHAINS; ++x)
#pragma unroll
            for (int b = 0; b < NB; ++b) part[x][b][0] = part[x][b][1] = part[x][b][2] = part[x][b][3] = 0.f;
#pragma unroll
        for (int t = 0; t < KS; ++t) {
            uint32_t a[4];
            ldmatrix4(a, at + 16 * swizzled<R::CH>(lane & 15, 2 * t + (lane >> 4)));
#pragma unroll
            for (int b = 0; b < NB; ++b) mma16816(part[t % CHAINS][b], a, q[b][t][0], q[b][t][1]);
        }
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                sc[b][u] = part[0][b][u];
#pragma unroll
                for (int x = 1; x < CHAINS; ++x) sc[b][u] += part[x][b][u];
            }
        bool raise = false;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (!whole) {
                    const int key = j + r() + 8 * (u >> 1);
                    if (absent || key >= end || key > qpos[b][u & 1]) sc[b][u] = -INFINITY;
                }
                raise |= sc[b][u] * f > m[b][u & 1] + MARGIN;
            }
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    float top = fmaxf(sc[b][w], sc[b][w + 2]) * f;
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                    const float up = fmaxf(m[b][w], top), lower = ex2(m[b][w] - up);
                    m[b][w] = up;
                    sum[b][w] *= lower;
#pragma unroll
                    for (int i = 0; i < KS; ++i) {
                        o[b][i][w] *= lower;
                        o[b][i][w + 2] *= lower;
                    }
                }
        }
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                float w[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    w[i] = ex2(fmaf(sc[b][2 * hf + i], f, -m[b][i]));
                    sum[b][i] += w[i];
                }
                const uint32_t x = pack_bf16x2(w[0], w[1]);
                hi[b][hf] = transpose8x8(x);
                lo[b][hf] = transpose8x8(pack_bf16x2(w[0] - __uint_as_float(x << 16), w[1] - __uint_as_float(x & 0xffff0000u)));
            }
    }
    // Their weighted value rows, at `at`, are added.
    __device__ __forceinline__ void values(uint32_t at, float*) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int i = 0; i < KS; ++i) {
            uint32_t a[4];
            ldmatrix4_trans(a, at + 16 * swizzled<R::CH>((lane & 7) + 8 * (lane >> 4), 2 * i + ((lane >> 3) & 1)));
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                mma16816(o[b][i], a, hi[b][0], hi[b][1]);
                mma16816(o[b][i], a, lo[b][0], lo[b][1]);
            }
        }
    }
    // out [ROWS][D] and stat [ROWS] (reference, sum) of this warp
    __device__ __forceinline__ void finish(float* out, float2* stat) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                float t = sum[b][w];
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) t += __shfl_xor_sync(0xffffffffu, t, x);
                const int row = 8 * b + 2 * c() + w;
                if (r() == 0) stat[row] = make_float2(m[b][w], t);
#pragma unroll
                for (int i = 0; i < KS; ++i) {
                    out[row * D + 16 * i + r()] = o[b][i][w];
                    out[row * D + 16 * i + 8 + r()] = o[b][i][w + 2];
                }
            }
    }
};

// ------------------------------------------------------------------ fp32: CUDA cores

__device__ __forceinline__ float4 shared4(uint32_t p) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(p) : "memory");
    return v;
}

// Scores: lane (r, c) takes quarter c of the dims for keys r and r + 8 and all rows; the quarters are
// added by exchanging halves, which leaves each lane RL rows, RL * c on.  Outputs: a lane takes 4
// dims of all rows for every 32 / (D / 4)-th key.  NB: rows, of which there are 4 or 8.
template <int D, int NB, int NW>
struct Math<float, D, NB, NW> {
    static constexpr int ROWS = NB, RL = ROWS / 4;
    static constexpr int QUARTER = D / 4 + 4;  // 4 floats between: the quarters lie in different banks
    static constexpr int DL = D / 4, KP = 32 / DL;
    static constexpr int SHARED = ROWS * 4 * QUARTER + NW * STEP * ROWS;  // floats: queries, weights
    using R = Ring<float, D>;
    float2 o[ROWS / 2][4];  // rows 2i, 2i + 1; dim
    float m[RL], sum[RL];
    int qpos[RL];

    static __device__ __forceinline__ int r() { return threadIdx.x & 7; }
    static __device__ __forceinline__ int c() { return (threadIdx.x & 31) >> 3; }
    static __device__ __forceinline__ float* weights(float* shared) {
        return shared + ROWS * 4 * QUARTER + (threadIdx.x >> 5) * STEP * ROWS;
    }

    template <class Row>
    __device__ __forceinline__ void load(float* shared, int nrows, Row row) {
        for (int i = threadIdx.x; i < ROWS * (D / 4); i += 32 * NW) {
            const int y = i / (D / 4), d4 = i % (D / 4);
            const float4 v = y < nrows ? __ldg(reinterpret_cast<const float4*>(row(y)) + d4) : make_float4(0.f, 0.f, 0.f, 0.f);
            *reinterpret_cast<float4*>(shared + (y * 4 + d4 / (D / 16)) * QUARTER + 4 * (d4 % (D / 16))) = v;
        }
    }
    __device__ __forceinline__ void reset(const RowBlock& B, int g) {
#pragma unroll
        for (int i = 0; i < ROWS / 2; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x) o[i][x] = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < RL; ++j) {
            const int row = RL * c() + j;
            m[j] = LOWEST;
            sum[j] = 0.f;
            qpos[j] = row < B.nrows ? B.pos + (B.row0 + row) / g : INT32_MIN;
        }
    }
    __device__ __forceinline__ void keys(uint32_t at, float* shared, int j, int end, bool whole, bool absent, float f) {
        const uint32_t sq = smem_u32(shared) + c() * QUARTER * 4;
        float2 acc[2][ROWS];
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int y = 0; y < ROWS; ++y) acc[k][y] = make_float2(0.f, 0.f);
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
            float4 k[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) k[i] = shared4(at + 16 * swizzled<R::CH>(r() + 8 * i, c() * (D / 16) + x));
#pragma unroll
            for (int y = 0; y < ROWS; ++y) {
                const float4 v = shared4(sq + (y * 4 * QUARTER + 4 * x) * 4);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    acc[i][y] = fma2(make_float2(k[i].x, k[i].y), make_float2(v.x, v.y), acc[i][y]);
                    acc[i][y] = fma2(make_float2(k[i].z, k[i].w), make_float2(v.z, v.w), acc[i][y]);
                }
            }
        }
        float sc[2][RL];  // key, row
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float h[ROWS / 2];
#pragma unroll
            for (int y = 0; y < ROWS / 2; ++y) {
                const float a = acc[i][y].x + acc[i][y].y, b = acc[i][ROWS / 2 + y].x + acc[i][ROWS / 2 + y].y;
                const float keep = c() & 2 ? b : a, give = c() & 2 ? a : b;
                h[y] = keep + __shfl_xor_sync(0xffffffffu, give, 16);
            }
#pragma unroll
            for (int y = 0; y < RL; ++y) {
                const float keep = c() & 1 ? h[RL + y] : h[y], give = c() & 1 ? h[y] : h[RL + y];
                sc[i][y] = keep + __shfl_xor_sync(0xffffffffu, give, 8);
            }
        }
        bool raise = false;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int y = 0; y < RL; ++y) {
                if (!whole) {
                    const int key = j + r() + 8 * i;
                    if (absent || key >= end || key > qpos[y]) sc[i][y] = -INFINITY;
                }
                raise |= sc[i][y] * f > m[y] + MARGIN;
            }
        if (__any_sync(0xffffffffu, raise)) {
            float lower[RL];
#pragma unroll
            for (int y = 0; y < RL; ++y) {
                float top = fmaxf(sc[0][y], sc[1][y]) * f;
#pragma unroll
                for (int x = 1; x < 8; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                const float up = fmaxf(m[y], top);
                lower[y] = ex2(m[y] - up);
                m[y] = up;
                sum[y] *= lower[y];
            }
#pragma unroll
            for (int y = 0; y < ROWS; ++y) {
                const float a = __shfl_sync(0xffffffffu, lower[y % RL], 8 * (y / RL));
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    if (y % 2 == 0) o[y / 2][x].x *= a;
                    else o[y / 2][x].y *= a;
                }
            }
        }
        float* w = weights(shared) + r() * ROWS + RL * c();
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int y = 0; y < RL; ++y) {
                const float x = ex2(fmaf(sc[i][y], f, -m[y]));
                sum[y] += x;
                w[8 * i * ROWS + y] = x;
            }
    }
    __device__ __forceinline__ void values(uint32_t at, float* shared) {  // after the warp has met
        const int lane = threadIdx.x & 31;
        const uint32_t sw = smem_u32(weights(shared));
#pragma unroll
        for (int i = 0; i < STEP / KP; ++i) {
            const int key = i * KP + lane / DL;
            const float4 v = shared4(at + 16 * swizzled<R::CH>(key, lane % DL));
            const float vx[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int y = 0; y < ROWS / 4; ++y) {
                const float4 a = shared4(sw + (key * ROWS + 4 * y) * 4);
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    o[2 * y][x] = fma2(make_float2(a.x, a.y), make_float2(vx[x], vx[x]), o[2 * y][x]);
                    o[2 * y + 1][x] = fma2(make_float2(a.z, a.w), make_float2(vx[x], vx[x]), o[2 * y + 1][x]);
                }
            }
        }
    }
    __device__ __forceinline__ void finish(float* out, float2* stat) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int y = 0; y < RL; ++y) {
            float t = sum[y];
#pragma unroll
            for (int x = 1; x < 8; x <<= 1) t += __shfl_xor_sync(0xffffffffu, t, x);
            if (r() == 0) stat[RL * c() + y] = make_float2(m[y], t);
        }
#pragma unroll
        for (int i = 0; i < ROWS / 2; ++i) {
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int k = DL; k < 32; k <<= 1) {
                    o[i][x].x += __shfl_xor_sync(0xffffffffu, o[i][x].x, k);
                    o[i][x].y += __shfl_xor_sync(0xffffffffu, o[i][x].y, k);
                }
            if (lane < DL) {
                reinterpret_cast<float4*>(out + 2 * i * D)[lane] = make_float4(o[i][0].x, o[i][1].x, o[i][2].x, o[i][3].x);
                reinterpret_cast<float4*>(out + (2 * i + 1) * D)[lane] = make_float4(o[i][0].y, o[i][1].y, o[i][2].y, o[i][3].y);
            }
        }
    }
};

// ------------------------------------------------------------------ the kernels

// Shared memory: the warps' rings, which later hold their outputs; queries and weights (fp32); the
// warps' statistics; in a cluster what the CTAs hand to this one: a slice of the columns, 16 parts at
// most of a share that gets smaller with their number, and every part's statistics.
template <typename T, int D, int NB, int NW>
struct Shared {
    using M = Math<T, D, NB, NW>;
    static constexpr int ROWS = M::ROWS, RING = Ring<T, D>::BYTES;
    static_assert(ROWS * D * 4 <= RING, "a warp's outputs take its ring's place");
    static constexpr int MORE = NW * RING, STAT = MORE + M::SHARED * 4, JOIN = STAT + NW * ROWS * 8;
    static constexpr int NT = 32 * NW, JOIN_STAT = JOIN + (ROWS * (D / 4) + NT - 1) / NT * NT * 16;
    static constexpr int bytes(bool cluster) { return cluster ? JOIN_STAT + 16 * ROWS * 8 : JOIN; }
};

// A CTA's NW warps over keys [k0, k1) of a unit; their outputs and statistics are in shared memory
// afterwards, for every thread to read.
template <typename T, int D, int NB, int NW>
__device__ __forceinline__ void attend(const AttnParams& P, const RowBlock& B, int s, int l, int h, int k0, int k1, uint8_t* smem) {
    using M = Math<T, D, NB, NW>;
    using R = Ring<T, D>;
    using S = Shared<T, D, NB, NW>;
    const int warp = threadIdx.x >> 5;
    uint8_t* mine = smem + warp * R::BYTES;
    float* shared = reinterpret_cast<float*>(smem + S::MORE);
    Feeder<T, D, NW> feed;
    feed.ring = smem_u32(mine);
    feed.begin(P, s, (static_cast<int64_t>(P.c.l_begin) + l) * P.c.n_pages * P.c.H + h, k0 + STEP * warp, k1);
    M math;
    math.load(shared, B.nrows, [&](int row) { return address<T>(P.query, l, place_of(P, B, h, row)); });
    static_assert(R::DEPTH >= 3, "a step's K, its V and the next K");
#pragma unroll
    for (int m = 0; m < R::DEPTH - 1; ++m) {
        if (m % 2 == 0) feed.template ask<0>(P, m / 2);
        else feed.template ask<1>(P, m / 2);
    }
    math.reset(B, P.g);
    if constexpr (M::SHARED > 0) __syncthreads();  // the queries
    // the part that is asked for while part m is used is m + DEPTH - 1, in the place of part m - 1
    constexpr int NEXT_K = (R::DEPTH - 1) % 2, NEXT_V = R::DEPTH % 2;
    int stage = 0;
    bool odd = false;  // values that are not finite have been taken out
    for (int n = 0; n < feed.steps; ++n) {
        copies_wait<R::DEPTH - 2>();
        const bool absent = (feed.absent >> stage) & 1;
        __syncwarp();  // every lane's copies of the part are there, and the part before it has been used
        feed.template ask<NEXT_K>(P, n + (R::DEPTH - 1) / 2);
        const int j = feed.first + feed.TILE * n;
        const bool whole = !absent && j + STEP <= k1 && j + STEP - 1 <= B.pos_lo;
        math.keys(feed.ring + stage * R::PART, shared, j, k1, whole, absent, P.scale_log2);
        stage = stage + 1 == R::DEPTH ? 0 : stage + 1;
        copies_wait<R::DEPTH - 2>();
        __syncwarp();
        feed.template ask<NEXT_V>(P, n + R::DEPTH / 2);
        if (j + STEP - 1 > B.pos_lo && B.pos_lo + 1 < k1) {  // some rows see keys of it that others do not
#pragma unroll 1
            for (int i = (threadIdx.x & 31) + max(B.pos_lo + 1 - j, 0) * R::CH; i < STEP * R::CH; i += 32) odd |= make_finite<T>(reinterpret_cast<uint4*>(mine + stage * R::PART)[i]);
            __syncwarp();
        }
        math.values(feed.ring + stage * R::PART, shared);
        stage = stage + 1 == R::DEPTH ? 0 : stage + 1;
    }
    copies_wait<0>();
    __syncwarp();
    math.finish(reinterpret_cast<float*>(mine), reinterpret_cast<float2*>(smem + S::STAT) + warp * S::ROWS);
    if (__syncthreads_or(odd)) {
#pragma unroll 1
        for (int i = threadIdx.x; i < B.nrows * D; i += 32 * NW) {  // row 0 .. of warp 0's outputs
            const int row = i / D, pos = B.pos + (B.row0 + row) / P.g;
            for (int j = max(k0, B.pos_lo + 1); j < k1 && j <= pos; ++j) {
                const float v = value_of<T>(P, s, l, h, j, i % D);
                if (not_finite(v)) reinterpret_cast<float*>(smem)[i] += v;
            }
        }
        __syncthreads();
    }
}

// Four columns of a row over a CTA's warps.
template <typename T, int D, int NB, int NW>
__device__ __forceinline__ Joined join_warps(const uint8_t* smem, int row, int d4) {
    using S = Shared<T, D, NB, NW>;
    const float2* stat = reinterpret_cast<const float2*>(smem + S::STAT) + row;
    Joined z;
#pragma unroll
    for (int w = 0; w < NW; ++w) z.reference(stat[w * S::ROWS]);
#pragma unroll
    for (int w = 0; w < NW; ++w) z.add(stat[w * S::ROWS], reinterpret_cast<const float4*>(smem + w * S::RING + row * D * 4)[d4]);
    return z;
}

// Many keys: the line of tiles, shared evenly by the CTAs that fit the GPU.
template <typename T, int D, int NB>
__global__ void __launch_bounds__(32 * WARPS, sizeof(T) == 2 && NB == 1 ? 4 : 1) line_kernel(const __grid_constant__ AttnParams P) {
    constexpr int NT = 32 * WARPS;
    using S = Shared<T, D, NB, WARPS>;
    constexpr int ROWS = S::ROWS;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int s_last;
    __shared__ LineStart s_start;
    __shared__ int s_scan[WARPS];

    int at, stop, share, l, e, h, first;
    if (!c8::line_start<ROWS, TILE, NT, LINE_UNIT_TILES, 4>(P, s_scan, &s_start, at, stop, share, l, e, h, first)) return;
    const int entries = P.q.n_seq * P.row_blocks;
    auto entry = [&](int x) { return c8::row_block(P, x / P.row_blocks, x % P.row_blocks, ROWS); };
    RowBlock B = entry(e);
    int tiles = c8::unit_tiles<TILE, LINE_UNIT_TILES>(B);

    for (;;) {  // one unit, or a piece of one, after another
        const int last = min(tiles, first + (stop - at));  // tiles [first, last), those without keys first
        const int k0 = max(first - LINE_UNIT_TILES, 0) * TILE, k1 = min(B.kv_end, (last - LINE_UNIT_TILES) * TILE);
        if (last > LINE_UNIT_TILES) {
            const int64_t unit = (static_cast<int64_t>(l) * entries + e) * P.c.H + h;
            attend<T, D, NB, WARPS>(P, B, e / P.row_blocks, l, h, k0, k1, smem);

            // the CTAs that share this unit, and this one's slot
            const int u0 = at - first, c0 = (u0 + LINE_UNIT_TILES) / share;
            const int pieces = (u0 + tiles - 1) / share - c0 + 1;
            const int64_t part0 = (2 * static_cast<int64_t>(blockIdx.x) + (first <= LINE_UNIT_TILES)) * ROWS;
            for (int i = threadIdx.x; i < B.nrows * (D / 4); i += NT) {
                const int row = i / (D / 4), d4 = i % (D / 4);
                const Joined z = join_warps<T, D, NB, WARPS>(smem, row, d4);
                if (pieces == 1) {
                    write_row<T>(P, l, place_of(P, B, h, row), d4, z);
                } else if (KVB_IN_BOUNDS(P.err, part0 + row, 1, P.slots * ROWS)) {
                    reinterpret_cast<float4*>(P.partial + (part0 + row) * D)[d4] = z.acc;
                    if (d4 == 0) P.part_stat[part0 + row] = make_float2(z.m, z.sum);
                }
            }
            if (pieces > 1)
                join_pieces<T, D, ROWS, NT>(P, B, Pieces{pieces, c0}, unit, l, h, &s_last, reinterpret_cast<float*>(smem), S::MORE / 4);
        }

        at += last - first;
        if (at >= stop) return;
        first = 0;
        if (++h == P.c.H) {
            h = 0;
            do {
                if (++e == entries) {
                    e = 0;
                    if (++l == P.c.n_layers) return;  // not reached while the call's arrays stay as they are
                }
                B = entry(e);
                tiles = c8::unit_tiles<TILE, LINE_UNIT_TILES>(B);
            } while (tiles == 0);
        }
        __syncthreads();  // shared memory is free for the next unit
    }
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Shared memory of CTA `rank` of the cluster, at the address that p has in this one.
__device__ __forceinline__ uint32_t of_rank(uint32_t p, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(p), "r"(rank));
    return r;
}
__device__ __forceinline__ void hand4(uint32_t p, float4 v) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(p), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}
__device__ __forceinline__ void hand2(uint32_t p, float2 v) {
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1,%2};" ::"r"(p), "f"(v.x), "f"(v.y) : "memory");
}

// Few keys: a cluster of CTAs for each unit, an even share of its keys each.  Every CTA hands each of
// the others its part of the columns that the other joins, through distributed shared memory: no
// global scratch, no atomics.  And many short units: a CTA for each, which waits for no other.
template <typename T, int D, int NB>
__global__ void __launch_bounds__(32 * WARPS, sizeof(T) == 2 && NB == 1 ? 4 : 1) cluster_kernel(const __grid_constant__ AttnParams P) {
    constexpr int NT = 32 * WARPS;
    using S = Shared<T, D, NB, WARPS>;
    constexpr int ROWS = S::ROWS;
    extern __shared__ __align__(128) uint8_t smem[];
    const int parts = P.cluster, part = static_cast<int>(blockIdx.x) % parts;  // a power of two, at most 16
    if (parts > 1) cluster_arrive();  // the others may be written to once all have come here
    int unit = static_cast<int>(blockIdx.x) / parts;
    const int h = unit % P.c.H;
    unit /= P.c.H;
    const int entries = P.q.n_seq * P.row_blocks;
    const int e = unit % entries, l = unit / entries;
    const RowBlock B = c8::row_block(P, e / P.row_blocks, e % P.row_blocks, ROWS);
    const int items = B.nrows * (D / 4);  // 0: none of the cluster has rows
    if (items > 0) {
        const int tiles = (B.kv_end + TILE - 1) / TILE;
        const int share = (tiles + parts - 1) / parts * TILE;
        attend<T, D, NB, WARPS>(P, B, e / P.row_blocks, l, h, min(B.kv_end, part * share), min(B.kv_end, (part + 1) * share), smem);
    }
    if (parts > 1) cluster_wait();
    // item i = four columns of a row: joined by CTA (i / per) % parts, as number i / NT * per + i % per of its own
    const int per = NT / parts;
    const uint32_t join = smem_u32(smem + S::JOIN), join_stat = smem_u32(smem + S::JOIN_STAT);
    for (int i = threadIdx.x; i < items; i += NT) {
        const int row = i / (D / 4), d4 = i % (D / 4);
        const Joined z = join_warps<T, D, NB, WARPS>(smem, row, d4);
        if (parts == 1) {
            write_row<T>(P, l, place_of(P, B, h, row), d4, z);
        } else {
            hand4(of_rank(join + 16 * ((i / NT * per + i % per) * parts + part), i / per % parts), z.acc);
            for (int x = d4; x < parts; x += D / 4) hand2(of_rank(join_stat + 8 * (row * parts + part), x), make_float2(z.m, z.sum));
        }
    }
    if (parts == 1) return;
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    // `parts` lanes take an item's parts, one each, and add them in a tree
    const float4* acc = reinterpret_cast<const float4*>(smem + S::JOIN);
    const float2* stat = reinterpret_cast<const float2*>(smem + S::JOIN_STAT);
    const int from = threadIdx.x % parts;
    for (int round = 0; round * NT + part * per < items; ++round) {
        const int y = round * per + static_cast<int>(threadIdx.x) / parts, i = round * NT + part * per + static_cast<int>(threadIdx.x) / parts;
        const int row = min(i, items - 1) / (D / 4), d4 = min(i, items - 1) % (D / 4);
        Joined z;
        const float2 st = stat[row * parts + from];
        z.m = st.x;
        for (int x = 1; x < parts; x <<= 1) z.m = fmaxf(z.m, __shfl_xor_sync(0xffffffffu, z.m, x));
        z.add(st, i < items ? acc[y * parts + from] : make_float4(0.f, 0.f, 0.f, 0.f));
        for (int x = 1; x < parts; x <<= 1) {
            z.sum += __shfl_xor_sync(0xffffffffu, z.sum, x);
            z.acc.x += __shfl_xor_sync(0xffffffffu, z.acc.x, x);
            z.acc.y += __shfl_xor_sync(0xffffffffu, z.acc.y, x);
            z.acc.z += __shfl_xor_sync(0xffffffffu, z.acc.z, x);
            z.acc.w += __shfl_xor_sync(0xffffffffu, z.acc.w, x);
        }
        if (i < items && from == 0) write_row<T>(P, l, place_of(P, B, h, row), d4, z);
    }
}

// One instance of the line: CTAs of it that fit an SM (P null), or its launch.
template <typename T, int D, int NB>
cudaError_t line_instance(const AttnParams* P, int ctas, cudaStream_t s, int* fit) {
    constexpr int smem = Shared<T, D, NB, WARPS>::bytes(false);
    const auto kernel = line_kernel<T, D, NB>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (!P) {
        static const int resident = [&] {
            int n = 0;
            return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, 32 * WARPS, smem) == cudaSuccess ? n : 0;
        }();
        *fit = resident;
        return cudaSuccess;
    }
    kernel<<<ctas, 32 * WARPS, smem, s>>>(*P);
    return cudaGetLastError();
}

// One instance of the clusters: how many of each size are resident at once (P null), or its launch.
template <typename T, int D, int NB>
cudaError_t cluster_instance(const AttnParams* P, int cluster, int ctas, cudaStream_t s, int* fit) {
    constexpr int smem = Shared<T, D, NB, WARPS>::bytes(true);
    const auto kernel = cluster_kernel<T, D, NB>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(32 * WARPS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(cluster);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (!P) {
        struct Resident {
            int n[5];
        };
        static const Resident resident = [&] {
            Resident r{};
            for (int i = 0; i < 5; ++i) {
                attr.val.clusterDim.x = 1u << i;
                cfg.gridDim = dim3(1u << i);
                if (cudaOccupancyMaxActiveClusters(&r.n[i], kernel, &cfg) != cudaSuccess) r.n[i] = 0;
            }
            (void)cudaGetLastError();
            return r;
        }();
        for (int i = 0; i < 5; ++i) fit[i] = resident.n[i];
        return cudaSuccess;
    }
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    return cudaLaunchKernelEx(&cfg, kernel, *P);
}

template <typename T, int D, int NB>
cudaError_t instance(const AttnParams* P, const AttnPlan& p, cudaStream_t s, int* fit) {
    return p.cluster ? cluster_instance<T, D, NB>(P, p.cluster, p.ctas, s, fit) : line_instance<T, D, NB>(P, p.ctas, s, fit);
}

template <typename T, int D>
cudaError_t instance_rows(const AttnPlan& p, const AttnParams* P, cudaStream_t s, int* fit) {
    if constexpr (sizeof(T) == 4) return p.rows == 4 ? instance<T, D, 4>(P, p, s, fit) : instance<T, D, 8>(P, p, s, fit);
    else if constexpr (D < 64) return p.rows == 32 ? instance<T, D, 4>(P, p, s, fit) : p.rows == 16 ? instance<T, D, 2>(P, p, s, fit) : instance<T, D, 1>(P, p, s, fit);
    else return p.rows == 16 ? instance<T, D, 2>(P, p, s, fit) : instance<T, D, 1>(P, p, s, fit);
}

template <typename T>
cudaError_t instance_dim(int d, const AttnPlan& p, const AttnParams* P, cudaStream_t s, int* fit) {
    switch (d) {
        case 16: return instance_rows<T, 16>(p, P, s, fit);
        case 32: return instance_rows<T, 32>(p, P, s, fit);
        case 64: return instance_rows<T, 64>(p, P, s, fit);
        default: return instance_rows<T, 128>(p, P, s, fit);
    }
}

cudaError_t pick(kvb_dtype dtype, int d, const AttnPlan& p, const AttnParams* P, cudaStream_t s, int* fit) {
    return dtype == KVB_BF16 ? instance_dim<__nv_bfloat16>(d, p, P, s, fit) : instance_dim<float>(d, p, P, s, fit);
}

// CTAs, at most `most`: where units of one length leave no CTA with parts of two, and not too few CTAs
// with the others' keys too, that many.  With two CTAs an SM of this file's kernel, 16 x 8192 / 16 x 32768 keys of one length
// take 86 / 310 us so and 90 / 321 on all of them, unequal ones (16 x 1024 .. 8192) 54 either way; more
// units than CTAs, unequal ones, 186 and 184.  The tcgen05 kernel
// has 152 and longer ways from one unit to the next: 128 of them 86 and 152 93 us, but unequal lengths 94 and 78.
int even_share(int64_t units, int most, bool tensor) {
    if (units > most && !tensor) return most;
    const int64_t n = units <= most ? units * (most / units) : (units + (units + most - 1) / most - 1) / ((units + most - 1) / most);
    return n * 20 >= most * (tensor ? 18 : 15) ? static_cast<int>(n) : most;
}

}  // namespace

AttnPlan plan_attention(const Pages& c, const Seqs& q, kvb_dtype dtype, int g, int num_sms) {
    AttnPlan p{};
    const int64_t most = static_cast<int64_t>(q.max_tokens) * g;  // rows of one sequence and head
    const int64_t max_kv = q.max_kv > 0 ? q.max_kv : 1;
    const double all_blocks = (static_cast<double>(c.l_begin) + c.n_layers) * c.n_pages * c.H;
    const int64_t shares = (max_kv + TILE - 1) / TILE;  // tiles of a unit
    const double units16 = static_cast<double>((most + 15) / 16) * c.n_layers * q.n_seq * c.H;  // of 16 rows
    const bool small = units16 * shares <= static_cast<double>(FEW_TILES) * num_sms || (most <= 128 && shares * c.d <= SHORT_KEYS);
    p.tensor = dtype == KVB_BF16 && c.d >= 64 && most > MMA_ROWS && !small && c.n_pages > 0 && all_blocks < 2147483648.0;  // (blocks are TMA coordinates)
    // blocks of up to 64 rows in the tcgen05 kernel, as small as their number allows
    const int64_t few = (most + 63) / 64, each = few > 0 ? (most + few - 1) / few : 1;
    p.rows = p.tensor ? (each <= 32 ? 32 : each <= 48 ? 48 : 64) : dtype == KVB_F32 ? (most <= 4 ? 4 : 8) : most <= 8 ? 8 : most <= 16 || c.d >= 64 ? 16 : 32;
    const double blocks = static_cast<double>((most + p.rows - 1) / p.rows);
    const double units = blocks * c.n_layers * q.n_seq * c.H;
    p.tiles = units * (shares + (p.tensor ? unit_tiles_of(p.rows) : LINE_UNIT_TILES));  // of 64 keys; the tcgen05 kernel's have 128
    if (p.tiles > static_cast<double>(1 << 30)) return p;  // refused
    p.row_blocks = static_cast<int>(blocks);
    p.units = static_cast<int64_t>(units);
    if (!p.tensor && p.units <= num_sms && shares <= FEW_SHARES * 16) {
        int most_of[5] = {};
        p.cluster = 1;
        pick(dtype, c.d, p, nullptr, nullptr, most_of);
        // the largest cluster of which all are resident at once, no larger than the keys have steps for
        for (int i = 1; i < 5; ++i)
            if (p.units <= most_of[i] && (1 << i) < 2 * shares) p.cluster = 1 << i;
        p.ctas = static_cast<int>(p.units) * p.cluster;
        if (p.units <= most_of[0] && shares <= static_cast<int64_t>(FEW_SHARES) * p.cluster) return p;
        p.cluster = 0;
    }
    if (!p.tensor && p.units > num_sms && (shares <= SHORT || p.units > SHORT * shares)) {
        p.cluster = 1;  // a CTA for each unit
        p.ctas = static_cast<int>(p.units);
        return p;
    }
    int fit = 1;
    if (!p.tensor) pick(dtype, c.d, p, nullptr, nullptr, &fit);
    // three CTAs an SM at most, although four fit: 16 x 32768 keys 299 us and 308, 64 of 1024 to 8192 177 and 185, 32 of 2048 to
    // 16384 176 and 183, 8 x 20000 103 and 108, 8 x 35000 169 and 176; but 64 x 8192 312 and 304, which no size that the
    // host knows tells from the others
    if (fit > 3) fit = 3;
    if (fit > 2 && p.units * MOST_PIECES < static_cast<int64_t>(num_sms) * fit) fit = 2;
    // the CTAs that fit the GPU, no more than the keys give the least share to
    p.min_tiles = p.tensor ? 1 : MIN_TILES;
    const double need = p.tensor ? units * ((max_kv + 127) / 128 + unit_tiles_of(p.rows)) : (p.tiles + p.min_tiles - 1) / p.min_tiles;
    p.ctas = even_share(p.units, num_sms * (fit > 0 ? fit : 1), p.tensor);
    if (need < p.ctas) p.ctas = static_cast<int>(need) < 1 ? 1 : static_cast<int>(need);
    p.slots = 2 * static_cast<int64_t>(p.ctas);
    p.counter_bytes = p.tensor ? 0 : (static_cast<size_t>(p.units) * sizeof(int) + 255) / 256 * 256;
    p.partial_bytes = static_cast<size_t>(p.slots) * p.rows * (c.d + 2) * sizeof(float);  // slots are even: a multiple of 16
    p.shared_bytes = p.tensor ? static_cast<size_t>(p.ctas) * 2 * sizeof(int4) : 0;
    return p;
}

cudaError_t launch_attention(const AttnParams& P, kvb_dtype dtype, const AttnPlan& p, cudaStream_t s) {
    return pick(dtype, P.c.d, p, &P, s, nullptr);
}

}  // namespace paged
}  // namespace kvb
