// Attention of new tokens over the paged cache of the model's own type: few query rows, many keys.
//
// For the g * n query rows of a (layer, sequence, KV head):
//     s_rj = scale * q_r . k_j,  p_rj = 2^(s_rj log2(e) - m_r),
//     o_r = sum_j p_rj v_j / sum_j p_rj,  lse_r = (m_r + log2 sum_j p_rj) ln 2
// in one pass over the keys, with a reference m_r that is raised when a score passes it by 2^8.
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
// The keys of all units (layer, sequence, row block, head) form one line of 64-key tiles that the
// CTAs which fit the GPU share evenly; the last CTA to arrive at a unit that several share joins
// its pieces in order, so results do not depend on timing.
#include <cfloat>

#include "cache8_attn.cuh"
#include "paged.h"

namespace kvb {
namespace paged {

namespace {

using c8::ex2;
using c8::LineStart;
using c8::Pieces;
using c8::RowBlock;

constexpr int WARPS = 4, NT = 32 * WARPS;
constexpr int STEP = 16;              // keys of a warp's step
constexpr int TILE = STEP * WARPS;    // of a CTA's
constexpr float MARGIN = 8.f;         // a reference is raised past this much (base 2)
constexpr float LOWEST = -FLT_MAX;    // reference of a row that has seen nothing
constexpr int MIN_TILES = 2;

// A step's K or V rows in shared memory: 16-byte chunks, chunk c of row r at c ^ swizzle(r), so that
// eight rows' chunks of one number, and a row's chunks, lie in different banks.
template <int CH>  // chunks of a row
__device__ __forceinline__ int swizzled(int row, int chunk) {
    if constexpr (CH >= 8) return row * CH + (chunk ^ (row & 7));
    else return row * CH + (chunk ^ ((row / (8 / CH)) & (CH - 1)));
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// 16 zero bytes unless taken (`any`: an address of the buffer, not read)
__device__ __forceinline__ void copy16_or_zero(uint32_t dst, const void* src, const void* any, bool take) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(take ? src : any), "r"(take ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Ring of one warp: steps of K and V rows.
template <typename T, int D>
struct Ring {
    static constexpr int CH = D * sizeof(T) / 16;          // chunks of a row
    static constexpr int PART = STEP * D * sizeof(T);      // bytes of K, and of V
    static constexpr int FIT = 24576 * (sizeof(T) / 2) / (2 * PART);
    static constexpr int DEPTH = FIT > 8 ? 8 : FIT;        // bf16 d 128: 3 steps of 8 KB
    static constexpr int BYTES = DEPTH * 2 * PART;
};

// What one warp reads in one unit: steps n = 0, 1, .. of keys first + TILE * n up to end.
template <typename T, int D>
struct Feeder {
    using R = Ring<T, D>;
    static constexpr int AT_ONCE = 32 / R::CH;        // rows that the warp copies at once
    static constexpr int COPIES = STEP / AT_ONCE;     // of a lane, for K and for V
    int s, first, end, steps;
    int64_t slab;     // block of page 0
    uint32_t ring;    // this warp's
    int now, next;    // pages of 32 steps, one a lane: those in use, and the 32 after them; -1: none
    int stage;        // that the next step is copied to
    uint32_t absent;  // bit of a stage: its page is not there

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
    // Asks for step n's rows, n = 0, 1, .. in turn: one group of copies, empty past the last step.
    __device__ __forceinline__ void ask(const AttnParams& P, int n) {
        if (n < steps) {
            if ((n & 31) == 0) {
                if (n > 0) now = next;
                if (n + 32 < steps) next = page_of(P, n + 32);
            }
            const int pid = __shfl_sync(0xffffffffu, now, n & 31);
            const int j = first + TILE * n;
            const int lane = threadIdx.x & 31, row = lane / R::CH, chunk = lane % R::CH;
            const int64_t at = ((slab + static_cast<int64_t>(max(pid, 0)) * P.c.H) << P.c.page_log2) + (j & (P.c.page - 1)) + row;
            const uint32_t dst = ring + stage * 2 * R::PART;
            const bool whole = pid >= 0 && j + STEP <= end;
            absent = pid < 0 ? absent | (1u << stage) : absent & ~(1u << stage);
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                const T* from = static_cast<const T*>(P.c.kv[kv]) + at * D + chunk * (16 / static_cast<int>(sizeof(T)));
#pragma unroll
                for (int i = 0; i < COPIES; ++i) {
                    const uint32_t to = dst + kv * R::PART + 16 * swizzled<R::CH>(row + i * AT_ONCE, chunk);
                    if (whole) copy16(to, from + i * AT_ONCE * D);
                    else copy16_or_zero(to, from + i * AT_ONCE * D, P.c.kv[kv], pid >= 0 && j + row + i * AT_ONCE < end);
                }
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
template <typename T, int D, int NB>
struct Math;

template <int D, int NB>
struct Math<__nv_bfloat16, D, NB> {
    static constexpr int ROWS = 8 * NB, KS = D / 16, SHARED = 0;
    using R = Ring<__nv_bfloat16, D>;
    uint32_t q[NB][KS][2];
    float o[NB][KS][4];
    float m[NB][2], sum[NB][2];
    int qpos[NB][2];

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
    // The step of keys j .. j + 15 at `at` in shared memory; f = scale * log2(e).  whole: all rows see all keys.
    __device__ __forceinline__ void step(uint32_t at, float*, int j, int end, bool whole, bool absent, float f) {
        const int lane = threadIdx.x & 31;
        float sc[NB][4];
#pragma unroll
        for (int b = 0; b < NB; ++b) sc[b][0] = sc[b][1] = sc[b][2] = sc[b][3] = 0.f;
#pragma unroll
        for (int t = 0; t < KS; ++t) {
            uint32_t a[4];
            ldmatrix4(a, at + 16 * swizzled<R::CH>(lane & 15, 2 * t + (lane >> 4)));
#pragma unroll
            for (int b = 0; b < NB; ++b) mma16816(sc[b], a, q[b][t][0], q[b][t][1]);
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
        uint32_t hi[NB][2], lo[NB][2];
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
#pragma unroll
        for (int i = 0; i < KS; ++i) {
            uint32_t a[4];
            ldmatrix4_trans(a, at + R::PART + 16 * swizzled<R::CH>((lane & 7) + 8 * (lane >> 4), 2 * i + ((lane >> 3) & 1)));
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

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {  // two in one instruction
    float2 d;
    asm("{\n\t.reg .b64 x, y, z, w;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float4 shared4(uint32_t p) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(p) : "memory");
    return v;
}

// Scores: lane (r, c) takes quarter c of the dims for keys r and r + 8 and all 8 rows; the quarters
// are added by exchanging halves, which leaves rows 2c and 2c + 1.  Outputs: a lane takes 4 dims of
// all rows for every 32 / (D / 4)-th key.
template <int D>
struct Math<float, D, 1> {
    static constexpr int ROWS = 8, QUARTER = D / 4 + 4;  // 4 floats between: the quarters lie in different banks
    static constexpr int DL = D / 4, KP = 32 / DL;
    static constexpr int SHARED = ROWS * 4 * QUARTER + WARPS * STEP * ROWS;  // floats: queries, weights
    using R = Ring<float, D>;
    float2 o[4][4];  // rows 2i, 2i + 1; dim
    float m[2], sum[2];
    int qpos[2];

    static __device__ __forceinline__ int r() { return threadIdx.x & 7; }
    static __device__ __forceinline__ int c() { return (threadIdx.x & 31) >> 3; }

    template <class Row>
    __device__ __forceinline__ void load(float* shared, int nrows, Row row) {
        for (int i = threadIdx.x; i < ROWS * (D / 4); i += NT) {
            const int y = i / (D / 4), d4 = i % (D / 4);
            const float4 v = y < nrows ? __ldg(reinterpret_cast<const float4*>(row(y)) + d4) : make_float4(0.f, 0.f, 0.f, 0.f);
            *reinterpret_cast<float4*>(shared + (y * 4 + d4 / (D / 16)) * QUARTER + 4 * (d4 % (D / 16))) = v;
        }
    }
    __device__ __forceinline__ void reset(const RowBlock& B, int g) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int x = 0; x < 4; ++x) o[i][x] = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int row = 2 * c() + j;
            m[j] = LOWEST;
            sum[j] = 0.f;
            qpos[j] = row < B.nrows ? B.pos + (B.row0 + row) / g : INT32_MIN;
        }
    }
    __device__ __forceinline__ void step(uint32_t at, float* shared, int j, int end, bool whole, bool absent, float f) {
        const uint32_t sq = smem_u32(shared) + c() * QUARTER * 4;
        float* weights = shared + ROWS * 4 * QUARTER + (threadIdx.x >> 5) * STEP * ROWS;
        float2 acc[2][8];
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int y = 0; y < 8; ++y) acc[k][y] = make_float2(0.f, 0.f);
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
            float4 k[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) k[i] = shared4(at + 16 * swizzled<R::CH>(r() + 8 * i, c() * (D / 16) + x));
#pragma unroll
            for (int y = 0; y < 8; ++y) {
                const float4 v = shared4(sq + (y * 4 * QUARTER + 4 * x) * 4);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    acc[i][y] = fma2(make_float2(k[i].x, k[i].y), make_float2(v.x, v.y), acc[i][y]);
                    acc[i][y] = fma2(make_float2(k[i].z, k[i].w), make_float2(v.z, v.w), acc[i][y]);
                }
            }
        }
        float sc[2][2];  // key, row
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float h[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const float a = acc[i][y].x + acc[i][y].y, b = acc[i][4 + y].x + acc[i][4 + y].y;
                const float keep = c() & 2 ? b : a, give = c() & 2 ? a : b;
                h[y] = keep + __shfl_xor_sync(0xffffffffu, give, 16);
            }
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const float keep = c() & 1 ? h[2 + y] : h[y], give = c() & 1 ? h[y] : h[2 + y];
                sc[i][y] = keep + __shfl_xor_sync(0xffffffffu, give, 8);
            }
        }
        bool raise = false;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                if (!whole) {
                    const int key = j + r() + 8 * i;
                    if (absent || key >= end || key > qpos[y]) sc[i][y] = -INFINITY;
                }
                raise |= sc[i][y] * f > m[y] + MARGIN;
            }
        if (__any_sync(0xffffffffu, raise)) {
            float lower[2];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                float top = fmaxf(sc[0][y], sc[1][y]) * f;
#pragma unroll
                for (int x = 1; x < 8; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                const float up = fmaxf(m[y], top);
                lower[y] = ex2(m[y] - up);
                m[y] = up;
                sum[y] *= lower[y];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a = __shfl_sync(0xffffffffu, lower[0], 8 * i), b = __shfl_sync(0xffffffffu, lower[1], 8 * i);
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    o[i][x].x *= a;
                    o[i][x].y *= b;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float2 w;
            w.x = ex2(fmaf(sc[i][0], f, -m[0]));
            w.y = ex2(fmaf(sc[i][1], f, -m[1]));
            sum[0] += w.x;
            sum[1] += w.y;
            *reinterpret_cast<float2*>(weights + (r() + 8 * i) * ROWS + 2 * c()) = w;
        }
        __syncwarp();
        const int lane = threadIdx.x & 31;
        const uint32_t sw = smem_u32(weights);
#pragma unroll
        for (int i = 0; i < STEP / KP; ++i) {
            const int key = i * KP + lane / DL;
            const float4 v = shared4(at + R::PART + 16 * swizzled<R::CH>(key, lane % DL));
            const float4 a = shared4(sw + key * ROWS * 4), b = shared4(sw + key * ROWS * 4 + 16);
            const float2 w[4] = {make_float2(a.x, a.y), make_float2(a.z, a.w), make_float2(b.x, b.y), make_float2(b.z, b.w)};
            const float vx[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int y = 0; y < 4; ++y)
#pragma unroll
                for (int x = 0; x < 4; ++x) o[y][x] = fma2(w[y], make_float2(vx[x], vx[x]), o[y][x]);
        }
    }
    __device__ __forceinline__ void finish(float* out, float2* stat) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            float t = sum[y];
#pragma unroll
            for (int x = 1; x < 8; x <<= 1) t += __shfl_xor_sync(0xffffffffu, t, x);
            if (r() == 0) stat[2 * c() + y] = make_float2(m[y], t);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
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

// ------------------------------------------------------------------ the kernel

template <typename T, int D, int NB>
constexpr size_t smem_bytes() {
    using M = Math<T, D, NB>;
    static_assert(M::ROWS * D * 4 <= Ring<T, D>::BYTES, "a warp's outputs take its ring's place");
    return WARPS * Ring<T, D>::BYTES + M::SHARED * 4 + WARPS * M::ROWS * sizeof(float2);
}

// Outputs and statistics of one row's parts, each with a reference.
struct Joined {
    float m = LOWEST, sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    __device__ __forceinline__ void reference(float2 st) { m = fmaxf(m, st.x); }
    __device__ __forceinline__ void add(float2 st, float4 o) {
        const float w = ex2(st.x - m);
        sum = fmaf(w, st.y, sum);
        acc.x = fmaf(w, o.x, acc.x);
        acc.y = fmaf(w, o.y, acc.y);
        acc.z = fmaf(w, o.z, acc.z);
        acc.w = fmaf(w, o.w, acc.w);
    }
    __device__ __forceinline__ float4 output() const {
        const float f = sum == 0.f ? 0.f : 1.f / sum;
        return make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
    }
    __device__ __forceinline__ float lse() const { return sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.693147180559945f; }
};

// Row `row` of a unit, in rows with strides and in [n_layers][Hq][T].
struct RowPlace {
    int head, token;
};
__device__ __forceinline__ RowPlace place_of(const AttnParams& P, const RowBlock& B, int h, int row) {
    const int gr = B.row0 + row, i = gr / P.g;
    return RowPlace{h * P.g + (gr - i * P.g), B.tok0 + i};
}
template <typename T>
__device__ __forceinline__ T* address(const Rows& r, int l, RowPlace at) {
    return static_cast<T*>(r.data) + (l * r.l + at.head * r.h + at.token * r.t);
}
template <typename T>
__device__ __forceinline__ void write_row(const AttnParams& P, int l, RowPlace at, int d4, const Joined& z) {
    const int64_t row = (static_cast<int64_t>(l) * P.c.H * P.g + at.head) * P.q.T + at.token;
    if (!KVB_IN_BOUNDS(P.err, row, 1, c8::rows_of(P))) return;
    c8::store_out(address<T>(P.out, l, at) + 4 * d4, z.output());
    if (d4 == 0 && P.lse) P.lse[row] = z.lse();
}

// After a piece of a unit is written: the last CTA of the unit to arrive joins the pieces, in order.
template <typename T, int D, int ROWS>
__device__ __forceinline__ void join_pieces(const AttnParams& P, const RowBlock& B, const Pieces& pieces, int64_t unit, int l, int h,
                                            int* s_last) {
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
        *s_last = false;
        if (KVB_IN_BOUNDS(P.err, unit, 1, P.units) && c8::pieces_in_bounds(P, pieces)) {
            const int n = atomicAdd(P.counters + unit, 1);
            *s_last = n == pieces.n - 1;
            if (n == pieces.n - 1) P.counters[unit] = 0;
        }
    }
    __syncthreads();
    if (!*s_last) return;
    __threadfence();
    for (int i = threadIdx.x; i < B.nrows * (D / 4); i += NT) {
        const int row = i / (D / 4), d4 = i % (D / 4);
        Joined z;
#pragma unroll 8
        for (int p = 0; p < pieces.n; ++p) z.reference(__ldcg(P.part_stat + pieces.slot(p) * ROWS + row));
#pragma unroll 8
        for (int p = 0; p < pieces.n; ++p)
            z.add(__ldcg(P.part_stat + pieces.slot(p) * ROWS + row),
                  __ldcg(reinterpret_cast<const float4*>(P.partial + (pieces.slot(p) * ROWS + row) * D) + d4));
        write_row<T>(P, l, place_of(P, B, h, row), d4, z);
    }
}

template <typename T, int D, int NB>
__global__ void __launch_bounds__(NT) attention_kernel(const __grid_constant__ AttnParams P) {
    using M = Math<T, D, NB>;
    using R = Ring<T, D>;
    constexpr int ROWS = M::ROWS;
    extern __shared__ __align__(128) uint8_t smem[];
    float* shared = reinterpret_cast<float*>(smem + WARPS * R::BYTES);
    float2* stat = reinterpret_cast<float2*>(shared + M::SHARED);  // [WARPS][ROWS]
    __shared__ int s_last;
    __shared__ LineStart s_start;
    __shared__ int s_scan[WARPS];
    const int warp = threadIdx.x >> 5;
    float* mine = reinterpret_cast<float*>(smem + warp * R::BYTES);  // the warp's ring, and later its outputs

    int at, stop, share, l, e, h, first;
    if (!c8::line_start<ROWS, TILE, NT>(P, s_scan, &s_start, at, stop, share, l, e, h, first)) return;
    const int entries = P.q.n_seq * P.row_blocks;
    auto entry = [&](int x) { return c8::row_block(P, x / P.row_blocks, x % P.row_blocks, ROWS); };
    RowBlock B = entry(e);
    int tiles = c8::unit_tiles<TILE>(B);

    for (;;) {  // one unit, or a piece of one, after another
        const int last = min(tiles, first + (stop - at));  // tiles [first, last)
        const int k0 = first * TILE, k1 = min(B.kv_end, last * TILE);
        const int64_t unit = (static_cast<int64_t>(l) * entries + e) * P.c.H + h;

        Feeder<T, D> feed;
        feed.ring = smem_u32(mine);
        feed.begin(P, e / P.row_blocks, (static_cast<int64_t>(P.c.l_begin) + l) * P.c.n_pages * P.c.H + h, k0 + STEP * warp, k1);
        M math;
        math.load(shared, B.nrows, [&](int row) { return address<T>(P.query, l, place_of(P, B, h, row)); });
#pragma unroll
        for (int n = 0; n < R::DEPTH - 1; ++n) feed.ask(P, n);
        math.reset(B, P.g);
        if constexpr (M::SHARED > 0) __syncthreads();  // the queries
        int stage = 0;
        for (int n = 0; n < feed.steps; ++n) {
            copies_wait<R::DEPTH - 2>();
            const bool absent = (feed.absent >> stage) & 1;
            __syncwarp();  // every lane's copies of step n are there, and step n - 1 has been used
            feed.ask(P, n + R::DEPTH - 1);
            const int j = feed.first + TILE * n;
            const bool whole = !absent && j + STEP <= k1 && j + STEP - 1 <= B.pos_lo;
            math.step(feed.ring + stage * 2 * R::PART, shared, j, k1, whole, absent, P.scale_log2);
            stage = stage + 1 == R::DEPTH ? 0 : stage + 1;
        }
        copies_wait<0>();
        __syncwarp();
        math.finish(mine, stat + warp * ROWS);
        __syncthreads();

        // the CTAs that share this unit, and this one's slot
        const int u0 = at - first, c0 = u0 / share;
        const int pieces = (u0 + tiles - 1) / share - c0 + 1;
        const int64_t part0 = (2 * static_cast<int64_t>(blockIdx.x) + (first == 0)) * ROWS;
        for (int i = threadIdx.x; i < B.nrows * (D / 4); i += NT) {
            const int row = i / (D / 4), d4 = i % (D / 4);
            Joined z;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) z.reference(stat[w * ROWS + row]);
#pragma unroll
            for (int w = 0; w < WARPS; ++w)
                z.add(stat[w * ROWS + row], reinterpret_cast<const float4*>(smem + w * R::BYTES + row * D * 4)[d4]);
            if (pieces == 1) {
                write_row<T>(P, l, place_of(P, B, h, row), d4, z);
            } else if (KVB_IN_BOUNDS(P.err, part0 + row, 1, P.slots * ROWS)) {
                reinterpret_cast<float4*>(P.partial + (part0 + row) * D)[d4] = z.acc;
                if (d4 == 0) P.part_stat[part0 + row] = make_float2(z.m, z.sum);
            }
        }
        if (pieces > 1) join_pieces<T, D, ROWS>(P, B, Pieces{pieces, c0}, unit, l, h, &s_last);

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
                tiles = c8::unit_tiles<TILE>(B);
            } while (tiles == 0);
        }
        __syncthreads();  // shared memory is free for the next unit
    }
}

// One instance: CTAs of it that fit an SM (P null), or its launch.
template <typename T, int D, int NB>
cudaError_t instance(const AttnParams* P, int ctas, cudaStream_t s, int* fit) {
    constexpr size_t smem = smem_bytes<T, D, NB>();
    const auto kernel = attention_kernel<T, D, NB>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    if (!P) {
        static const int resident = [&] {
            int n = 0;
            return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, NT, smem) == cudaSuccess ? n : 0;
        }();
        *fit = resident;
        return cudaSuccess;
    }
    kernel<<<ctas, NT, smem, s>>>(*P);
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t instance_rows(int rows, const AttnParams* P, int ctas, cudaStream_t s, int* fit) {
    if constexpr (sizeof(T) == 2) {
        if (rows == 32) return instance<T, D, 4>(P, ctas, s, fit);
        if (rows == 16) return instance<T, D, 2>(P, ctas, s, fit);
    }
    return instance<T, D, 1>(P, ctas, s, fit);
}

template <typename T>
cudaError_t instance_dim(int d, int rows, const AttnParams* P, int ctas, cudaStream_t s, int* fit) {
    switch (d) {
        case 16: return instance_rows<T, 16>(rows, P, ctas, s, fit);
        case 32: return instance_rows<T, 32>(rows, P, ctas, s, fit);
        case 64: return instance_rows<T, 64>(rows, P, ctas, s, fit);
        default: return instance_rows<T, 128>(rows, P, ctas, s, fit);
    }
}

cudaError_t pick(kvb_dtype dtype, int d, int rows, const AttnParams* P, int ctas, cudaStream_t s, int* fit) {
    return dtype == KVB_BF16 ? instance_dim<__nv_bfloat16>(d, rows, P, ctas, s, fit) : instance_dim<float>(d, rows, P, ctas, s, fit);
}

}  // namespace

AttnPlan plan_attention(const Pages& c, const Seqs& q, kvb_dtype dtype, int g, int num_sms) {
    AttnPlan p{};
    const int64_t most = static_cast<int64_t>(q.max_tokens) * g;  // rows of one sequence and head
    const int64_t max_kv = q.max_kv > 0 ? q.max_kv : 1;
    p.rows = dtype == KVB_F32 || most <= 8 ? 8 : most <= 16 ? 16 : 32;
    const double blocks = static_cast<double>((most + p.rows - 1) / p.rows);
    const double units = blocks * c.n_layers * q.n_seq * c.H;
    p.tiles = units * ((max_kv + TILE - 1) / TILE);
    if (p.tiles > static_cast<double>(1 << 30)) return p;  // refused
    p.row_blocks = static_cast<int>(blocks);
    p.units = static_cast<int64_t>(units);
    int fit = 1;
    pick(dtype, c.d, p.rows, nullptr, 0, nullptr, &fit);
    // the CTAs that fit the GPU, no more than the keys give the least share to
    p.min_tiles = MIN_TILES;
    const double need = (p.tiles + p.min_tiles - 1) / p.min_tiles;
    p.ctas = num_sms * (fit > 0 ? fit : 1);
    if (need < p.ctas) p.ctas = static_cast<int>(need) < 1 ? 1 : static_cast<int>(need);
    p.slots = 2 * static_cast<int64_t>(p.ctas);
    p.counter_bytes = (static_cast<size_t>(p.units) * sizeof(int) + 255) / 256 * 256;
    p.partial_bytes = static_cast<size_t>(p.slots) * p.rows * (c.d + 2) * sizeof(float);
    return p;
}

cudaError_t launch_attention(const AttnParams& P, kvb_dtype dtype, const AttnPlan& p, cudaStream_t s) {
    return pick(dtype, P.c.d, p.rows, &P, p.ctas, s, nullptr);
}

}  // namespace paged
}  // namespace kvb
