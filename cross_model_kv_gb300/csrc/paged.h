// Paged cache of the model's own type, rows with strides, and what the kernels that append to
// the two paged caches share.
#pragma once

#include "cache8.h"

namespace kvb {
namespace paged {

using c8::Err;
using c8::Seqs;

struct Pages {
    void* kv[2];  // [layer][page][kv head][slot][dim]
    int64_t n_pages;
    int H, d, d_log2, page, page_log2;
    int l_begin, n_layers;
};

// Element e of (layer, head, token) at data + layer * l + head * h + token * t + e.
struct Rows {
    void* data;
    int64_t l, h, t;
};

struct AppendParams {
    Pages c;       // pages of the model's type; for the 8-bit cache only its sizes
    Seqs q;
    Rows src[2];   // k, v
    Rows qs, qo;   // queries, or null data
    int Hq;        // 0 without queries
    bool rotate;
    const float2* tab;  // cos, sin [max_pos][d/2]
    int max_pos;
    Err err;
};

cudaError_t launch_append(const AppendParams& P, kvb_dtype dtype, int num_sms, cudaStream_t s);
cudaError_t launch_append8(const AppendParams& P, const c8::Cache& c, kvb_dtype dtype, int num_sms, cudaStream_t s);
// CTAs of the two launches (they have to stay below 2^31).
double append_ctas(const AppendParams& P, kvb_dtype dtype, int num_sms);

// Tiles that a unit itself counts as in the tcgen05 kernel's line: its first scores, its outputs and the hand-overs between
// take about as long.  64 sequences of up to 2000 keys, 8 heads, 0 / 4 / 8 tiles: 24 rows 84 / 62 / 65 us, 40 rows
// 156 / 80 / 78, 64 rows 180 / 108 / 97; 16 of 8192 each 94 / 94 / 96, 96 / 98 / 101, 104 / 104 / 104.
constexpr int unit_tiles_of(int rows) { return rows <= 48 ? 4 : 8; }

struct AttnParams {
    Pages c;
    Seqs q;
    Rows query, out;
    float* lse;  // [n_layers][Hq][T], or null
    int g;       // query heads of a KV head
    int row_blocks;
    int min_tiles;     // a CTA's least share of the line of tiles
    int cluster;       // CTAs of a unit's cluster, a power of two, or 0: the line
    float scale_log2;  // scale * log2(e)
    int* counters;     // [units], 0 before and after a call of the line
    int4* shared;      // tcgen05: [ctas][2], the unit that begins in a CTA and ends in another: pieces (0: none), rows,
                       // first row, first token; layer, head
    float* partial;    // [slots][rows][d]
    float2* part_stat; // [slots][rows] reference, sum
    int64_t units, slots;
    Err err;
};

// How a call is cut: blocks of `rows` query rows, and their keys over CTAs.
struct AttnPlan {
    bool tensor;  // the tcgen05 kernel
    int rows, row_blocks, min_tiles, cluster, ctas;
    int64_t units, slots;
    double tiles;
    size_t counter_bytes, partial_bytes, shared_bytes;
};
AttnPlan plan_attention(const Pages& c, const Seqs& q, kvb_dtype dtype, int g, int num_sms);
cudaError_t launch_attention(const AttnParams& P, kvb_dtype dtype, const AttnPlan& p, cudaStream_t s);
cudaError_t launch_attention_rows(const AttnParams& P, const AttnPlan& p, cudaStream_t s, std::string* why);  // bf16, d 64 and 128

}  // namespace paged
}  // namespace kvb
