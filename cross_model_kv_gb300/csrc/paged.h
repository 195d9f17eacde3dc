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
    int* counters;     // [units], 0 before and after a call
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
    size_t counter_bytes, partial_bytes;
};
AttnPlan plan_attention(const Pages& c, const Seqs& q, kvb_dtype dtype, int g, int num_sms);
cudaError_t launch_attention(const AttnParams& P, kvb_dtype dtype, const AttnPlan& p, cudaStream_t s);
cudaError_t launch_attention_rows(const AttnParams& P, const AttnPlan& p, cudaStream_t s, std::string* why);  // bf16, d 64 and 128

}  // namespace paged
}  // namespace kvb
