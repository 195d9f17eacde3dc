// What the entry points of the paged caches share: argument checks, the attention workspace.
#pragma once

#include "cache8.h"
#include "kvb_host.h"

namespace kvb {
namespace c8 {

// A call's sizes, sequences and cache buffers; fills the kernels' view of the sequences.
kvb_status check_call(kvb_ctx* c, int page_tokens, int64_t n_pages, std::initializer_list<const void*> buffers,
                      const kvb_seqs* seqs, int32_t l_begin, int32_t n_layers, kvb_dtype dtype, int64_t T, const char* what,
                      Seqs* sv);
// The same for the 8-bit cache; fills its view too.
kvb_status check_cache8(kvb_ctx* c, const kvb_cache8* cache, const kvb_seqs* seqs, int32_t l_begin, int32_t n_layers,
                        kvb_dtype dtype, int64_t T, const char* what, Cache* cv, Seqs* sv);
// Items of a read or write: (layer, head, sequence, page that its tokens can touch).
bool too_many_blocks(const Cache& c, const Seqs& q);
// Counters (zeroed once; every call leaves them at zero) and partial results of an attention call.
kvb_status ensure_attn_ws(kvb_ctx* c, size_t counter_bytes, size_t part_bytes, const char* what, cudaStream_t s);

inline int log2_of(int x) { return x == 16 ? 4 : x == 32 ? 5 : x == 64 ? 6 : 7; }
inline bool empty_call(const Seqs& q, int n_layers) {
    return q.T == 0 || q.n_seq == 0 || n_layers == 0 || q.max_tokens == 0;
}
inline Err call_err(const kvb_ctx* c) { return Err{c->err_dev, c->err_mirror, c->timeout_ns}; }

}  // namespace c8
}  // namespace kvb
