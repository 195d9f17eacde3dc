// Entry points of the paged 8-bit cache: argument checks, workspace, launches.
#include <cmath>

#include "cache8.h"
#include "kvb_host.h"

using namespace kvb;

namespace {

// What the three calls check alike; fills the kernels' views.
kvb_status check_call(kvb_ctx* c, const kvb_cache8* cache, const kvb_seqs* seqs, int32_t l_begin, int32_t n_layers,
                      kvb_dtype dtype, int64_t T, const char* what, c8::Cache* cv, c8::Seqs* sv) {
    const std::string w(what);
    if (!c) return fail(KVB_ERR_INVALID_ARG, "ctx is NULL");
    if (!cache || !seqs) return fail(KVB_ERR_INVALID_ARG, w + ": cache or seqs is NULL");
    if (dtype != KVB_F32 && dtype != KVB_BF16) return fail(KVB_ERR_UNSUPPORTED, "dtype must be KVB_F32 or KVB_BF16");
    if (c->d != 16 && c->d != 32 && c->d != 64 && c->d != 128)
        return fail(KVB_ERR_UNSUPPORTED, w + " supports head_dim 16, 32, 64 or 128");
    const int pt = cache->page_tokens;
    if (pt != 16 && pt != 32 && pt != 64 && pt != 128)
        return fail(KVB_ERR_UNSUPPORTED, w + ": page_tokens must be 16, 32, 64 or 128");
    if (cache->n_pages < 0 || cache->n_pages > 0x7fffffffLL) return fail(KVB_ERR_INVALID_ARG, w + ": bad n_pages");
    if (l_begin < 0 || n_layers < 0 || l_begin > c->L_t - n_layers)
        return fail(KVB_ERR_INVALID_ARG, w + ": layers outside [0, L_tgt)");
    if (T < 0) return fail(KVB_ERR_INVALID_ARG, "T < 0");
    if (T > 0x7fffffffLL) return fail(KVB_ERR_UNSUPPORTED, "T above 2^31-1");
    if (seqs->n_seq < 0 || seqs->max_pages < 0 || seqs->max_tokens < 0 || seqs->max_kv < 0)
        return fail(KVB_ERR_INVALID_ARG, w + ": negative size in seqs");
    if (seqs->max_tokens > T) return fail(KVB_ERR_INVALID_ARG, w + ": max_tokens above T");
    kvb_status st;
    if ((st = take_device_error(c)) != KVB_OK) return st;
    if (T > 0 && seqs->n_seq > 0 && n_layers > 0 && seqs->max_tokens > 0) {
        if ((st = check_device_ptrs({cache->k, cache->v, cache->k_scale, cache->v_scale}, what)) != KVB_OK) return st;
        for (const int32_t* p : {seqs->page_table, seqs->seq_off, seqs->seq_pos}) {
            if (!p) return fail(KVB_ERR_INVALID_ARG, w + ": null device pointer in seqs");
            if (reinterpret_cast<uintptr_t>(p) & 3u)
                return fail(KVB_ERR_INVALID_ARG, w + ": device pointer in seqs not 4-byte aligned");
        }
        if (reinterpret_cast<uintptr_t>(seqs->kv_len) & 3u)
            return fail(KVB_ERR_INVALID_ARG, w + ": device pointer in seqs not 4-byte aligned");
    }
    cv->code[0] = static_cast<uint8_t*>(cache->k);
    cv->code[1] = static_cast<uint8_t*>(cache->v);
    cv->scale[0] = cache->k_scale;
    cv->scale[1] = cache->v_scale;
    cv->n_pages = cache->n_pages;
    cv->H = c->H;
    cv->d = c->d;
    cv->d_log2 = c->d == 16 ? 4 : c->d == 32 ? 5 : c->d == 64 ? 6 : 7;
    cv->page = pt;
    cv->page_log2 = pt == 16 ? 4 : pt == 32 ? 5 : pt == 64 ? 6 : 7;
    cv->l_begin = l_begin;
    cv->n_layers = n_layers;
    sv->page_table = seqs->page_table;
    sv->off = seqs->seq_off;
    sv->pos = seqs->seq_pos;
    sv->kv_len = seqs->kv_len;
    sv->n_seq = seqs->n_seq;
    sv->max_pages = seqs->max_pages;
    sv->max_tokens = seqs->max_tokens;
    const int64_t room = static_cast<int64_t>(seqs->max_pages) * pt;
    const int64_t kv = seqs->max_kv > 0 && seqs->max_kv < room ? seqs->max_kv : room;
    if (kv > c8::MAX_KEYS) return fail(KVB_ERR_UNSUPPORTED, w + ": more than 2^31 - 1024 cache positions in a sequence");
    sv->max_kv = static_cast<int>(kv);
    sv->T = T;
    return KVB_OK;
}

bool empty(const c8::Cache& c, const c8::Seqs& q) {
    return q.T == 0 || q.n_seq == 0 || c.n_layers == 0 || q.max_tokens == 0;
}

c8::Err call_err(const kvb_ctx* c) { return c8::Err{c->err_dev, c->err_mirror, c->timeout_ns}; }

// Items of a read or write: (layer, head, sequence, page that its tokens can touch).
bool too_many_blocks(const c8::Cache& c, const c8::Seqs& q) {
    const double items = (static_cast<double>(q.max_tokens) + c.page - 2) / c.page + 1;
    return items * q.n_seq * c.H * c.n_layers > 2147483647.0;
}

// One buffer of the attention workspace made large enough, with room for calls to come; the
// old one is kept until the context goes (its sizes grow by a quarter at least, so all of
// them together stay within five times the last).
kvb_status grow(kvb_ctx* c, void** buf, size_t* have, size_t need, size_t bytes, bool zeroed, cudaStream_t s) {
    if (need <= *have) return KVB_OK;
    cudaStreamCaptureStatus capturing = cudaStreamCaptureStatusNone;
    cudaError_t e = cudaStreamIsCapturing(s, &capturing);
    if (e != cudaSuccess) return cuda_fail(e, "growing the attention workspace");
    if (capturing != cudaStreamCaptureStatusNone)
        return fail(KVB_ERR_UNSUPPORTED,
                    "kvb_cache8_attention: the workspace would have to grow on a stream that is being captured; make this call once before");
    try {
        c->attn_outgrown.reserve(c->attn_outgrown.size() + 1);
    } catch (...) {
        return fail(KVB_ERR_OOM, "host allocation failed");
    }
    void* p = nullptr;
    if ((e = cudaMalloc(&p, bytes)) != cudaSuccess) return cuda_fail(e, "cudaMalloc attention workspace");
    if (zeroed && (e = cudaMemsetAsync(p, 0, bytes, s)) != cudaSuccess) {
        cudaFree(p);
        return cuda_fail(e, "zeroing the attention workspace");
    }
    if (*buf) c->attn_outgrown.push_back(*buf);
    *buf = p;
    *have = bytes;
    return KVB_OK;
}

// Counters (zeroed once; every call leaves them at zero), and the partial outputs with what is noted of units.
kvb_status ensure_attn_ws(kvb_ctx* c, const c8::AttnPlan& p, cudaStream_t s) {
    const size_t parts = p.partial_bytes + p.unit_bytes;
    const kvb_status st = grow(c, &c->attn_counters, &c->attn_counters_bytes, p.counter_bytes,
                               p.counter_bytes < 65536 ? 65536 : 2 * p.counter_bytes, true, s);
    return st != KVB_OK ? st : grow(c, &c->attn_parts, &c->attn_parts_bytes, parts, parts + parts / 4, false, s);
}

}  // namespace

extern "C" {

kvb_status kvb_cache8_write(kvb_ctx* c, const kvb_cache8* cache, const kvb_seqs* seqs, int32_t l_begin,
                            int32_t n_layers, kvb_dtype dtype, const void* k, const void* v, int64_t T, void* stream) {
    g_last_error.clear();
    c8::Cache cv{};
    c8::Seqs sv{};
    kvb_status st = check_call(c, cache, seqs, l_begin, n_layers, dtype, T, "kvb_cache8_write", &cv, &sv);
    if (st != KVB_OK) return st;
    if (empty(cv, sv)) return KVB_OK;
    if ((st = check_device_ptrs({k, v}, "kvb_cache8_write")) != KVB_OK) return st;
    if (too_many_blocks(cv, sv)) return fail(KVB_ERR_UNSUPPORTED, "kvb_cache8_write: more than 2^31-1 blocks in one call");
    DeviceGuard g(c->device);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    ProfScope ps(c, s, "cache8_write");
    const cudaError_t e = c8::launch_write(cv, sv, dtype, k, v, call_err(c), s);
    return e == cudaSuccess ? KVB_OK : cuda_fail(e, "cache8 write launch");
}

kvb_status kvb_cache8_read(kvb_ctx* c, const kvb_cache8* cache, const kvb_seqs* seqs, int32_t l_begin,
                           int32_t n_layers, kvb_dtype dtype, void* k, void* v, int64_t T, void* stream) {
    g_last_error.clear();
    c8::Cache cv{};
    c8::Seqs sv{};
    kvb_status st = check_call(c, cache, seqs, l_begin, n_layers, dtype, T, "kvb_cache8_read", &cv, &sv);
    if (st != KVB_OK) return st;
    if (empty(cv, sv)) return KVB_OK;
    if ((st = check_device_ptrs({k, v}, "kvb_cache8_read")) != KVB_OK) return st;
    if (too_many_blocks(cv, sv)) return fail(KVB_ERR_UNSUPPORTED, "kvb_cache8_read: more than 2^31-1 blocks in one call");
    DeviceGuard g(c->device);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    ProfScope ps(c, s, "cache8_read");
    const cudaError_t e = c8::launch_read(cv, sv, dtype, k, v, call_err(c), s);
    return e == cudaSuccess ? KVB_OK : cuda_fail(e, "cache8 read launch");
}

kvb_status kvb_cache8_attention(kvb_ctx* c, const kvb_cache8* cache, const kvb_seqs* seqs, int32_t l_begin,
                                int32_t n_layers, kvb_dtype dtype, const void* q, int32_t n_q_heads, int64_t T,
                                double scale, void* out, float* lse, void* stream) {
    g_last_error.clear();
    c8::AttnParams a{};
    kvb_status st = check_call(c, cache, seqs, l_begin, n_layers, dtype, T, "kvb_cache8_attention", &a.c, &a.q);
    if (st != KVB_OK) return st;
    if (n_q_heads < c->H || n_q_heads % c->H)
        return fail(KVB_ERR_INVALID_ARG, "n_q_heads must be a positive multiple of the KV heads");
    if (!(scale >= 0.0) || !std::isfinite(scale)) return fail(KVB_ERR_INVALID_ARG, "scale must be finite and >= 0");
    if (empty(a.c, a.q)) return KVB_OK;
    if ((st = check_device_ptrs({q, out}, "kvb_cache8_attention")) != KVB_OK) return st;
    if (reinterpret_cast<uintptr_t>(lse) & 3u)
        return fail(KVB_ERR_INVALID_ARG, "kvb_cache8_attention: lse not 4-byte aligned");
    DeviceGuard g(c->device);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    a.query = q;
    a.out = out;
    a.lse = lse;
    a.g = n_q_heads / c->H;
    a.scale_log2 = static_cast<float>((scale > 0.0 ? scale : 1.0 / std::sqrt(static_cast<double>(c->d))) * 1.4426950408889634);
    a.err = call_err(c);
    const c8::AttnPlan p = c8::plan_attention(a.c, a.q, dtype, a.g, c->num_sms);
    // the kernels count rows of a sequence, units and tiles of 64 or 128 keys in 32 bits
    constexpr double most = 1 << 30;
    if (static_cast<double>(p.units) * (p.tensor ? 8 : 1) > most || p.tiles > most || static_cast<double>(a.q.max_tokens) * a.g > most)
        return fail(KVB_ERR_UNSUPPORTED, "kvb_cache8_attention: more query rows, sequences, layers or keys than one call takes (2^30 tiles of 64 keys)");
    if ((st = ensure_attn_ws(c, p, s)) != KVB_OK) return st;
    a.counters = static_cast<int*>(c->attn_counters);  // the tcgen05 kernel has no use for them
    a.partial = static_cast<float*>(c->attn_parts);
    a.shared_by = reinterpret_cast<int2*>(static_cast<char*>(c->attn_parts) + p.partial_bytes);
    a.part_stat = reinterpret_cast<float4*>(a.partial + static_cast<size_t>(p.slots) * p.rows * c->d);
    a.units = p.units;
    a.slots = p.slots;
    a.row_blocks = p.row_blocks;
    a.min_tiles = p.min_tiles;
    ProfScope ps(c, s, p.tensor ? "cache8_attention_tcgen05" : "cache8_attention");
    const cudaError_t e = p.tensor ? c8::launch_prefill(a, p, s) : c8::launch_decode(a, dtype, p, s);
    return e == cudaSuccess ? KVB_OK : cuda_fail(e, "cache8 attention launch");
}

}  // extern "C"
