// Entry points of the paged cache of the model's own type and of the appends with rotation:
// argument checks, workspace, launches.
#include <cmath>

#include "cache_host.h"
#include "paged.h"

using namespace kvb;

namespace {

// A call's body; what it throws becomes a status.
template <class F>
kvb_status guarded(F&& f) {
    try {
        g_last_error.clear();
        return f();
    } catch (const std::exception&) {
        return KVB_ERR_OOM;  // the only one thrown below: host memory for a message or a record ran out
    }
}

size_t bytes_of(kvb_dtype dtype) { return dtype == KVB_BF16 ? 2 : 4; }

// One kvb_rows of `heads` heads; written: rows of different (layer, head, token) must not overlap.
kvb_status check_rows(const kvb_rows* r, const char* name, const char* what, int n_layers, int heads, int64_t T, int d,
                      kvb_dtype dtype, bool written, paged::Rows* out) {
    const std::string w = std::string(what) + ": " + name;
    if (!r || !r->data) return fail(KVB_ERR_INVALID_ARG, w + " is NULL");
    if (!aligned16(r->data)) return fail(KVB_ERR_INVALID_ARG, w + " is not 16-byte aligned");
    const int64_t unit = 16 / static_cast<int64_t>(bytes_of(dtype));
    struct Axis {
        int64_t size, stride;
    } axis[3] = {{n_layers, r->layer}, {heads, r->head}, {T, r->token}};
    for (Axis& a : axis) {
        if (a.size <= 1) a.stride = 0;  // one index: the stride means nothing
        if (a.stride % unit) return fail(KVB_ERR_INVALID_ARG, w + " has a stride that is not a multiple of 16 bytes");
        if (a.stride < 0 || static_cast<double>(a.stride) * static_cast<double>(a.size) > 1e18)  // three of them, in bytes, in 64 bits
            return fail(KVB_ERR_INVALID_ARG, w + " has a stride that is negative or too large");
    }
    out->data = r->data;
    out->l = axis[0].stride;
    out->h = axis[1].stride;
    out->t = axis[2].stride;
    if (written) {  // each axis steps over all that the axes of smaller stride cover
        for (int i = 0; i < 2; ++i)
            for (int j = 0; j + 1 < 3; ++j)
                if (axis[j].stride > axis[j + 1].stride) std::swap(axis[j], axis[j + 1]);
        int64_t covered = d;
        for (const Axis& a : axis) {
            if (a.size <= 1) continue;
            if (a.stride < covered) return fail(KVB_ERR_INVALID_ARG, w + " has rows that overlap");
            covered += a.stride * (a.size - 1);
        }
    }
    return KVB_OK;
}

kvb_status check_paged(kvb_ctx* c, const kvb_paged_cache* cache, const kvb_seqs* seqs, int32_t l_begin, int32_t n_layers,
                       int64_t T, const char* what, paged::Pages* pv, c8::Seqs* sv) {
    if (!c) return fail(KVB_ERR_INVALID_ARG, "ctx is NULL");
    if (!cache || !seqs) return fail(KVB_ERR_INVALID_ARG, std::string(what) + ": cache or seqs is NULL");
    const kvb_status st = c8::check_call(c, cache->page_tokens, cache->n_pages, {cache->k, cache->v}, seqs, l_begin, n_layers,
                                         cache->dtype, T, what, sv);
    if (st != KVB_OK) return st;
    *pv = paged::Pages{{cache->k, cache->v}, cache->n_pages, c->H, c->d, c8::log2_of(c->d), cache->page_tokens,
                       c8::log2_of(cache->page_tokens), l_begin, n_layers};
    return KVB_OK;
}

// What the two appends check alike after their caches; fills the rows.
kvb_status check_append(kvb_ctx* c, const kvb_rows* k, const kvb_rows* v, const kvb_rows* q, const kvb_rows* q_out,
                        int32_t n_q_heads, kvb_dtype dtype, int32_t rotate, const char* what, paged::AppendParams* P) {
    const std::string w(what);
    if (rotate != 0 && rotate != 1) return fail(KVB_ERR_INVALID_ARG, w + ": rotate must be 0 or 1");
    if (!q != !q_out) return fail(KVB_ERR_INVALID_ARG, w + ": q and q_out go together");
    if (q && !rotate) return fail(KVB_ERR_INVALID_ARG, w + ": queries need rotate = 1");
    if (q && (n_q_heads < c->H || n_q_heads % c->H))
        return fail(KVB_ERR_INVALID_ARG, "n_q_heads must be a positive multiple of the KV heads");
    P->rotate = rotate != 0;
    P->Hq = q ? n_q_heads : 0;
    P->tab = c->tab_t;
    P->max_pos = c->max_pos;
    P->err = c8::call_err(c);
    if (c8::empty_call(P->q, P->c.n_layers)) return KVB_OK;
    kvb_status st;
    const int L = P->c.n_layers;
    const int64_t T = P->q.T;
    if ((st = check_rows(k, "k", what, L, c->H, T, c->d, dtype, false, &P->src[0])) != KVB_OK) return st;
    if ((st = check_rows(v, "v", what, L, c->H, T, c->d, dtype, false, &P->src[1])) != KVB_OK) return st;
    if (q) {
        if ((st = check_rows(q, "q", what, L, n_q_heads, T, c->d, dtype, false, &P->qs)) != KVB_OK) return st;
        if ((st = check_rows(q_out, "q_out", what, L, n_q_heads, T, c->d, dtype, true, &P->qo)) != KVB_OK) return st;
        if (P->qs.data == P->qo.data && (P->qs.l != P->qo.l || P->qs.h != P->qo.h || P->qs.t != P->qo.t))
            return fail(KVB_ERR_INVALID_ARG, w + ": q_out in the place of q needs its strides");
    }
    if (paged::append_ctas(*P, dtype, c->num_sms) > 2147483647.0)
        return fail(KVB_ERR_UNSUPPORTED, w + ": more layers, sequences and tokens than one call takes (2^31 - 1 blocks)");
    return KVB_OK;
}

}  // namespace

extern "C" {

kvb_status kvb_paged_append(kvb_ctx* c, const kvb_paged_cache* cache, const kvb_seqs* seqs, int32_t l_begin,
                            int32_t n_layers, const kvb_rows* k, const kvb_rows* v, const kvb_rows* q, const kvb_rows* q_out,
                            int32_t n_q_heads, int64_t T, int32_t rotate, void* stream) {
    return guarded([&] {
        const char* what = "kvb_paged_append";
        paged::AppendParams P{};
        kvb_status st = check_paged(c, cache, seqs, l_begin, n_layers, T, what, &P.c, &P.q);
        if (st != KVB_OK) return st;
        if ((st = check_append(c, k, v, q, q_out, n_q_heads, cache->dtype, rotate, what, &P)) != KVB_OK) return st;
        if (c8::empty_call(P.q, n_layers)) return KVB_OK;
        DeviceGuard g(c->device);
        cudaStream_t s = static_cast<cudaStream_t>(stream);
        ProfScope ps(c, s, "paged_append");
        const cudaError_t e = paged::launch_append(P, cache->dtype, c->num_sms, s);
        return e == cudaSuccess ? KVB_OK : cuda_fail(e, "paged append launch");
    });
}

kvb_status kvb_cache8_append(kvb_ctx* c, const kvb_cache8* cache, const kvb_seqs* seqs, int32_t l_begin, int32_t n_layers,
                             kvb_dtype dtype, const kvb_rows* k, const kvb_rows* v, const kvb_rows* q, const kvb_rows* q_out,
                             int32_t n_q_heads, int64_t T, int32_t rotate, void* stream) {
    return guarded([&] {
        const char* what = "kvb_cache8_append";
        paged::AppendParams P{};
        c8::Cache cv{};
        kvb_status st = c8::check_cache8(c, cache, seqs, l_begin, n_layers, dtype, T, what, &cv, &P.q);
        if (st != KVB_OK) return st;
        P.c = paged::Pages{{nullptr, nullptr}, cv.n_pages, cv.H, cv.d, cv.d_log2, cv.page, cv.page_log2, l_begin, n_layers};
        if ((st = check_append(c, k, v, q, q_out, n_q_heads, dtype, rotate, what, &P)) != KVB_OK) return st;
        if (c8::empty_call(P.q, n_layers)) return KVB_OK;
        if (c8::too_many_blocks(cv, P.q))
            return fail(KVB_ERR_UNSUPPORTED, "kvb_cache8_append: more than 2^31-1 blocks in one call");
        DeviceGuard g(c->device);
        cudaStream_t s = static_cast<cudaStream_t>(stream);
        ProfScope ps(c, s, "cache8_append");
        const cudaError_t e = paged::launch_append8(P, cv, dtype, c->num_sms, s);
        return e == cudaSuccess ? KVB_OK : cuda_fail(e, "cache8 append launch");
    });
}

kvb_status kvb_paged_attention(kvb_ctx* c, const kvb_paged_cache* cache, const kvb_seqs* seqs, int32_t l_begin,
                               int32_t n_layers, const kvb_rows* q, int32_t n_q_heads, int64_t T, double scale,
                               const kvb_rows* out, float* lse, void* stream) {
    return guarded([&] {
        const char* what = "kvb_paged_attention";
        paged::AttnParams a{};
        kvb_status st = check_paged(c, cache, seqs, l_begin, n_layers, T, what, &a.c, &a.q);
        if (st != KVB_OK) return st;
        if (n_q_heads < c->H || n_q_heads % c->H)
            return fail(KVB_ERR_INVALID_ARG, "n_q_heads must be a positive multiple of the KV heads");
        if (!(scale >= 0.0) || !std::isfinite(scale)) return fail(KVB_ERR_INVALID_ARG, "scale must be finite and >= 0");
        if (c8::empty_call(a.q, n_layers)) return KVB_OK;
        if ((st = check_rows(q, "q", what, n_layers, n_q_heads, T, c->d, cache->dtype, false, &a.query)) != KVB_OK) return st;
        if ((st = check_rows(out, "out", what, n_layers, n_q_heads, T, c->d, cache->dtype, true, &a.out)) != KVB_OK) return st;
        if (out->data == q->data) return fail(KVB_ERR_INVALID_ARG, "kvb_paged_attention: out in the place of q");
        if (reinterpret_cast<uintptr_t>(lse) & 3u)
            return fail(KVB_ERR_INVALID_ARG, "kvb_paged_attention: lse not 4-byte aligned");
        DeviceGuard g(c->device);
        cudaStream_t s = static_cast<cudaStream_t>(stream);
        a.lse = lse;
        a.g = n_q_heads / c->H;
        a.scale_log2 = static_cast<float>((scale > 0.0 ? scale : 1.0 / std::sqrt(static_cast<double>(c->d))) * 1.4426950408889634);
        if (!(a.scale_log2 > 0.f) || !std::isfinite(a.scale_log2))
            return fail(KVB_ERR_INVALID_ARG, "scale outside the range of fp32");
        a.err = c8::call_err(c);
        const paged::AttnPlan p = paged::plan_attention(a.c, a.q, cache->dtype, a.g, c->num_sms);
        // the kernel counts rows of a sequence, units and tiles of 64 keys in 32 bits
        constexpr double most = 1 << 30;
        if (static_cast<double>(p.units) > most || p.tiles > most || static_cast<double>(a.q.max_tokens) * a.g > most)
            return fail(KVB_ERR_UNSUPPORTED, "kvb_paged_attention: more query rows, sequences, layers or keys than one call takes (2^30 tiles of 64 keys)");
        if (!p.cluster && (st = c8::ensure_attn_ws(c, p.counter_bytes, p.partial_bytes + p.shared_bytes, what, s)) != KVB_OK) return st;
        a.counters = static_cast<int*>(c->attn_counters);
        a.partial = static_cast<float*>(c->attn_parts);
        a.part_stat = reinterpret_cast<float2*>(a.partial + static_cast<size_t>(p.slots) * p.rows * c->d);
        a.shared = reinterpret_cast<int4*>(static_cast<char*>(c->attn_parts) + p.partial_bytes);
        a.units = p.units;
        a.slots = p.slots;
        a.row_blocks = p.row_blocks;
        a.min_tiles = p.min_tiles;
        a.cluster = p.cluster;
        std::string why;
        ProfScope ps(c, s, p.tensor ? "paged_attention_tcgen05" : "paged_attention");
        const cudaError_t e = p.tensor ? paged::launch_attention_rows(a, p, s, &why) : paged::launch_attention(a, cache->dtype, p, s);
        if (e != cudaSuccess && !why.empty()) return fail(KVB_ERR_CUDA, "paged attention launch: " + why);
        return e == cudaSuccess ? KVB_OK : cuda_fail(e, "paged attention launch");
    });
}

}  // extern "C"
