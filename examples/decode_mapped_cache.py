#!/usr/bin/env python
"""Decode from a mapped cache kept in 8 bits.

A source model's prefilled cache is mapped to the target model (kvb_map_apply)
and stored in the paged 8-bit cache (kvb_cache8_write).  Then the target decodes:
for every new token and layer its key and value are written into the cache and
its queries attend over it (kvb_cache8_attention).  At the end the 8-bit cache is
read back (kvb_cache8_read) and its attention outputs are compared with those of
the bf16 cache (kvb_attention_cosine).

Synthetic data of the given shapes stands in for the two models: the queries, keys
and values that a model would compute for each new token are random draws.

    python examples/decode_mapped_cache.py [--layers-src 8 --layers-tgt 12 --prefix 4096 --tokens 64]
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import cross_model_kv_gb300 as kvb  # noqa: E402
import synth  # noqa: E402


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layers-src", type=int, default=8)
    ap.add_argument("--layers-tgt", type=int, default=12)
    ap.add_argument("--kv-heads", type=int, default=8)
    ap.add_argument("--q-heads", type=int, default=64)
    ap.add_argument("--prefix", type=int, default=4096)
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--page", type=int, default=64)
    a = ap.parse_args(argv)
    L_s, L_t, H, Hq, d, k, T = a.layers_src, a.layers_tgt, a.kv_heads, a.q_heads, 128, 4, a.prefix
    dev, bf = "cuda", torch.bfloat16
    spec = lambda n: {"n_layers": n, "n_kv_heads": H, "head_dim": d, "rope_theta": 1e6}
    total = T + a.tokens
    ctx = kvb.kvb_ctx_create(spec(L_s), spec(L_t), k, total)

    # the source's prefix, mapped to the target
    src_k, src_v = (synth.torch_content(s, L_s, H, T, d, 0.5, bf, dev) for s in (1, 2))
    sel = synth.hidden_selection(3, L_s, L_t, k)
    (W_k, b_k), (W_v, b_v) = (synth.torch_weights(s, L_t, k * H * d, H * d, bf, dev) for s in (4, 5))
    pos = torch.arange(T, dtype=torch.int32, device=dev)
    map_k, map_v = (torch.empty((L_t, H, T, d), dtype=bf, device=dev) for _ in range(2))
    kvb.kvb_map_apply(ctx, src_k, src_v, pos, sel, sel, W_k, W_v, b_k, b_v, map_k, map_v)

    # stored in 8 bits: one sequence, its pages in any order
    n_pages = -(-total // a.page)
    cache = kvb.kvb_cache8_create(ctx, n_pages, a.page)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    table = torch.randperm(n_pages, device=dev).to(torch.int32)[None]
    kvb.kvb_cache8_write(ctx, cache, kvb.Seqs(table, i32([0, T]), i32([0]), max_tokens=T), map_k, map_v)

    # decoding: the call's tensors stay in place, only the position moves on
    new_k, new_v = (synth.torch_content(s, L_t, H, a.tokens, d, 0.5, bf, dev) for s in (6, 7))
    new_q = synth.torch_content(8, L_t, Hq, a.tokens, d, 0.5, bf, dev)
    at = i32([T])
    seqs = kvb.Seqs(table, i32([0, 1]), at, max_tokens=1, max_kv=total)
    tok_k, tok_v = (torch.empty((1, H, 1, d), dtype=bf, device=dev) for _ in range(2))
    tok_q = torch.empty((1, Hq, 1, d), dtype=bf, device=dev)
    out = torch.empty((L_t, Hq, a.tokens, d), dtype=bf, device=dev)
    o = torch.empty_like(tok_q)

    def token(i):
        for l in range(L_t):
            tok_k.copy_(new_k[l:l + 1, :, i:i + 1])
            tok_v.copy_(new_v[l:l + 1, :, i:i + 1])
            tok_q.copy_(new_q[l:l + 1, :, i:i + 1])
            kvb.kvb_cache8_write(ctx, cache, seqs, tok_k, tok_v, l_begin=l)
            kvb.kvb_cache8_attention(ctx, cache, seqs, tok_q, o, l_begin=l)
            out[l, :, i].copy_(o[0, :, 0])
        at.add_(1)

    t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    t0.record()
    for i in range(a.tokens):
        token(i)
    t1.record()
    torch.cuda.synchronize()
    kvb.kvb_ctx_check(ctx)

    # the 8-bit cache against the bf16 one, every decoded token a query
    whole = kvb.Seqs(table, i32([0, total]), i32([0]), max_tokens=total)
    back_k, back_v = (torch.empty((L_t, H, total, d), dtype=bf, device=dev) for _ in range(2))
    kvb.kvb_cache8_read(ctx, cache, whole, back_k, back_v)
    full_k, full_v = torch.cat([map_k, new_k], dim=2), torch.cat([map_v, new_v], dim=2)
    cos = torch.empty((L_t, Hq, a.tokens), device=dev)
    where = torch.arange(total, dtype=torch.int32, device=dev)
    kvb.kvb_attention_cosine(ctx, new_q, where[T:].contiguous(), back_k, back_v, full_k, full_v, where, cos)
    torch.cuda.synchronize()
    kvb.kvb_ctx_check(ctx)
    bits8, bits16 = (cache.k.numel() + cache.v.numel()) / 2 ** 20, 2 * (full_k.numel() + full_v.numel()) / 2 ** 20
    print(f"{T} mapped + {a.tokens} decoded tokens, {L_t} layers: cache {bits8:.1f} MiB in 8 bits, {bits16:.1f} MiB in bf16")
    print(f"{t0.elapsed_time(t1) / a.tokens:.3f} ms a token (write + attention, {L_t} layers)")
    print(f"attention-output cosine, 8 bits against bf16: mean {cos.mean():.5f}, min {cos.min():.5f}")
    return {"cos_mean": float(cos.mean()), "cos_min": float(cos.min()), "out": out}


if __name__ == "__main__":
    main()
