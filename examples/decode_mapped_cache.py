#!/usr/bin/env python
"""Decode from a mapped cache.

A source model's prefilled cache is mapped to the target model (kvb_map_apply) and
stored in a paged cache: in 8 bits (kvb_cache8_write) or, with --cache model, in the
model's own type (kvb_paged_append).  Then the target decodes: for every new token and
layer its projection's output, q, k and v heads in one row and no RoPE yet, is appended
with the rotation on the way (kvb_cache8_append, kvb_paged_append) and its rotated
queries attend over the cache (kvb_cache8_attention, kvb_paged_attention).  At the end
the cache is read back and its attention outputs are compared with those of a plain bf16
cache that torch has rotated (kvb_attention_cosine).

Synthetic data of the given shapes stands in for the two models: the queries, keys
and values that a model would compute for each new token are random draws.

    python examples/decode_mapped_cache.py [--cache model --layers-src 8 --layers-tgt 12 --prefix 4096 --tokens 64]
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import cross_model_kv_gb300 as kvb  # noqa: E402
import synth  # noqa: E402


THETA = 1e6


def rotated(x, pos):
    """x [..., T, d] with RoPE of the positions, rotate-half, in fp32."""
    d = x.shape[-1]
    angle = pos.double()[:, None] * THETA ** (-torch.arange(0, d, 2, device=x.device).double() / d)
    c, s = angle.cos().float(), angle.sin().float()
    lo, hi = x.float().split(d // 2, dim=-1)
    return torch.cat([lo * c - hi * s, hi * c + lo * s], dim=-1).to(x.dtype)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layers-src", type=int, default=8)
    ap.add_argument("--layers-tgt", type=int, default=12)
    ap.add_argument("--kv-heads", type=int, default=8)
    ap.add_argument("--q-heads", type=int, default=64)
    ap.add_argument("--prefix", type=int, default=4096)
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--page", type=int, default=64)
    ap.add_argument("--cache", choices=["8bit", "model"], default="8bit", help="what the paged cache holds")
    a = ap.parse_args(argv)
    L_s, L_t, H, Hq, d, k, T = a.layers_src, a.layers_tgt, a.kv_heads, a.q_heads, 128, 4, a.prefix
    dev, bf = "cuda", torch.bfloat16
    spec = lambda n: {"n_layers": n, "n_kv_heads": H, "head_dim": d, "rope_theta": THETA}
    total = T + a.tokens
    ctx = kvb.kvb_ctx_create(spec(L_s), spec(L_t), k, total)

    # the source's prefix, mapped to the target
    src_k, src_v = (synth.torch_content(s, L_s, H, T, d, 0.5, bf, dev) for s in (1, 2))
    sel = synth.hidden_selection(3, L_s, L_t, k)
    (W_k, b_k), (W_v, b_v) = (synth.torch_weights(s, L_t, k * H * d, H * d, bf, dev) for s in (4, 5))
    pos = torch.arange(T, dtype=torch.int32, device=dev)
    map_k, map_v = (torch.empty((L_t, H, T, d), dtype=bf, device=dev) for _ in range(2))
    kvb.kvb_map_apply(ctx, src_k, src_v, pos, sel, sel, W_k, W_v, b_k, b_v, map_k, map_v)

    # stored in pages: one sequence, its pages in any order
    eight = a.cache == "8bit"
    n_pages = -(-total // a.page)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    table = torch.randperm(n_pages, device=dev).to(torch.int32)[None]
    prefix = kvb.Seqs(table, i32([0, T]), i32([0]), max_tokens=T)
    if eight:
        cache = kvb.kvb_cache8_create(ctx, n_pages, a.page)
        kvb.kvb_cache8_write(ctx, cache, prefix, map_k, map_v)
        append, attend = kvb.kvb_cache8_append, kvb.kvb_cache8_attention
    else:
        cache = kvb.kvb_paged_create(ctx, n_pages, a.page, bf)
        kvb.kvb_paged_append(ctx, cache, prefix, map_k, map_v, rotate=False)
        append, attend = kvb.kvb_paged_append, kvb.kvb_paged_attention

    # decoding: the call's tensors stay in place, only the position moves on
    heads = synth.torch_content(6, L_t, Hq + 2 * H, a.tokens, d, 0.5, bf, dev)  # no RoPE
    at = i32([T])
    seqs = kvb.Seqs(table, i32([0, 1]), at, max_tokens=1, max_kv=total)
    row = torch.empty((1, Hq + 2 * H, 1, d), dtype=bf, device=dev)  # a token's projection
    tok_q, tok_k, tok_v = row.split([Hq, H, H], dim=1)
    rot_q, o = (torch.empty((1, Hq, 1, d), dtype=bf, device=dev) for _ in range(2))
    out, all_q = (torch.empty((L_t, Hq, a.tokens, d), dtype=bf, device=dev) for _ in range(2))

    def token(i):
        for l in range(L_t):
            row.copy_(heads[l:l + 1, :, i:i + 1])
            append(ctx, cache, seqs, tok_k, tok_v, q=tok_q, q_out=rot_q, l_begin=l)
            attend(ctx, cache, seqs, rot_q, o, l_begin=l)
            out[l, :, i].copy_(o[0, :, 0])
            all_q[l, :, i].copy_(rot_q[0, :, 0])
        at.add_(1)

    t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    t0.record()
    for i in range(a.tokens):
        token(i)
    t1.record()
    torch.cuda.synchronize()
    kvb.kvb_ctx_check(ctx)

    # the cache against a plain one, every decoded token a query
    where = torch.arange(total, dtype=torch.int32, device=dev)
    back_k, back_v = (torch.empty((L_t, H, total, d), dtype=bf, device=dev) for _ in range(2))
    if eight:
        kvb.kvb_cache8_read(ctx, cache, kvb.Seqs(table, i32([0, total]), i32([0]), max_tokens=total), back_k, back_v)
    else:
        for x, back in ((cache.k, back_k), (cache.v, back_v)):
            back.copy_(x[:, table[0].long()].transpose(1, 2).flatten(2, 3)[:, :, :total])
    new_k, new_v = heads[:, Hq:Hq + H], heads[:, Hq + H:]
    full_k, full_v = torch.cat([map_k, rotated(new_k, where[T:])], dim=2), torch.cat([map_v, new_v], dim=2)
    cos = torch.empty((L_t, Hq, a.tokens), device=dev)
    kvb.kvb_attention_cosine(ctx, all_q, where[T:].contiguous(), back_k, back_v, full_k, full_v, where, cos)
    torch.cuda.synchronize()
    kvb.kvb_ctx_check(ctx)
    mib = (cache.k.numel() + cache.v.numel()) * cache.k.element_size() / 2 ** 20
    print(f"{T} mapped + {a.tokens} decoded tokens, {L_t} layers: cache {mib:.1f} MiB ({'8 bits' if eight else 'bf16'})")
    print(f"{t0.elapsed_time(t1) / a.tokens:.3f} ms a token (append + attention, {L_t} layers)")
    print(f"attention-output cosine against a plain bf16 cache: mean {cos.mean():.5f}, min {cos.min():.5f}")
    return {"cos_mean": float(cos.mean()), "cos_min": float(cos.min()), "out": out}


if __name__ == "__main__":
    main()
