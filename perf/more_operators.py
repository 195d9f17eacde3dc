"""Cases and plain forms of a decoding step over a paged cache that keeps the
model's own type: appending a call's keys and values (and its queries) with the
position rotation applied on the way, the same append into the 8-bit cache, and
attention of new tokens over the pages.

  rotate   a row x at position p, pairs (i, i + d/2), w_i = theta^(-2i/d):
           x'_i       = x_i cos(p w_i) - x_{i+d/2} sin(p w_i)
           x'_{i+d/2} = x_{i+d/2} cos(p w_i) + x_i sin(p w_i)
           with cos and sin as 32-bit numbers (of 64-bit angles); every product
           and the sum are rounded to 32 bits, the result once to its type
  append   rotated k and plain v of every token into its slot of the pages,
           rotated q into an output of its own
  append8  the same into e4m3 codes with a power-of-two scale 2^e for each block
           (layer, page, head); slots [0, s0) of the block written earlier:
           e_new = the smallest e in [-117, 119] with max|x'| <= 448 * 2^e
           e     = max(e_old, e_new) if s0 > 0, else e_new
           c_j   = e4m3(x'_j * 2^-e), to nearest, ties to even, saturating at 448
           and, where e > e_old, c_i = e4m3(c_i * 2^(e_old - e)) before s0
  attend   s_ij = q_i . k_j / sqrt(d) for every key j up to the position of query i,
           o_i = sum_j softmax_j(s_ij) v_j, lse_i = log sum_j exp(s_ij); query
           head hq reads KV head hq // g

Rows are [layer][head][token][dim] with strides of their own.  "token" layout is
that of a fused projection, [layer][token][q heads, k heads, v heads][dim]; "head"
layout is a plain cache.  Pages are [layer][page][head][slot][dim].  Sequence s owns
tokens off[s] .. off[s+1]-1 of the call, the first at position pos[s] of the sequence;
page_table[s][p] is the page of its positions p*page .. p*page+page-1.
"""
from __future__ import annotations

import math
import random

import torch

own = False

BF16, F32 = "bf16", "f32"
DT = {BF16: torch.bfloat16, F32: torch.float32}
THETA = 1e6
E_MIN, E_MAX, CODE_MAX = -117, 119, 448.0


# --------------------------------------------------------------------- the cases

def _case(name, op, dtype, L, H, g, d, page, n_seq, kv, new, ragged, layout, rotate, with_q, mix):
    c = {"op": op, "dtype": dtype, "L": L, "H": H, "g": g, "d": d, "page": page, "n_seq": n_seq, "kv": kv, "new": new,
         "ragged": ragged, "layout": layout, "rotate": rotate, "with_q": with_q, "mix": mix}
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one layer's new token of one sequence being decoded, straight from the fused projection: the smallest
        # append, once per layer and token, where latency counts
        _case("append_one_token", "append", BF16, 1, 8, 8, 128, 64, 1, 4096, 1, False, "token", True, True, 1),
        # the same for a serving batch: 64 sequences at unequal positions
        _case("append_batch_token", "append", BF16, 1, 8, 8, 128, 64, 64, 8192, 1, True, "token", True, True, 2),
        # one layer's 8192-token prompt: 64 query and 8 KV heads
        _case("append_prompt_layer", "append", BF16, 1, 8, 8, 128, 64, 1, 8192, 8192, False, "token", True, True, 3),
        # a mapped cache (its keys rotated already): all 64 target layers of an 8192-token prefix into pages; the largest
        _case("append_mapped_cache", "append", BF16, 64, 8, 8, 128, 64, 1, 8192, 8192, False, "head", False, False, 4),
        # fp32 caches of a 28-layer target without rotation applied yet, ragged packed sequences that continue inside a page
        _case("append_ragged_f32", "append", F32, 28, 8, 2, 128, 32, 5, 2500, 1111, True, "head", True, False, 5),
        # a serving batch's new tokens into the 8-bit cache, most of them inside a page
        _case("append8_batch_token", "append8", BF16, 1, 8, 8, 128, 64, 64, 8192, 1, True, "token", True, True, 6),
        # one layer's 8192-token prompt into the 8-bit cache
        _case("append8_prompt_layer", "append8", BF16, 1, 8, 8, 128, 64, 1, 8192, 8192, False, "token", True, True, 7),
        # decoding one sequence: one layer, one token over 4096 keys; latency counts
        _case("decode_one_4k", "attend", BF16, 1, 8, 8, 128, 64, 1, 4096, 1, False, "token", False, True, 8),
        # decoding a serving batch: 64 sequences of 1K to 8K tokens
        _case("decode_batch_ragged", "attend", BF16, 1, 8, 8, 128, 64, 64, 8192, 1, True, "token", False, True, 9),
        # decoding 16 sequences of 32768 tokens, the length of the map benchmark: the largest read
        _case("decode_batch_32k", "attend", BF16, 1, 8, 8, 128, 64, 16, 32768, 1, False, "token", False, True, 10),
        # fp32 decoding of a small-head model, pages of 16, odd lengths
        _case("decode_f32_d64", "attend", F32, 2, 8, 4, 64, 16, 16, 3001, 1, True, "head", False, True, 11),
        # several tokens a sequence at once (drafted tokens being checked): 16 sequences x up to 5 tokens
        _case("verify_5_tokens", "attend", BF16, 1, 8, 8, 128, 64, 16, 8192, 5, True, "token", False, True, 12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["append", "append", "append8", "attend", "attend"])
    dtype = rng.choice([BF16, BF16, F32])
    H = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 3, 4, 5, 7, 8])
    d = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    layout = rng.choice(["token", "token", "head"])
    mix = rng.randrange(1 << 30)
    ragged = rng.random() < 0.7
    half = 1 if dtype == BF16 else 2
    if op == "attend":
        L = rng.choice([1, 1, 1, 2, 3])
        n_seq = _log_int(rng, 1, 64)
        kv = _log_int(rng, 17, 32768)
        new = 1 if rng.random() < 0.7 else min(kv, _log_int(rng, 2, 8))
        # no more keys than the largest listed case
        while L * H * n_seq * kv > 8 * 16 * 32768 // half:
            n_seq = max(1, n_seq // 2)
            kv = kv if n_seq > 1 else kv // 2
        return _case(None, op, dtype, L, H, g, d, page, n_seq, kv, min(new, kv), ragged, layout, False, True, mix)
    L = rng.choice([1, 1, 2, 28, 64])
    n_seq = _log_int(rng, 1, 64)
    new = _log_int(rng, 1, 8192)
    rotate = op == "append8" or rng.random() < 0.8
    with_q = rotate and rng.random() < 0.6
    # no more elements than the largest listed case
    while L * H * (2 + (g if with_q else 0)) * n_seq * new > 2 * 64 * 8 * 8192 // half:
        n_seq = max(1, n_seq // 2)
        new = new if n_seq > 1 else max(1, new // 2)
    kv = new + _log_int(rng, 1, 4000) - 1
    return _case(None, op, dtype, L, H, g, d, page, n_seq, kv, new, ragged, layout, rotate, with_q, mix)


def _lengths(c):
    """(tokens of the call, position of the first) of each sequence; the case alone decides."""
    rng = random.Random(c["mix"])
    out = []
    for _ in range(c["n_seq"]):
        n = rng.randint((c["new"] + 3) // 4, c["new"]) if c["ragged"] else c["new"]
        kv = rng.randint(max(n, c["kv"] // 8), max(n, c["kv"])) if c["ragged"] else c["kv"]
        out.append((n, kv - n))
    return out


def work(case):
    c, ln = case, _lengths(case)
    el = 2 if c["dtype"] == BF16 else 4
    tok = sum(n for n, _ in ln)
    row = c["L"] * c["H"] * c["d"]
    if c["op"] == "attend":
        keys = sum(p + n for n, p in ln)
        seen = sum(n * p + n * (n + 1) // 2 for n, p in ln)
        rows = c["L"] * c["H"] * c["g"]
        return {"bytes": 2 * keys * row * el + 2 * tok * rows * c["d"] * el + 4 * tok * rows,
                "flops": 4 * c["d"] * rows * seen}
    q = c["g"] if c["with_q"] else 0
    rotated = tok * row * ((1 if c["rotate"] else 0) + q)
    moved = 2 * tok * row * (el + (1 if c["op"] == "append8" else el)) + 2 * tok * row * q * el
    if c["op"] == "append8":
        blocks = sum((p + n - 1) // c["page"] - p // c["page"] + 1 for n, p in ln)
        moved += 2 * 4 * blocks * c["L"] * c["H"]
    return {"bytes": moved, "flops": 3 * rotated + (2 * tok * row if c["op"] == "append8" else 0)}


# --------------------------------------------------------------------- inputs

class State:
    pass


def _rows(gen, L, T, heads, d, dt, dev, layout):
    """Rows [L][heads][T][d] in the layout asked for: normal draws with a log-normal scale for each head and channel."""
    base = torch.empty((L, T, heads, d) if layout == "token" else (L, heads, T, d), dtype=dt, device=dev)
    view = base.transpose(1, 2) if layout == "token" else base
    for l in range(L):  # a layer at a time bounds the fp32 temporaries
        s = torch.exp(0.5 * torch.randn((heads, 1, d), generator=gen, device=dev))
        view[l] = (torch.randn((heads, T, d), generator=gen, device=dev) * s).to(dt)
    return view


def prepare(case, seed):
    c = case
    dev = torch.device("cuda" if torch.cuda.is_available() else "cpu")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    ln = _lengths(c)
    L, H, g, d, page, B = c["L"], c["H"], c["g"], c["d"], c["page"], c["n_seq"]
    dt = DT[c["dtype"]]
    st = State()
    st.case = c
    st.max_new = max(n for n, _ in ln)
    st.max_kv = max(n + p for n, p in ln)
    st.T = sum(n for n, _ in ln)
    off = [0]
    for n, _ in ln:
        off.append(off[-1] + n)
    per = [-(-(n + p) // page) for n, p in ln]
    n_pages = sum(per) + 3  # a pool with some pages to spare, handed out in no order
    ids = torch.randperm(n_pages, generator=gen, device=dev)[: sum(per)].to(torch.int32)
    owner = torch.repeat_interleave(torch.arange(B), torch.tensor(per))
    column = torch.cat([torch.arange(n) for n in per])
    st.page_table = torch.zeros((B, max(per)), dtype=torch.int32, device=dev)
    st.page_table[owner.to(dev), column.to(dev)] = ids
    st.off = torch.tensor(off, dtype=torch.int32, device=dev)
    st.pos = torch.tensor([p for _, p in ln], dtype=torch.int32, device=dev)
    # the pages, filled with what earlier calls left there
    st.pages, st.scales = [], []
    filled = c["op"] == "attend" or any(p for _, p in ln)
    for _ in ("k", "v"):
        x = torch.zeros((L, n_pages, H, page, d), dtype=torch.float8_e4m3fn if c["op"] == "append8" else dt, device=dev)
        scale = torch.ones((L, n_pages, H), device=dev) if c["op"] == "append8" else None
        if filled:
            for l in range(L):
                s = torch.exp(0.5 * torch.randn((1, H, 1, d), generator=gen, device=dev))
                y = torch.randn((n_pages, H, page, d), generator=gen, device=dev) * s
                if scale is not None:
                    e = _exponent(y.abs().amax(dim=(2, 3)))
                    scale[l] = _pow2(e)
                    y = y * _pow2(-e)[:, :, None, None]
                x[l] = y.to(x.dtype)
        st.pages.append(x)
        st.scales.append(scale)
    if c["op"] == "attend":
        st.q = _rows(gen, L, st.T, H * g, d, dt, dev, c["layout"])
    elif c["layout"] == "token":
        x = _rows(gen, L, st.T, H * g + 2 * H, d, dt, dev, "token")  # what one projection gives
        st.q, st.k, st.v = x[:, : H * g], x[:, H * g: H * g + H], x[:, H * g + H:]
    else:
        st.k, st.v = (_rows(gen, L, st.T, H, d, dt, dev, "head") for _ in range(2))
        st.q = _rows(gen, L, st.T, H * g, d, dt, dev, "head") if c["with_q"] else None
    st.out = None
    if c["with_q"]:
        st.out = torch.empty((L, st.T, H * g, d) if c["layout"] == "token" else (L, H * g, st.T, d), dtype=dt, device=dev)
        st.out = st.out.transpose(1, 2) if c["layout"] == "token" else st.out
    st.lse = torch.empty((L, H * g, st.T), device=dev) if c["op"] == "attend" else None
    # cos and sin of every position, as a program that rotates keeps them
    w = THETA ** (-torch.arange(d // 2, dtype=torch.float64, device=dev) / (d // 2))
    angle = torch.arange(st.max_kv, dtype=torch.float64, device=dev)[:, None] * w[None]
    st.cos, st.sin = torch.cos(angle).float(), torch.sin(angle).float()
    if own:
        import cross_model_kv_gb300 as kvb

        spec = lambda n: {"n_layers": n, "n_kv_heads": H, "head_dim": d, "rope_theta": THETA}  # noqa: E731
        st.kvb = kvb
        st.ctx = kvb.kvb_ctx_create(spec(1), spec(L), 1, st.max_kv, 0)
        if c["op"] == "append8":
            st.cache = kvb.Cache8(st.ctx, st.pages[0], st.pages[1], st.scales[0], st.scales[1])
        else:
            st.cache = kvb.PagedCache(st.ctx, st.pages[0], st.pages[1])
        st.seqs = kvb.Seqs(st.page_table, st.off, st.pos, max_tokens=st.max_new, max_kv=st.max_kv)
    return st


# --------------------------------------------------------------------- one pass

def run(st):
    c = st.case
    if own:
        if c["op"] == "attend":
            st.kvb.kvb_paged_attention(st.ctx, st.cache, st.seqs, st.q, st.out, st.lse)
            return {"out": st.out, "lse": st.lse}
        append = st.kvb.kvb_cache8_append if c["op"] == "append8" else st.kvb.kvb_paged_append
        if c["with_q"]:
            append(st.ctx, st.cache, st.seqs, st.k, st.v, st.q, st.out, rotate=c["rotate"])
        else:
            append(st.ctx, st.cache, st.seqs, st.k, st.v, rotate=c["rotate"])
        return _appended(st)
    if c["op"] == "attend":
        return _plain_attend(st)
    s, at = _owner(st)
    if c["with_q"]:
        st.out.copy_(_rotate(st, st.q.float(), at))
    k = _rotate(st, st.k.float(), at) if c["rotate"] else st.k.float()
    if c["op"] == "append8":
        _plain_quantise(st, k, 0)
        _plain_quantise(st, st.v.float(), 1)
    else:
        ids, slot = st.page_table.long()[s, at // c["page"]], at % c["page"]
        st.pages[0][:, ids, :, slot] = k.permute(2, 0, 1, 3).to(DT[c["dtype"]])
        st.pages[1][:, ids, :, slot] = st.v.permute(2, 0, 1, 3)
    return _appended(st)


def _appended(st):
    res = {"k": st.pages[0], "v": st.pages[1]}
    if st.case["op"] == "append8":
        res |= {"k_scale": st.scales[0], "v_scale": st.scales[1]}
    if st.case["with_q"]:
        res["q"] = st.out
    return res


def _owner(st):
    """For each token of the call its sequence and its position there."""
    t = torch.arange(st.T, dtype=torch.int32, device=st.off.device)
    s = (t[:, None] >= st.off[None, 1:]).sum(dim=1)
    return s, (st.pos[s] + t - st.off[s]).long()


def _rotate(st, x, at):
    half = x.shape[-1] // 2
    cos, sin = st.cos[at], st.sin[at]  # [T][d/2]
    lo, hi = x[..., :half], x[..., half:]
    return torch.cat([lo * cos - hi * sin, hi * cos + lo * sin], dim=-1)


def _exponent(amax):
    """The smallest e in [-117, 119] with amax <= 448 * 2^e, as an int32 tensor."""
    m, x = torch.frexp(amax)  # amax = m 2^x, 1/2 <= m < 1; 448 = 0.875 * 2^9
    e = x - 9 + (m > 0.875).to(x.dtype)
    return torch.where(amax > 0, e, torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX)


def _pow2(e):
    """2^e in fp32 for integers e (0 below 2^-126), from its bits: exp2 need not be exact."""
    return torch.where(e < -126, torch.zeros_like(e), (e.clamp(min=-126) + 127) << 23).view(torch.float32)


def _round_e4m3(x):
    """x to the nearest e4m3 number (3 bits after the leading one, 2^-9 at the least), ties to even."""
    x = x.clamp(-CODE_MAX, CODE_MAX)
    _, ex = torch.frexp(x)
    step = _pow2((ex - 1).clamp(min=-6) - 3)
    return torch.round(x / step) * step


def _plain_quantise(st, x, kv):
    """x [L][H][T][d] in 32 bits into the codes and scales of the blocks that the call's tokens touch."""
    page = st.case["page"]
    dev = x.device
    n_items = (st.max_new + page - 2) // page + 1
    n = (st.off[1:] - st.off[:-1]).long()[:, None, None]
    first = st.pos.long()[:, None, None]
    logical = first // page + torch.arange(n_items, device=dev)[None, :, None]
    index = logical * page + torch.arange(page, device=dev)[None, None, :]  # [B][items][page]
    new = (index >= first) & (index < first + n)
    token = torch.where(new, st.off[:-1].long()[:, None, None] + index - first, torch.zeros_like(index))
    ids = torch.gather(st.page_table.long(), 1, logical[:, :, 0].clamp(max=st.page_table.shape[1] - 1))
    keep = new.any(dim=2).reshape(-1).nonzero()[:, 0]  # blocks that the call writes to
    ids, token, new, before = (t.reshape((-1,) + t.shape[2:])[keep] for t in (ids, token, new, index < first))
    m = new[None, None, :, :, None]
    xs = torch.where(m, x[:, :, token], torch.zeros((), device=dev))  # [L][H][blocks][page][d]
    e_new = _exponent(xs.abs().amax(dim=(3, 4)))
    old = st.pages[kv][:, ids].transpose(1, 2).float()
    e_old = torch.frexp(st.scales[kv][:, ids].transpose(1, 2))[1] - 1
    e = torch.where(before.any(dim=1), torch.maximum(e_old, e_new), e_new)
    lowered = _round_e4m3(old * _pow2((e_old - e).clamp(max=0))[..., None, None])
    codes = torch.where(m, _round_e4m3(xs * _pow2(-e)[..., None, None]), torch.where(before[:, :, None], lowered, old))
    st.pages[kv][:, ids] = codes.transpose(1, 2).to(torch.float8_e4m3fn)
    st.scales[kv][:, ids] = _pow2(e).transpose(1, 2)


def _plain_attend(st):
    c = st.case
    L, H, g, d, page, B = c["L"], c["H"], c["g"], c["d"], c["page"], c["n_seq"]
    n = st.max_new
    cols = -(-st.max_kv // page)
    ids = st.page_table[:, :cols].long()
    k, v = (x[:, ids].float().transpose(2, 3).reshape(L, B, H, cols * page, d) for x in st.pages)
    # queries padded to n a sequence: [L][B][H][g n][d]
    i = torch.arange(n, device=st.off.device)
    have = i[None] < (st.off[1:] - st.off[:-1])[:, None]
    token = torch.where(have, st.off[:-1].long()[:, None] + i[None], torch.zeros_like(i)[None])
    q = st.q[:, :, token].float().reshape(L, H, g, B, n, d).permute(0, 3, 1, 2, 4, 5).reshape(L, B, H, g * n, d)
    s = torch.matmul(q, k.transpose(-1, -2)) * (1.0 / math.sqrt(d))
    see = torch.arange(cols * page, device=st.off.device)[None, None] <= (st.pos[:, None] + i[None])[:, :, None]
    see = see[None, :, None, None]  # [1][B][1][1][n][keys]
    s = s.reshape(L, B, H, g, n, cols * page)
    s = torch.where(see, s, torch.full((), -math.inf, device=s.device))
    m = s.amax(dim=-1, keepdim=True)
    p = torch.exp(s - m)
    total = p.sum(dim=-1, keepdim=True)
    o = torch.matmul(p.reshape(L, B, H, g * n, -1), v).reshape(L, B, H, g, n, d) / total
    lse = (m + torch.log(total))[..., 0]
    where = have.reshape(-1).nonzero()[:, 0]
    o = o.permute(0, 2, 3, 1, 4, 5).reshape(L, H * g, B * n, d)[:, :, where]
    lse = lse.permute(0, 2, 3, 1, 4).reshape(L, H * g, B * n)[:, :, where]
    return {"out": o.to(DT[c["dtype"]]), "lse": lse}


# --------------------------------------------------------------------- 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "attend":
        return _exact_attend(st, case, _lengths(case))
    return _exact_append(st, case, _lengths(case))


def _turned(x, first, d):
    """Rows x [...][n][d] in 64 bits at positions first, first + 1, ...: each pair as a complex number times e^(i p w)."""
    n = x.shape[-2]
    p = torch.arange(first, first + n, dtype=torch.float64, device=x.device)
    i = torch.arange(0, d, 2, dtype=torch.float64, device=x.device)
    angle = p[:, None] * torch.exp(-math.log(THETA) * i / d)[None]
    z = torch.complex(x[..., : d // 2].contiguous(), x[..., d // 2:].contiguous()) * torch.polar(torch.ones_like(angle), angle)
    return torch.cat([z.real, z.imag], dim=-1)


def _grid(dev):
    """The non-negative e4m3 numbers in order (exponent field E, fraction F) and whether each one's F is even."""
    vals, even = [], []
    for E in range(16):
        for F in range(8):
            if (E, F) != (15, 7):
                vals.append(F * 2.0 ** -9 if E == 0 else (8 + F) * 2.0 ** (E - 10))
                even.append(F % 2 == 0)
    return torch.tensor(vals, dtype=torch.float64, device=dev), torch.tensor(even, device=dev)


def _nearest(x, grid, even):
    """The grid's number nearest to each |x| (the even one of two as near), with x's sign."""
    a = x.abs()
    hi = torch.searchsorted(grid, a.contiguous()).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - a, a - grid[lo]
    take = (up < down) | ((up == down) & even[hi])
    return torch.where(take, grid[hi], grid[lo]) * torch.sign(x)


def _pow2_64(e):
    return ((e + 1023) << 52).view(torch.float64)


def _exact_append(st, c, ln):
    page, off, d = c["page"], st.off.tolist(), c["d"]
    L, H, g = c["L"], c["H"], c["g"]
    eight = c["op"] == "append8"
    elements = st.T * L * H * d * (2 + (g if c["with_q"] else 0))
    pages = sum(x.numel() for x in st.pages)
    if elements > (4e8 if eight else 1.2e9) or pages > 1.3e9 or c["n_seq"] * L * (1 + st.max_new // page) > 20000:
        return None
    table = st.page_table.tolist()
    dev = st.off.device
    grid, even = _grid(dev)
    wide = torch.float32 if eight or L * H * d * st.T > 2e8 else torch.float64  # codes are exact in 32 bits; the rest to save room
    res = {name: x.to(wide) for name, x in zip("kv", st.pages)}
    if eight:
        res |= {"k_scale": st.scales[0].clone(), "v_scale": st.scales[1].clone()}
    if c["with_q"]:
        res["q"] = torch.empty(st.q.shape, dtype=torch.float64, device=dev)
    for s, (n, first) in enumerate(ln):
        for l in range(L):
            mine = slice(off[s], off[s] + n)
            if c["with_q"]:
                res["q"][l, :, mine] = _turned(st.q[l, :, mine].double(), first, d)
            for name, x in (("k", st.k[l, :, mine].double()), ("v", st.v[l, :, mine].double())):
                x = _turned(x, first, d) if name == "k" and c["rotate"] else x
                at = first
                while at < first + n:
                    pid, s0 = table[s][at // page], at % page
                    m = min(page - s0, first + n - at)
                    new = x[:, at - first: at - first + m]
                    if not eight:
                        res[name][l, pid, :, s0: s0 + m] = new.to(wide)
                    else:
                        top = new.abs().flatten(1).amax(dim=1)
                        e = torch.ceil(torch.log2(top / CODE_MAX)).clamp(E_MIN, E_MAX).long()
                        e = torch.where(top <= CODE_MAX * _pow2_64(e - 1), e - 1, torch.where(top > CODE_MAX * _pow2_64(e), e + 1, e))
                        e = e.clamp(E_MIN, E_MAX)
                        scale = res[name + "_scale"]
                        if s0:
                            was = (scale[l, pid].double().view(torch.int64) >> 52) - 1023
                            e = torch.maximum(e, was)
                            res[name][l, pid, :, :s0] = _nearest(res[name][l, pid, :, :s0].double() * _pow2_64(was - e)[:, None, None], grid, even).float()
                        res[name][l, pid, :, s0: s0 + m] = _nearest(new * _pow2_64(-e)[:, None, None], grid, even).float()
                        scale[l, pid] = _pow2_64(e).float()
                    at += m
    return res


def _exact_attend(st, c, ln):
    page, off, table, g = c["page"], st.off.tolist(), st.page_table.long(), c["g"]
    out = torch.zeros(st.q.shape, dtype=torch.float64, device=st.q.device)
    lse = torch.full(st.q.shape[:3], -math.inf, dtype=torch.float64, device=st.q.device)
    for s, (n, first) in enumerate(ln):
        kv = first + n
        ids = table[s, :-(-kv // page)]
        for l in range(c["L"]):
            for h in range(c["H"]):
                k, v = (x[l, :, h][ids].double().reshape(-1, c["d"])[:kv] for x in st.pages)
                q = st.q[l, h * g:(h + 1) * g, off[s]:off[s] + n].double()
                sc = (q @ k.T) / math.sqrt(c["d"])
                hide = torch.arange(kv, device=q.device)[None] > first + torch.arange(n, device=q.device)[:, None]
                sc = sc.masked_fill(hide[None], -math.inf)
                z = torch.logsumexp(sc, dim=-1)
                out[l, h * g:(h + 1) * g, off[s]:off[s] + n] = torch.exp(sc - z[..., None]) @ v
                lse[l, h * g:(h + 1) * g, off[s]:off[s] + n] = z
    return {"out": out, "lse": lse}
