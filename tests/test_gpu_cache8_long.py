"""8-bit cache attention where a CTA has much to do: many tiles, many sequences, more
pages than one list holds; and what only one of the two kernels was tested with before.

Sequences share the pages of a small pool (any number may read a page), so that long ones cost
little.  Tolerances are those of test_gpu_cache8.py unless a test derives its own.
"""
import numpy as np
import pytest

from cases import to_host64
from test_gpu_cache8 import BF, F32, Pool, attend, check_attention, i32, kvb, offsets  # noqa: F401  (kvb: the fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

INF = float("inf")


def shared_pool(kvb, H, d, page, pages, n_seq, cols, seed):  # noqa: F811
    """A pool of `pages` written pages, and n_seq sequences of cols pages drawn from it."""
    P = Pool(kvb, 1, H, d, page, 1, pages * page, seed=seed, spare=0)
    P.fill([pages * page])
    P.table = P.table[0][P.rng.integers(0, pages, (n_seq, cols))]
    P.dtab = i32(P.table)
    P.lens = np.asarray([cols * page])
    return P


def queries(P, g, T, dtype, sigma=1.5):
    return torch.from_numpy(sigma * P.rng.standard_normal((1, P.H * g, T, P.d))).to(dtype).cuda()


def compare(P, q, n, lens, **kw):
    pos = np.asarray(lens) - n
    out, lse = attend(P, q, offsets(n), pos, **kw)
    P.kvb.kvb_ctx_check(P.ctx)
    check_attention(P, q, offsets(n), pos, out, lse)
    o2, z2 = attend(P, q, offsets(n), pos, **kw)
    assert torch.equal(out, o2) and torch.equal(lse, z2)


# ------------------------------------------------------------------ the prompt kernel

@pytest.mark.parametrize("d,page", [(64, 64), (64, 16), (128, 32), (128, 128)])
def test_prompts_with_many_tiles_for_each_cta(kvb, d, page):  # noqa: F811
    # 48 sequences x 2 heads of up to 9000 keys: above 20 tiles of 128 keys for each of 152 CTAs, in
    # segments of up to that many (rings of 8 and stages of 2 go round several times), and more
    # sequences than one warp searches
    P = shared_pool(kvb, 2, d, page, 160 * 16 // page, 48, -(-9000 // page), seed=d + page)
    lens = P.rng.integers(6000, 9001, 48)
    lens[[3, 17, 40]] = [1, 129, 9000]
    n = np.minimum(P.rng.integers(5, 10, 48), lens)
    n[20] = 0
    assert 2 * (lens // 128).sum() > 20 * 152
    compare(P, queries(P, 8, n.sum(), BF), n, lens)


@pytest.mark.parametrize("d", [64, 128])
def test_prompts_of_many_sequences(kvb, d):  # noqa: F811
    # more sequences than the CTA has threads (640): the search for a CTA's first goes round twice
    P = shared_pool(kvb, 1, d, 16, 60, 1500, 19, seed=d)
    lens = P.rng.integers(1, 301, 1500)
    n = np.minimum(P.rng.integers(0, 14, 1500), lens)
    n[700], lens[700] = 13, 300
    compare(P, queries(P, 4, n.sum(), BF), n, lens, max_tokens=13)


@pytest.mark.parametrize("d", [64, 128])
def test_a_prompt_among_single_tokens(kvb, d):  # noqa: F811
    # row blocks follow the longest sequence: most of the others' are empty
    P = shared_pool(kvb, 2, d, 32, 80, 40, -(-2500 // 32), seed=d + 1)
    n = np.ones(40, dtype=int)
    n[[0, 13, 39]] = [0, 300, 65]
    lens = np.maximum(n, P.rng.integers(1, 2501, 40))
    lens[13] = 2500
    compare(P, queries(P, 8, n.sum(), BF), n, lens)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), INF, -INF])
def test_a_prompt_s_query_that_is_not_finite_stays_in_its_row(kvb, d, bad):  # noqa: F811
    P = Pool(kvb, 1, 1, d, 64, 1, 700)
    P.fill([700])
    q = queries(P, 2, 160, BF)
    clean, zc = attend(P, q, [0, 160], [540])
    q2 = q.clone()
    rows = [(0, 0, 7), (1, 77, 0), (0, 159, d - 1)]
    for h, i, e in rows:
        q2[0, h, i, e] = bad
    out, z = attend(P, q2, [0, 160], [540])
    P.kvb.kvb_ctx_check(P.ctx)
    for h, i, _ in rows:
        assert torch.isnan(out[0, h, i]).all() and torch.isnan(z[0, h, i])
        out[0, h, i], z[0, h, i] = clean[0, h, i], zc[0, h, i]
    assert torch.equal(out, clean) and torch.equal(z, zc)


def test_prompts_captured_on_a_side_stream_while_the_cache_grows(kvb):  # noqa: F811
    P = Pool(kvb, 1, 2, 128, 64, 2, 900)
    P.fill([600, 300])
    side = torch.cuda.Stream()
    n = 30
    off, pos = i32([0, n, 2 * n]), i32([600, 300])
    k, v = (torch.randn(1, 2, 2 * n, 128, device="cuda").to(BF) for _ in range(2))
    q = torch.randn(1, 16, 2 * n, 128, device="cuda").to(BF)
    out, lse = torch.empty_like(q), torch.empty(1, 16, 2 * n, device="cuda")
    seqs = kvb.Seqs(P.dtab, off, pos, max_tokens=n, max_kv=900)
    kvb.kvb_cache8_attention(P.ctx, P.cache, seqs, q, out, lse)  # sizes the workspace
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        kvb.kvb_cache8_write(P.ctx, P.cache, seqs, k, v)
        kvb.kvb_cache8_attention(P.ctx, P.cache, seqs, q, out, lse)
    for i in range(4):
        at = [600 + i * n, 300 + i * n]
        with torch.cuda.stream(side):
            for t in (k, v, q):
                t.normal_()
            pos.copy_(i32(at))
            graph.replay()
        side.synchronize()
        for kv, x in enumerate((k, v)):
            P.ref.write(kv, to_host64(x), P.table, [0, n, 2 * n], at)
        P.lens = np.asarray(at) + n
        check_attention(P, q, [0, n, 2 * n], np.asarray(at), out, lse)
    kvb.kvb_ctx_check(P.ctx)


# ------------------------------------------------------------------ the kernel of few rows

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,g", [(16, 1), (32, 3), (64, 2), (64, 12), (128, 8), (128, 16)])
def test_more_pages_than_one_list_holds(kvb, d, g, dtype):  # noqa: F811
    # pages of 16 keys, lists of 256 pages, four CTAs an SM at most: above 4 x 152 x 256 pages a CTA
    # takes two lists.  Every key counts as often as its page comes; a CTA adds 2 of 16 keys a
    # thread and step, kv / 32 / (2 x 152) steps at most (two CTAs an SM at least).
    page, cols = 16, 700 * 256 + 77
    kv = cols * page
    P = shared_pool(kvb, 1, d, page, 50, 1, cols, seed=d + g)
    q = queries(P, g, 1, dtype, 4.0)
    out, lse = attend(P, q, [0, 1], [kv - 1])
    kvb.kvb_ctx_check(P.ctx)
    ids, times = np.unique(P.table[0], return_counts=True)
    k, v = (P.ref.sequence(x, ids, len(ids) * page, 0, 0) for x in (0, 1))
    s = to_host64(q)[0, :, 0] @ k.T / np.sqrt(d)
    w = np.exp(s - s.max(axis=1, keepdims=True)) * np.repeat(times, page)
    z = s.max(axis=1) + np.log(w.sum(axis=1))
    w /= w.sum(axis=1, keepdims=True)
    reach = (np.abs(to_host64(q)[0, :, 0]) @ np.abs(k).T).max(axis=1) / np.sqrt(d)
    ds = (d / 16 + 4) * 2.0 ** -23 * reach[:, None] + kv / 32 / 304 * 2.0 ** -23
    bits = 2.0 ** -11 if dtype == BF else 2.0 ** -21
    tol = (w @ np.abs(v)) * (2 * (ds + 2.0 ** -21) + bits) + np.abs(w @ v) * (2.0 ** -8 if dtype == BF else 2.0 ** -23)
    tol += kv * 2.0 ** -31 * np.abs(v).max()
    assert (np.abs(to_host64(out)[0, :, 0] - w @ v) <= tol).all()
    assert (np.abs(to_host64(lse)[0, :, 0] - z) <= ds[:, 0] + 2.0 ** -21 + 2.0 ** -22 * np.abs(z)).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,g", [(32, 1), (64, 4), (128, 8)])
def test_single_tokens_of_many_sequences(kvb, d, g, dtype):  # noqa: F811
    # more sequences than the CTA has threads, eight rows over few and over many keys
    for n_seq, longest in ((300, 40), (900, 700)):
        P = shared_pool(kvb, 1, d, 16, 60, n_seq, -(-longest // 16), seed=d + n_seq)
        lens = P.rng.integers(1, longest + 1, n_seq)
        n = np.ones(n_seq, dtype=int)
        n[[5, n_seq - 1]] = 0
        compare(P, queries(P, g, n.sum(), dtype), n, lens, max_kv=longest)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("bad", [INF, -INF])
def test_an_infinite_query_stays_in_its_row(kvb, dtype, bad):  # noqa: F811
    P = Pool(kvb, 1, 1, 128, 64, 1, 300)
    P.fill([300])
    q = queries(P, 8, 2, dtype)
    clean, zc = attend(P, q, [0, 2], [298])
    q2 = q.clone()
    q2[0, 3, 1, 7] = bad
    out, z = attend(P, q2, [0, 2], [298])
    P.kvb.kvb_ctx_check(P.ctx)
    assert torch.isnan(out[0, 3, 1]).all() and torch.isnan(z[0, 3, 1])
    out[0, 3, 1], z[0, 3, 1] = clean[0, 3, 1], zc[0, 3, 1]
    assert torch.equal(out, clean) and torch.equal(z, zc)


# ------------------------------------------------------------------ two parts of a cache

@pytest.mark.parametrize("dtype,g,n", [(BF, 3, 1), (F32, 3, 1), (F32, 2, 9), (BF, 2, 40)])
def test_parts_join_by_their_sums(kvb, dtype, g, n):  # noqa: F811
    # attention over [0, 48) and over [48, 136), the second as a sequence of its own whose pages and
    # positions start there; joined by lse they are attention over all of it.  Each part's output
    # is rounded once (2^-8 or 2^-23) and its weights are fp16 (2^-11) or pairs (2^-21); all sums 40 2^-23.
    d, page, cut, kv = 128, 16, 48, 136
    P = Pool(kvb, 1, 2, d, page, 1, kv)
    P.fill([kv])
    q = queries(P, g, n, dtype)
    pos = [kv - n]
    whole, z = attend(P, q, [0, n], pos)
    a, za = attend(P, q, [0, n], pos, kv_len=i32([cut]))
    check_attention(P, q, [0, n], pos, whole, z)
    check_attention(P, q, [0, n], pos, a, za, kv_len=[cut])
    tail = i32(P.table[:, cut // page:].copy())
    b, zb = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    kvb.kvb_cache8_attention(P.ctx, P.cache, kvb.Seqs(tail, i32([0, n]), i32([pos[0] - cut]), max_tokens=n), q, b, zb)
    kvb.kvb_ctx_check(P.ctx)
    a, b, whole, za, zb, z = (to_host64(t) for t in (a, b, whole, za, zb, z))
    joined = np.logaddexp(za, zb)
    fa, fb = np.exp(za - joined)[..., None], np.exp(zb - joined)[..., None]
    o, zo, A, B = P.ref.attention(to_host64(q), P.table, [0, n], pos)
    ds = (d / 16 + 4) * 2.0 ** -23 * B
    bits, last = (2.0 ** -11, 2.0 ** -8) if dtype == BF else (2.0 ** -21, 2.0 ** -23)
    tol = A * (2 * (ds[..., None] + 2.0 ** -21) + 40 * 2.0 ** -23 + bits) + kv * 2.0 ** -31 * np.abs(P.ref.sequence(1, P.table[0], kv, 0, 0)).max()
    rounded = last * (np.abs(fa * a) + np.abs(fb * b) + np.abs(whole))
    assert (np.abs(fa * a + fb * b - whole) <= 2 * tol + rounded).all()
    assert (np.abs(fa * a + fb * b - o) <= tol + rounded).all()
    slack = ds + 2.0 ** -20 + 40 * 2.0 ** -23 + 2.0 ** -22 * np.abs(zo)
    assert (np.abs(joined - z) <= 2 * slack).all() and (np.abs(joined - zo) <= slack).all()
