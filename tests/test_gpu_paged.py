"""The paged cache of the model's own type: appends bit for bit, attention within bounds
derived from the formats; the append into the 8-bit cache bit for bit.

Append.  Every product and sum is rounded to fp32 by itself and the result once to its
type, which NumPy's float32 arithmetic repeats exactly (oracle.paged.rotate32).

Attention tolerance, per row, with spread A = sum p|v| and reach B = max_j scale *
sum_e |q_e k_je| (natural log units):
  * a score is d products summed in fp32, at most d/8 + 6 roundings of 2^-23 relative
    to B with the scaling and the difference from the reference: |ds| <= (d/8 + 6) 2^-23 B;
  * the exponential adds 2^-21 to a weight's relative error, and numerator and
    denominator both carry the weights' errors: 2 (|ds| + 2^-21) A;
  * sums over kv keys: a warp's steps are 64 keys apart and add the 16 keys of a step in
    at most 16 roundings, then 4 warps and the pieces are joined: (kv/4 + 64) 2^-24 A;
  * weights as bf16 pairs (bf16 calls): 2^-16 A;
  * the output's own rounding: 2^-8 |o| (bf16), 2^-24 |o| (fp32).
"""
import numpy as np
import pytest

from cases import spec, to_host64
from oracle import cache8 as C8
from oracle import paged as PG

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
INVALID_ARG, UNSUPPORTED, NUMERIC = 1, 3, 5
THETA = 1e6


@pytest.fixture(scope="module")
def kvb():
    from cross_model_kv_gb300 import build
    build.build()
    import cross_model_kv_gb300 as m
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return m


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def offsets(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(int)


def status_of(kvb, f):
    with pytest.raises(kvb.KvbError) as e:
        f()
    return e.value.status


def laid_out(x, layout, dtype):
    """x [L][heads][T][d] on the device as rows of a plain cache, of a projection's output, or with room between them."""
    t = torch.from_numpy(np.ascontiguousarray(x)).to(dtype).cuda()
    if layout == "head":
        return t
    if layout == "token":
        return t.transpose(1, 2).contiguous().transpose(1, 2)
    L, heads, T, d = t.shape
    room = torch.full((T + 1, L, heads + 2, 2 * d), float("nan"), dtype=dtype, device="cuda")  # tokens, then layers, then heads
    view = room[1:, :, 1:heads + 1, d // 2:d // 2 + d].permute(1, 2, 0, 3)
    view.copy_(t)
    return view


class Pool:
    """A paged cache on the device and the oracle's, with sequences whose pages come in no order; filled with NaN."""

    def __init__(self, kvb, L, H, d, page, n_seq, max_len, dtype, seed=0, spare=3, max_pos=None, eight=False):
        self.kvb, self.L, self.H, self.d, self.page, self.dtype = kvb, L, H, d, page, dtype
        self.max_pos = max_pos or max(max_len, 1)
        self.ctx = kvb.kvb_ctx_create(spec(1, H, d, 1e4), spec(L, H, d, THETA), 1, self.max_pos)
        cols = -(-max_len // page)
        self.rng = np.random.default_rng(seed)
        self.n_pages = n_seq * cols + spare
        self.table = self.rng.permutation(self.n_pages)[:n_seq * cols].reshape(n_seq, cols)
        if eight:
            self.cache = kvb.kvb_cache8_create(self.ctx, self.n_pages, page)
            self.ref = C8.Cache8(L, self.n_pages, H, page, d)
            for x in self.ref.scales:
                x.fill(2.0 ** -117)  # what a scale of 0 counts as
        else:
            self.cache = kvb.kvb_paged_create(self.ctx, self.n_pages, page, dtype)
            for t in (self.cache.k, self.cache.v):
                t.fill_(float("nan"))
            self.ref = PG.Paged(L, self.n_pages, H, page, d)
        self.dtab = i32(self.table)
        self.cos, self.sin = PG.table(THETA, d, self.max_pos)

    def seqs(self, off, pos, **kw):
        off, pos = np.asarray(off), np.asarray(pos)
        kw.setdefault("max_tokens", int(np.diff(off).max()) if len(off) > 1 else 0)
        return self.kvb.Seqs(self.dtab, i32(off), i32(pos), **kw)

    def rows(self, n_layers, heads, T, layout="head", sigma=1.0):
        return laid_out(sigma * self.rng.standard_normal((n_layers, heads, T, self.d)), layout, self.dtype)

    def positions(self, off, pos, T):
        at = np.full(T, -1)
        for s in range(len(pos)):
            at[off[s]:off[s + 1]] = pos[s] + np.arange(off[s + 1] - off[s])
        return at

    def turned(self, x, off, pos):
        """What rotating x gives, in float32."""
        return PG.rotate32(x.float().cpu().numpy(), self.positions(off, pos, x.shape[2]), self.cos, self.sin)

    def append(self, off, pos, layout="head", rotate=True, l_begin=0, n_layers=None, T=None, g=0, sigma=1.0):
        """Append random rows on both sides; returns (q, q_out)."""
        n_layers = self.L if n_layers is None else n_layers
        T = int(off[-1]) if T is None else T
        k, v = (self.rows(n_layers, self.H, T, layout, sigma) for _ in range(2))
        q = self.rows(n_layers, self.H * g, T, layout) if g else None
        q_out = laid_out(np.full(q.shape, 7.0), layout, self.dtype) if g else None
        call = self.kvb.kvb_paged_append if isinstance(self.ref, PG.Paged) else self.kvb.kvb_cache8_append
        call(self.ctx, self.cache, self.seqs(off, pos), k, v, q, q_out, l_begin=l_begin, rotate=rotate)
        rk = self.turned(k, off, pos) if rotate else k.float().cpu().numpy()
        if call is self.kvb.kvb_paged_append:
            rk = torch.from_numpy(np.ascontiguousarray(rk)).to(self.dtype).float().numpy()
        add = self.ref.write if call is self.kvb.kvb_cache8_append else self.ref.append
        for kv, x in enumerate((rk, v.float().cpu().numpy())):
            add(kv, x.astype(np.float64), self.table, off, pos, l_begin)
        return q, q_out

    def check_pages(self):
        """Every slot equals the oracle's, NaN where nothing was stored."""
        for kv, t in enumerate((self.cache.k, self.cache.v)):
            assert np.array_equal(to_host64(t), self.ref.codes[kv], equal_nan=True)

    def fill(self, lens):
        self.lens = np.asarray(lens)
        self.append(offsets(lens), np.zeros(len(lens), dtype=int), rotate=False)


# ------------------------------------------------------------------ append

GEOMETRY = [(16, 16, 1, 1), (32, 128, 3, 2), (64, 32, 2, 3), (128, 64, 2, 8), (128, 128, 1, 5), (128, 16, 5, 1)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layout", ["head", "token", "spaced"])
@pytest.mark.parametrize("d,page,H,g", GEOMETRY)
def test_append_bit_for_bit_growing_pages(kvb, d, page, H, g, layout, dtype):
    P = Pool(kvb, 2, H, d, page, 4, 5 * page + 40, dtype, seed=d + page)
    lens = np.zeros(4, dtype=int)
    for n in ([1, 0, page, 3 * page + 7], [5, page - 1, 1, 2 * page - 3], [1, 1, 1, 1], [17, 2, 30, 0], [0, page + 20, 0, 1]):
        off = offsets(n)
        q, q_out = P.append(off, lens, layout, g=g)
        want = torch.from_numpy(P.turned(q, off, lens)).to(dtype)
        assert torch.equal(q_out.cpu(), want)
        lens = lens + np.asarray(n)
    kvb.kvb_ctx_check(P.ctx)
    P.check_pages()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_append_without_rotation_and_of_some_layers(kvb, dtype):
    P = Pool(kvb, 5, 2, 64, 32, 2, 100, dtype)
    P.append([0, 40, 73], [0, 5], "token", rotate=False, l_begin=1, n_layers=3)
    P.append([0, 1, 2], [40, 38], "spaced", rotate=True, l_begin=4, n_layers=1)
    kvb.kvb_ctx_check(P.ctx)
    P.check_pages()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [16, 128])
def test_rotation_is_near_the_float64_one_at_far_positions(kvb, d, dtype):
    # against float64 angles: table, products and sum 3 half-steps of 2^-24 of the pair, then the type's
    from oracle import kvb_oracle as O
    at = [0, 1, 4095, 100000, 262143]
    P = Pool(kvb, 1, 1, d, 16, 1, 16, dtype, max_pos=262144)
    q = P.rows(1, 3, 5)
    out = torch.empty_like(q)
    k = P.rows(1, 1, 5)
    # five sequences of one token, each with a page that it repeats
    tab = i32(np.arange(5)[:, None].repeat(262144 // 16, 1))
    seqs = kvb.Seqs(tab, i32(np.arange(6)), i32(at), max_tokens=1)
    cache = kvb.kvb_paged_create(P.ctx, 5, 16, dtype)
    kvb.kvb_paged_append(P.ctx, cache, seqs, k, k.clone(), q, out)
    kvb.kvb_ctx_check(P.ctx)
    x = to_host64(q)
    want = O.rope(x, np.asarray(at), THETA)
    pair = np.abs(x) + np.abs(np.roll(x, d // 2, axis=-1))
    err = 3 * 2.0 ** -24 * pair
    assert (np.abs(to_host64(out) - want) <= err + (2.0 ** -8 if dtype == BF else 2.0 ** -24) * (np.abs(want) + err)).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [1, 77])
def test_queries_in_place_and_the_odd_head(kvb, n, dtype):
    P = Pool(kvb, 1, 3, 128, 64, 2, 200, dtype)
    off, pos = [0, n, 2 * n], [9, 0]
    q = P.rows(1, 9, 2 * n, "token")
    want = torch.from_numpy(P.turned(q, off, pos)).to(dtype)
    k, v = P.rows(1, 3, 2 * n), P.rows(1, 3, 2 * n)
    kvb.kvb_paged_append(P.ctx, P.cache, P.seqs(off, pos), k, v, q, q)
    assert torch.equal(q.cpu(), want)
    # one query head over one KV head: half of a job is empty
    P = Pool(kvb, 1, 1, 64, 64, 2, 200, dtype)
    q, out = P.append(off, pos, g=1)
    assert torch.equal(out.cpu(), torch.from_numpy(P.turned(q, off, pos)).to(dtype))
    P.check_pages()


def test_tokens_that_no_sequence_owns_are_left_alone(kvb):
    P = Pool(kvb, 1, 2, 64, 16, 3, 64, BF)
    off, pos = np.array([2, 5, 5, 9]), [3, 0, 10]
    q, out = P.append(off, pos, T=12, g=2)
    kvb.kvb_ctx_check(P.ctx)
    P.check_pages()
    want = torch.from_numpy(P.turned(q, off, pos)).to(BF)
    assert torch.equal(out[:, :, 2:9].cpu(), want[:, :, 2:9])
    assert torch.all(out[:, :, :2] == 7) and torch.all(out[:, :, 9:] == 7)


def test_infinities_and_nan_are_stored(kvb):
    P = Pool(kvb, 1, 1, 32, 16, 1, 16, F32)
    k, v = P.rows(1, 1, 4), P.rows(1, 1, 4)
    k[0, 0, 1, 3], k[0, 0, 2, 20], v[0, 0, 3, 5] = float("inf"), float("nan"), -float("inf")
    kvb.kvb_paged_append(P.ctx, P.cache, P.seqs([0, 4], [2]), k, v)
    kvb.kvb_ctx_check(P.ctx)
    got = P.cache.k[0, P.table[0, 0], 0, 2:6].cpu().numpy()
    assert np.array_equal(got, P.turned(k, [0, 4], [2])[0, 0], equal_nan=True)
    assert torch.equal(P.cache.v[0, P.table[0, 0], 0, 2:6], v[0, 0])


@pytest.mark.parametrize("eight", [False, True])
def test_append_reports_positions_and_pages_outside(kvb, eight):
    P = Pool(kvb, 1, 2, 64, 16, 2, 64, BF, max_pos=50, eight=eight)
    call = kvb.kvb_cache8_append if eight else kvb.kvb_paged_append
    if eight:
        for t in (P.cache.k, P.cache.v):
            t.view(torch.uint8).fill_(0x7f)
    bits = lambda: (P.cache.k.view(torch.uint8).clone(), P.cache.v.view(torch.uint8).clone())
    before = bits()
    k, v, q = P.rows(1, 2, 4), P.rows(1, 2, 4), P.rows(1, 4, 4)
    out = torch.full_like(q, 7.0)
    # positions 48 .. 51 of which the table holds two: the others' rows are 0, in the pages too
    call(P.ctx, P.cache, P.seqs([0, 0, 4], [0, 48]), k, v, q, out)
    assert status_of(kvb, lambda: kvb.kvb_ctx_check(P.ctx)) == INVALID_ARG
    assert torch.equal(out.cpu(), torch.from_numpy(P.turned(q, [0, 0, 4], [0, 48])).to(BF))
    assert torch.all(out[:, :, 2:] == 0) and torch.any(out[:, :, :2] != 0)
    for t in (P.cache.k, P.cache.v):
        page = t[0, P.table[1, 3]].float()
        assert torch.all(page[:, 2:4] == 0) and torch.any(page[:, :2] != 0)
    for t, b in zip((P.cache.k, P.cache.v), before):
        t.view(torch.uint8).copy_(b)
    # bad pages, sequences that do not fit: nothing is stored
    bad, neg = P.dtab.clone(), P.dtab.clone()
    bad[1], neg[1] = P.n_pages, -1
    cases = [kvb.Seqs(x, i32([0, 0, 4]), i32([0, 20]), max_tokens=4) for x in (bad, neg)]
    cases += [kvb.Seqs(P.dtab, i32(off), i32(pos), max_tokens=4) for off, pos in
              (([0, 5, 4], [0, 0]), ([0, 0, 9], [0, 0]), ([-1, 0, 0], [0, 0]), ([0, 0, 4], [0, -4]), ([0, 0, 4], [0, 2 ** 31 - 2]))]
    for s in cases:
        call(P.ctx, P.cache, s, k, v, q, out)
        assert status_of(kvb, lambda: kvb.kvb_ctx_check(P.ctx)) == INVALID_ARG
        kvb.kvb_ctx_check(P.ctx)
        assert all(torch.equal(a, b) for a, b in zip(bits(), before))
    # past the page table, without rotation
    call(P.ctx, P.cache, P.seqs([0, 0, 4], [0, 64]), k, v, rotate=False)
    assert status_of(kvb, lambda: kvb.kvb_ctx_check(P.ctx)) == INVALID_ARG
    assert all(torch.equal(a, b) for a, b in zip(bits(), before))


# ------------------------------------------------------------------ append into the 8-bit cache

def check_codes(P, lens):
    for kv, (c, s) in enumerate(((P.cache.k, P.cache.k_scale), (P.cache.v, P.cache.v_scale))):
        got, gs = c.view(torch.uint8).cpu().numpy(), s.cpu().numpy()
        for q, n in enumerate(lens):
            for p in range(-(-int(n) // P.page)):
                m, pid = min(P.page, int(n) - p * P.page), P.table[q, p]
                assert np.array_equal(gs[:, pid], P.ref.scales[kv][:, pid])
                assert np.array_equal(got[:, pid, :, :m], P.ref.codes[kv][:, pid, :, :m])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layout", ["head", "token", "spaced"])
@pytest.mark.parametrize("d,page,H,g", GEOMETRY)
def test_append8_bit_for_bit_growing_pages(kvb, d, page, H, g, layout, dtype):
    # tokens grow, so that scales rise and earlier codes are rounded again
    P = Pool(kvb, 2, H, d, page, 4, 5 * page + 40, dtype, seed=d + page, eight=True)
    lens = np.zeros(4, dtype=int)
    for step, n in enumerate(([1, 0, page, 3 * page + 7], [5, page - 1, 1, 2 * page - 3], [1, 1, 1, 1], [17, 2, 30, 0], [0, page + 20, 0, 1])):
        off = offsets(n)
        q, q_out = P.append(off, lens, layout, g=g if step % 2 else 0, sigma=1.7 ** step)
        if q is not None:
            assert torch.equal(q_out.cpu(), torch.from_numpy(P.turned(q, off, lens)).to(dtype))
        lens = lens + np.asarray(n)
    kvb.kvb_ctx_check(P.ctx)
    check_codes(P, lens)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_append8_without_rotation_is_the_write(kvb, dtype):
    P = Pool(kvb, 3, 2, 128, 64, 2, 200, dtype, eight=True)
    other = kvb.kvb_cache8_create(P.ctx, P.n_pages, 64)
    for t in (P.cache, other):
        t.k.view(torch.uint8).zero_(), t.v.view(torch.uint8).zero_()
    for off, pos in (([0, 100, 133], [0, 0]), ([0, 7, 8], [100, 33])):
        k, v = P.rows(2, 2, off[-1], "token", 3.0), P.rows(2, 2, off[-1], "token")
        kvb.kvb_cache8_append(P.ctx, P.cache, P.seqs(off, pos), k, v, l_begin=1, rotate=False)
        kvb.kvb_cache8_write(P.ctx, other, P.seqs(off, pos), k.contiguous(), v.contiguous(), l_begin=1)
    kvb.kvb_ctx_check(P.ctx)
    for a, b in ((P.cache.k, other.k), (P.cache.v, other.v), (P.cache.k_scale, other.k_scale), (P.cache.v_scale, other.v_scale)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_append8_of_values_that_are_not_finite(kvb):
    P = Pool(kvb, 1, 1, 32, 16, 1, 16, F32, eight=True)
    k, v = P.rows(1, 1, 4), P.rows(1, 1, 4)
    k[0, 0, 1, 3], v[0, 0, 3, 5] = float("inf"), float("nan")
    k[0, 0, 2, 1] = k[0, 0, 2, 17] = 3e38  # finite, but the rotated pair may not be
    kvb.kvb_cache8_append(P.ctx, P.cache, P.seqs([0, 4], [2]), k, v)
    assert status_of(kvb, lambda: kvb.kvb_ctx_check(P.ctx)) == NUMERIC
    P.ref.write(0, P.turned(k, [0, 4], [2]).astype(np.float64), P.table, [0, 4], [2])
    P.ref.write(1, to_host64(v), P.table, [0, 4], [2])
    for kv, (c, s) in enumerate(((P.cache.k, P.cache.k_scale), (P.cache.v, P.cache.v_scale))):
        pid = P.table[0, 0]
        assert np.array_equal(s[0, pid].cpu().numpy(), P.ref.scales[kv][0, pid])
        got = c.view(torch.uint8)[0, pid, 0, 2:6].cpu().numpy()
        want = P.ref.codes[kv][0, pid, 0, 2:6]
        assert np.array_equal(np.where(got == 0x80, 0, got), np.where(want == 0x80, 0, want))


# ------------------------------------------------------------------ attention

def attend(P, q, off, pos, lse=True, l_begin=0, scale=0.0, layout="head", **kw):
    out = laid_out(np.full(q.shape, np.nan), layout, q.dtype)
    z = torch.full(q.shape[:3], float("nan"), device="cuda") if lse else None
    P.kvb.kvb_paged_attention(P.ctx, P.cache, P.seqs(off, pos, **kw), q, out, z, l_begin=l_begin, scale=scale)
    return out, z


def check_attention(P, q, off, pos, out, lse, kv_len=None, l_begin=0, scale=None):
    d, dtype = q.shape[3], q.dtype
    o, z, A, B = P.ref.attention(to_host64(q), P.table, off, pos, kv_len, l_begin, scale)
    kv = int(max(np.asarray(pos) + np.diff(off)) if kv_len is None else max(kv_len))
    ds = (d / 8 + 6) * 2.0 ** -23 * B
    sums = (max(kv, 0) / 4 + 64) * 2.0 ** -24
    tol = A * (2 * (ds[..., None] + 2.0 ** -21) + sums + (2.0 ** -16 if dtype == BF else 0.0))
    tol = tol + (np.abs(o) + tol) * (2.0 ** -8 if dtype == BF else 2.0 ** -24)
    got = to_host64(out)
    assert np.isfinite(got).all()
    assert (np.abs(got - o) <= tol).all(), float((np.abs(got - o) / np.maximum(tol, 1e-300)).max())
    empty = np.isneginf(z)
    if lse is not None:
        gz = to_host64(lse)
        assert np.array_equal(np.isneginf(gz), empty)
        err = np.abs(np.where(empty, 0, gz) - np.where(empty, 0, z))
        assert (err <= ds + 2.0 ** -21 + sums + 2.0 ** -22 * np.abs(np.where(empty, 0, z))).all()
    assert np.all(got[empty] == 0)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layout", ["head", "token", "spaced"])
@pytest.mark.parametrize("d,page,H,g", [(16, 16, 2, 1), (32, 32, 1, 3), (64, 128, 2, 4), (128, 64, 2, 8), (128, 16, 1, 5),
                                        (64, 16, 3, 16), (128, 128, 1, 12), (32, 16, 2, 9), (16, 32, 1, 40)])
def test_one_token_over_ragged_lengths(kvb, d, page, H, g, layout, dtype):
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 250]
    P = Pool(kvb, 2, H, d, page, len(lens), 250, dtype, seed=g)
    P.fill(lens)
    q = P.rows(2, H * g, len(lens), layout, 1.5)
    off, pos = np.arange(len(lens) + 1), np.asarray(lens) - 1
    out, lse = attend(P, q, off, pos, layout=layout)
    kvb.kvb_ctx_check(P.ctx)
    check_attention(P, q, off, pos, out, lse)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,g,n", [(128, 8, [3, 0, 20, 1, 130]), (64, 2, [8, 7, 33, 0, 64]), (32, 5, [1, 2, 40, 9, 0]),
                                   (128, 1, [200, 5, 0, 129, 64]), (16, 6, [11, 0, 3, 1, 50]), (128, 4, [4, 4, 3, 4, 0])])
def test_several_tokens_are_causal(kvb, d, g, n, dtype):
    lens = np.asarray([40, 9, 20, 300, 333])
    n = np.minimum(n, lens)
    P = Pool(kvb, 1, 2, d, 32, 5, 333, dtype, seed=d + g)
    P.fill(lens)
    q = P.rows(1, 2 * g, int(n.sum()), sigma=1.5)
    out, lse = attend(P, q, offsets(n), lens - n)
    kvb.kvb_ctx_check(P.ctx)
    check_attention(P, q, offsets(n), lens - n, out, lse)


@pytest.mark.parametrize("d,page,H,g,n,lens", [(128, 16, 2, 8, 3, [3, 70, 64, 129]), (128, 32, 1, 5, 5, [5, 63, 200, 1000]),
                                               (128, 128, 3, 8, 5, [500, 5, 128, 127]), (64, 16, 2, 20, 1, [1, 16, 17, 300]),
                                               (64, 64, 2, 4, 33, [33, 40, 400, 64]), (64, 128, 1, 17, 8, [8, 130, 640, 9]),
                                               (128, 64, 1, 128, 1, [1, 65, 2000, 64]), (128, 64, 2, 3, 100, [100, 101, 1000, 333])])
@pytest.mark.parametrize("layout", ["head", "token", "spaced"])
def test_many_rows(kvb, d, page, H, g, n, lens, layout):
    lens = np.asarray(lens)
    P = Pool(kvb, 2, H, d, page, 4, int(lens.max()), BF, seed=d + g)
    P.fill(lens)
    q = P.rows(2, H * g, 4 * n, layout, 1.5)
    out, lse = attend(P, q, offsets([n] * 4), lens - n, layout=layout)
    kvb.kvb_ctx_check(P.ctx)
    check_attention(P, q, offsets([n] * 4), lens - n, out, lse)
    again, z = attend(P, q, offsets([n] * 4), lens - n, layout=layout)
    assert torch.equal(out, again) and torch.equal(lse, z)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,g,n,lens", [(128, 8, 1, [9000, 4097, 8191]), (64, 4, 1, [9000, 4097, 8191]), (128, 4, 4, [9000, 4097, 8191]),
                                        (32, 3, 9, [9000, 4097, 8191]), (64, 8, 8, [9000, 4097, 8191]), (128, 8, 5, [9000, 4097, 8191]),
                                        (128, 8, 5, [2500, 40, 1300]), (64, 5, 5, [9000, 64, 128]), (128, 20, 3, [600, 601, 8])])
def test_long_cache_split_over_ctas_joins_and_repeats_bit_for_bit(kvb, d, g, n, lens, dtype):
    lens = np.asarray(lens)
    P = Pool(kvb, 1, 1, d, 64, 3, int(lens.max()), dtype, seed=5)
    P.fill(lens)
    q = P.rows(1, g, 3 * n, sigma=1.5)
    off, pos = offsets([n] * 3), lens - n
    out, lse = attend(P, q, off, pos)
    check_attention(P, q, off, pos, out, lse)
    for _ in range(3):
        again, z = attend(P, q, off, pos)
        assert torch.equal(out, again) and torch.equal(lse, z)
    kvb.kvb_ctx_check(P.ctx)


@pytest.mark.parametrize("dtype,g", [(BF, 3), (F32, 3), (BF, 10)])
def test_rows_that_see_nothing_and_cache_lengths(kvb, dtype, g):
    P = Pool(kvb, 1, 2, 64, 32, 5, 100, dtype)
    P.fill([100] * 5)
    q = P.rows(1, 2 * g, 10)
    off, pos = offsets([2] * 5), np.array([-1, 50, 50, -2, 98])
    for lens in ([100, 0, 20, 100, 100], [0, 0, 0, 0, 0], [1, 51, 52, 1, -3]):
        out, lse = attend(P, q, off, pos, kv_len=i32(lens))
        kvb.kvb_ctx_check(P.ctx)
        check_attention(P, q, off, pos, out, lse, kv_len=lens)
    assert torch.all(out[:, :, 6:8] == 0) and torch.all(torch.isinf(lse[:, :, 6:8]))


def test_rows_of_tokens_that_no_sequence_owns_are_left_alone(kvb):
    P = Pool(kvb, 1, 1, 64, 32, 2, 100, BF)
    P.fill([100, 30])
    q = P.rows(1, 4, 7)
    out, lse = torch.full_like(q, 7.0), torch.full((1, 4, 7), 7.0, device="cuda")
    kvb.kvb_paged_attention(P.ctx, P.cache, P.seqs([2, 3, 5], [99, 28]), q, out, lse)
    kvb.kvb_ctx_check(P.ctx)
    assert torch.all(out[:, :, :2] == 7) and torch.all(out[:, :, 5:] == 7) and torch.all(lse[:, :, 5:] == 7)
    o = P.ref.attention(to_host64(q[:, :, 2:5]), P.table, [0, 1, 3], [99, 28])[0]
    assert np.abs(to_host64(out[:, :, 2:5]) - o).max() < 0.05


@pytest.mark.parametrize("dtype,copies", [(BF, 1), (F32, 1), (BF, 10)])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_that_rise_and_fall_over_the_tiles(kvb, sign, dtype, copies):
    # the reference is raised at every step, or never again after the first
    d, n = 64, 700
    P = Pool(kvb, 1, 1, d, 16, 1, n, dtype)
    k = np.zeros((1, 1, n, d))
    k[..., 0] = sign * np.linspace(-60, 60, n)
    v = P.rng.standard_normal((1, 1, n, d))
    dk, dv = laid_out(k, "head", dtype), laid_out(v, "head", dtype)
    kvb.kvb_paged_append(P.ctx, P.cache, P.seqs([0, n], [0]), dk, dv, rotate=False)
    for kv, x in enumerate((dk, dv)):
        P.ref.append(kv, to_host64(x), P.table, [0, n], [0])
    q = np.zeros((1, 3 * copies, 1, d))
    q[0, :, 0, 0] = [8.0, -8.0, 400.0] * copies
    q = laid_out(q, "head", dtype)
    out, lse = attend(P, q, [0, 1], [n - 1])
    check_attention(P, q, [0, 1], [n - 1], out, lse)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_scores_near_the_ends_of_fp32(kvb, dtype):
    # scores of -2e38 and of 3e37: a reference far below zero is a reference too
    d = 16
    P = Pool(kvb, 1, 1, d, 16, 2, 16, dtype)
    k = np.zeros((1, 1, 6, d))
    k[0, 0, :, 0] = [1.0, 1.0, 1.0, 1.0, 2.0, 1.0]
    v = P.rng.standard_normal((1, 1, 6, d))
    dk, dv = laid_out(k, "head", dtype), laid_out(v, "head", dtype)
    kvb.kvb_paged_append(P.ctx, P.cache, P.seqs([0, 3, 6], [0, 0]), dk, dv, rotate=False)
    q = np.zeros((1, 1, 2, d))
    q[0, 0, :, 0] = [-2.0 ** 127, 2.0 ** 124]
    out, lse = attend(P, laid_out(q, "head", dtype), [0, 1, 2], [2, 2], scale=1.0)
    kvb.kvb_ctx_check(P.ctx)
    got, hv = to_host64(out)[0, 0], to_host64(dv)[0, 0]
    tol = (2.0 ** -8 + 2.0 ** -16 if dtype == BF else 2.0 ** -20) * np.abs(hv).max()
    assert np.abs(got[0] - hv[:3].mean(0)).max() <= tol  # three equal scores
    assert np.abs(got[1] - hv[4]).max() <= tol           # one that is far above the others
    assert np.allclose(to_host64(lse)[0, 0], [-2.0 ** 127, 2.0 ** 125], rtol=2.0 ** -21)


def test_scale_layers_and_no_lse(kvb):
    P = Pool(kvb, 4, 2, 128, 64, 2, 150, BF)
    P.fill([150, 77])
    q = P.rows(2, 8, 2)
    out, _ = attend(P, q, [0, 1, 2], [149, 76], lse=False, l_begin=1, scale=0.3)
    kvb.kvb_ctx_check(P.ctx)
    check_attention(P, q, [0, 1, 2], [149, 76], out, None, l_begin=1, scale=0.3)


@pytest.mark.parametrize("dtype,g", [(BF, 8), (F32, 8), (BF, 40)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_query_that_is_not_finite_stays_in_its_row(kvb, bad, dtype, g):
    P = Pool(kvb, 1, 1, 128, 64, 2, 300, dtype)
    P.fill([300, 300])
    q = P.rows(1, g, 2)
    good, z = attend(P, q, [0, 1, 2], [299, 299])
    q2 = q.clone()
    q2[0, 3, 1, 5] = bad
    out, lse = attend(P, q2, [0, 1, 2], [299, 299])
    keep = torch.ones(g, 2, dtype=torch.bool, device="cuda")
    keep[3, 1] = False
    assert torch.equal(out[0][keep], good[0][keep]) and torch.equal(lse[0][keep], z[0][keep])
    assert torch.isnan(out[0, 3, 1]).any() or torch.isinf(lse[0, 3, 1])


@pytest.mark.parametrize("dtype,H,d,page,g,n", [(BF, 1, 128, 64, 2, 5), (BF, 2, 64, 16, 1, 3), (BF, 1, 32, 32, 3, 9), (BF, 160, 16, 16, 3, 4), (F32, 1, 64, 64, 1, 7),
                                                (F32, 2, 128, 16, 2, 4), (F32, 160, 16, 32, 3, 4), (BF, 2, 128, 64, 8, 5), (BF, 1, 64, 16, 16, 4), (BF, 2, 64, 128, 4, 8),
                                                (BF, 1, 128, 16, 9, 40), (F32, 1, 128, 64, 9, 40), (BF, 1, 32, 64, 9, 40)])
def test_new_tokens_that_are_not_finite_stay_hidden_from_earlier_ones(kvb, dtype, H, d, page, g, n):
    lens = np.array([130, n, 2500, 64 + n // 2])
    P = Pool(kvb, 1, H, d, page, 4, 2500, dtype)
    P.fill(lens)
    pos, off = lens - n, offsets([n] * 4)
    q = P.rows(1, H * g, 4 * n)
    good, z = attend(P, q, off, pos)

    def put(x, token, dim, value):  # in every sequence and head
        for s in range(4):
            at = int(pos[s]) + token
            x[:, P.table[s, at // page], :, at % page, dim] = value

    inf, nan = float("inf"), float("nan")
    put(P.cache.v, 2, 0, nan), put(P.cache.v, 2, 1, inf), put(P.cache.v, n - 1, 1, -inf if n > 3 else nan), put(P.cache.v, n - 1, d - 1, inf)
    want = good.clone().view(1, H * g, 4, n, d)
    want[..., 2:, 0] = nan
    want[..., 2:, 1] = inf
    want[..., n - 1, 1] = nan
    want[..., n - 1, d - 1] = inf
    for _ in range(2):
        out, lse = attend(P, q, off, pos)
        assert torch.equal(lse, z)
        # infinite or NaN: a weight w goes into its product as hi + lo with lo = bf16(w - hi), which is 0 or negative for
        # half of all w, so that hi * inf + lo * inf = inf + NaN or inf - inf where the block sees all of the keys
        assert torch.equal(torch.isfinite(out), torch.isfinite(want.view_as(out)))
        assert torch.equal(out.nan_to_num(0, 0, 0), want.view_as(out).nan_to_num(0, 0, 0))
    put(P.cache.k, n - 1, 3, nan)
    out, lse = (x.view(1, H * g, 4, n, -1) for x in attend(P, q, off, pos))
    assert torch.isnan(out[..., n - 1, :]).all() and torch.isnan(lse[..., n - 1, :]).all()
    out, want = out[..., :n - 1, :], want[..., :n - 1, :]
    assert torch.equal(torch.isfinite(out), torch.isfinite(want)) and torch.equal(out.nan_to_num(0, 0, 0), want.nan_to_num(0, 0, 0))
    kvb.kvb_ctx_check(P.ctx)


@pytest.mark.parametrize("dtype,g", [(BF, 4), (F32, 4), (BF, 20)])
def test_a_bad_page_is_absent_and_reported(kvb, dtype, g):
    P = Pool(kvb, 1, 2, 64, 16, 3, 200, dtype)
    P.fill([200, 200, 200])
    q = P.rows(1, 2 * g, 3)
    off, pos = [0, 1, 2, 3], [199, 199, 199]
    good, _ = attend(P, q, off, pos)
    for wrong in (P.n_pages, -1, 2 ** 31 - 1):
        tab = P.dtab.clone()
        tab[1] = wrong
        tab[2, 3:7] = wrong
        out, lse = torch.empty_like(q), torch.empty(1, 2 * g, 3, device="cuda")
        kvb.kvb_paged_attention(P.ctx, P.cache, kvb.Seqs(tab, i32(off), i32(pos), max_tokens=1), q, out, lse)
        assert status_of(kvb, lambda: kvb.kvb_ctx_check(P.ctx)) == INVALID_ARG
        assert torch.equal(out[:, :, 0], good[:, :, 0])
        assert torch.all(out[:, :, 1] == 0) and torch.all(lse[:, :, 1] == -float("inf"))
        keys = np.r_[0:48, 112:200]  # sequence 2 without its pages 3 .. 6
        for h in range(2 * g):
            k, v = (P.ref.sequence(x, P.table[2], 200, 0, h // g)[keys] for x in (0, 1))
            s = to_host64(q)[0, h, 2] @ k.T / 8
            w = np.exp(s - s.max())
            assert np.abs(to_host64(out)[0, h, 2] - (w / w.sum()) @ v).max() < (2.0 ** -6 if dtype == BF else 2.0 ** -17)
    kvb.kvb_ctx_check(P.ctx)
    # sequences outside the call
    out, lse = torch.empty_like(q), torch.empty(1, 2 * g, 3, device="cuda")
    for off, pos, kw in (([0, 5, 4, 4], [0, 0, 0], {}), ([0, 0, 0, 9], [0, 0, 0], {}), ([-1, 0, 0, 0], [0, 0, 0], {}),
                         ([0, 1, 2, 3], [0, 0, 2 ** 31 - 1], {}), ([0, 1, 2, 3], [199, 199, 199], {"max_kv": 150})):
        kvb.kvb_paged_attention(P.ctx, P.cache, kvb.Seqs(P.dtab, i32(off), i32(pos), max_tokens=1, **kw), q, out, lse)
        assert status_of(kvb, lambda: kvb.kvb_ctx_check(P.ctx)) == INVALID_ARG


def test_pages_beyond_four_gib(kvb):
    # a pool whose offsets pass 2^32 elements; the sequence lives at its far end
    n_pages, page, d, H = 70000, 64, 128, 8
    ctx = kvb.kvb_ctx_create(spec(1, H, d, 1e6), spec(1, H, d, THETA), 1, 256)
    cache = kvb.kvb_paged_create(ctx, n_pages, page)
    assert cache.k.numel() > 2 ** 32
    seqs = lambda off, pos: kvb.Seqs(i32([[n_pages - 1, 3, n_pages - 2]]), i32(off), i32(pos), max_tokens=int(off[-1]))
    k, v, q = (torch.randn(1, h, 150, d, device="cuda").to(BF) for h in (H, H, 2 * H))
    kvb.kvb_paged_append(ctx, cache, seqs([0, 150], [0]), k, v, rotate=False)
    for x, c in ((k, cache.k), (v, cache.v)):
        got = torch.cat([c[0, n_pages - 1], c[0, 3], c[0, n_pages - 2]], dim=1)[:, :150]
        assert torch.equal(got, x[0])
    ref = PG.Paged(1, 3, H, page, d)
    for kv, x in enumerate((k, v)):
        ref.append(kv, to_host64(x), [[2, 0, 1]], [0, 150], [0])
    out, lse = torch.empty_like(q[:, :, :1]), torch.empty(1, 2 * H, 1, device="cuda")
    one = q[:, :, 149:150].contiguous()
    kvb.kvb_paged_attention(ctx, cache, seqs([0, 1], [149]), one, out, lse)
    kvb.kvb_ctx_check(ctx)
    o, z, A, _ = ref.attention(to_host64(one), np.array([[2, 0, 1]]), [0, 1], [149])
    assert (np.abs(to_host64(out) - o) <= 2.0 ** -8 * np.abs(o) + 2.0 ** -12 * A).all()


@pytest.mark.parametrize("d,g,dtype", [(16, 1, BF), (64, 2, F32), (128, 8, BF), (64, 40, BF)])
def test_the_last_positions_that_a_call_may_name(kvb, d, g, dtype):
    # 2^31 - 1024 positions, the most that is accepted, on three pages that repeat.  Each CTA adds the keys of
    # its share one after another in fp32, 64 keys a step and 16 roundings at most in it: shares of
    # 1 / 152, in numerator and denominator; then the formats' part.
    page, kv = 128, 0x7ffffc00
    P = Pool(kvb, 1, 1, d, page, 1, 3 * page, dtype, spare=0)
    P.fill([3 * page])
    table = i32(P.table[0])[torch.arange(kv // page, device="cuda") % 3][None].contiguous()
    q = P.rows(1, g, 1, sigma=4.0)  # few keys decide
    out, lse = torch.empty_like(q), torch.empty((1, g, 1), device="cuda")
    kvb.kvb_paged_attention(P.ctx, P.cache, kvb.Seqs(table, i32([0, 1]), i32([kv - 1]), max_tokens=1), q, out, lse)
    kvb.kvb_ctx_check(P.ctx)
    k, v = (P.ref.sequence(x, P.table[0], 3 * page, 0, 0) for x in (0, 1))
    pages = kv // page
    times = np.repeat([(pages + 2) // 3, (pages + 1) // 3, pages // 3], page)
    s = to_host64(q)[0, :, 0] @ k.T / np.sqrt(d)
    w = np.exp(s - s.max(axis=1, keepdims=True)) * times
    z = s.max(axis=1) + np.log(w.sum(axis=1))
    w /= w.sum(axis=1, keepdims=True)
    steps = kv / 152 / 4
    tol = (w @ np.abs(v)) * (2 * steps * 2.0 ** -24 + 2.0 ** -12) + np.abs(w @ v) * 2.0 ** -8
    assert (np.abs(to_host64(out)[0, :, 0] - w @ v) <= tol).all()
    assert (np.abs(to_host64(lse)[0, :, 0] - z) <= steps * 2.0 ** -24 + 2.0 ** -12).all()


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_mapped_prefix_is_decoded_from(kvb, dtype):
    """A prefix stored as it is, then tokens one by one: append (keys and queries rotated) and attend, layer by layer;
    the outputs against the oracle, and against the plain cache's by cosine."""
    L, H, g, d, page, T, N = 2, 2, 4, 128, 64, 100, 40
    P = Pool(kvb, L, H, d, page, 2, T + N, dtype, seed=9)
    pre = [P.rows(L, H, 2 * T) for _ in range(2)]
    off = [0, T, 2 * T]
    kvb.kvb_paged_append(P.ctx, P.cache, P.seqs(off, [0, 0]), *pre, rotate=False)
    for kv in range(2):
        P.ref.append(kv, to_host64(pre[kv]), P.table, off, [0, 0])
    at = i32([T, T])
    seqs = kvb.Seqs(P.dtab, i32([0, 1, 2]), at, max_tokens=1, max_kv=T + N)
    cos = torch.empty((L, H * g, N), device="cuda")
    qs = []
    for i in range(N):
        x = [P.rows(1, H * g + 2 * H, 2, "token") for _ in range(L)]  # what the layers' projections give
        o, qr = torch.empty((L, 2, H * g, d), dtype=dtype, device="cuda").transpose(1, 2), torch.empty((L, H * g, 2, d), dtype=dtype, device="cuda")
        for l in range(L):
            q, k, v = x[l][:, :H * g], x[l][:, H * g:H * g + H], x[l][:, H * g + H:]
            kvb.kvb_paged_append(P.ctx, P.cache, seqs, k, v, q, qr[l:l + 1], l_begin=l)
            kvb.kvb_paged_attention(P.ctx, P.cache, seqs, qr[l:l + 1], o[l:l + 1], l_begin=l)
            tk = torch.from_numpy(P.turned(k, [0, 1, 2], [T + i] * 2)).to(dtype)
            P.ref.append(0, to_host64(tk), P.table, [0, 1, 2], [T + i] * 2, l)
            P.ref.append(1, to_host64(v), P.table, [0, 1, 2], [T + i] * 2, l)
        at.add_(1)
        P.lens = np.array([T + i + 1] * 2)
        check_attention(P, qr, [0, 1, 2], [T + i] * 2, o, None)
        qs.append(qr[:, :, 0])
    kvb.kvb_ctx_check(P.ctx)
    # sequence 0's cache in the plain layout gives the same attention outputs
    ids = P.dtab[0, :-(-(T + N) // page)].long()
    plain = [t[:, ids].transpose(1, 2).reshape(L, H, -1, d)[:, :, :T + N].contiguous() for t in (P.cache.k, P.cache.v)]
    where = torch.arange(T + N, dtype=torch.int32, device="cuda")
    q = torch.stack(qs, dim=2).contiguous()
    kvb.kvb_attention_cosine(P.ctx, q, where[T:].contiguous(), *plain, *plain, where, cos)
    assert (cos > 1 - 1e-4).all()


def test_on_another_stream_and_captured_while_the_cache_grows(kvb):
    P = Pool(kvb, 1, 2, 128, 64, 2, 200, BF)
    P.fill([100, 63])
    side = torch.cuda.Stream()
    pos = i32([100, 63])
    x = P.rows(1, 20, 2, "token")
    q, k, v = x[:, :16], x[:, 16:18], x[:, 18:]
    turned, out, lse = torch.empty_like(q), torch.empty_like(q), torch.empty(1, 16, 2, device="cuda")
    seqs = kvb.Seqs(P.dtab, i32([0, 1, 2]), pos, max_tokens=1, max_kv=200)
    kvb.kvb_paged_attention(P.ctx, P.cache, seqs, q, out, lse)  # sizes the workspace
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        kvb.kvb_paged_append(P.ctx, P.cache, seqs, k, v, q, turned)
        kvb.kvb_paged_attention(P.ctx, P.cache, seqs, turned, out, lse)
    for i in range(5):
        at = [100 + i, 63 + i]
        with torch.cuda.stream(side):
            x.normal_()
            pos.copy_(i32(at))
            graph.replay()
        side.synchronize()
        tk = torch.from_numpy(P.turned(k, [0, 1, 2], at)).to(BF)
        P.ref.append(0, to_host64(tk), P.table, [0, 1, 2], at)
        P.ref.append(1, to_host64(v), P.table, [0, 1, 2], at)
        assert torch.equal(turned.cpu(), torch.from_numpy(P.turned(q, [0, 1, 2], at)).to(BF))
        check_attention(P, turned, np.arange(3), at, out, lse)
    kvb.kvb_ctx_check(P.ctx)
    P.check_pages()


def test_both_caches_attentions_share_a_context(kvb):
    """Calls of both kinds in turn on one context: counters and partial results are left as each needs them."""
    P = Pool(kvb, 1, 2, 128, 64, 1, 6000, BF)
    P.fill([6000])
    eight = kvb.kvb_cache8_create(P.ctx, P.n_pages, 64)
    k, v = P.rows(1, 2, 6000), P.rows(1, 2, 6000)
    kvb.kvb_cache8_append(P.ctx, eight, P.seqs([0, 6000], [0]), k, v)
    q = P.rows(1, 16, 1)
    s = P.seqs([0, 1], [5999])
    a, b = torch.empty_like(q), torch.empty_like(q)
    kvb.kvb_paged_attention(P.ctx, P.cache, s, q, a)
    kvb.kvb_cache8_attention(P.ctx, eight, s, q, b)
    for _ in range(4):
        x, y = torch.empty_like(q), torch.empty_like(q)
        kvb.kvb_paged_attention(P.ctx, P.cache, s, q, x)
        kvb.kvb_cache8_attention(P.ctx, eight, s, q, y)
        assert torch.equal(a, x) and torch.equal(b, y)
    kvb.kvb_ctx_check(P.ctx)


def test_contexts_of_their_own_on_two_streams(kvb):
    P = Pool(kvb, 1, 2, 128, 64, 2, 5000, BF)
    P.fill([5000, 4000])
    other = kvb.kvb_ctx_create(spec(1, 2, 128, 1e4), spec(1, 2, 128, THETA), 1, 64)
    q = P.rows(1, 16, 2)
    want, z = attend(P, q, [0, 1, 2], [4999, 3999])
    streams = [torch.cuda.Stream() for _ in range(2)]
    seqs = P.seqs([0, 1, 2], [4999, 3999])
    outs = [torch.empty((20,) + tuple(q.shape), dtype=BF, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(20):
        for ctx, s, o in zip((P.ctx, other), streams, outs):
            kvb.kvb_paged_attention(ctx, P.cache, seqs, q, o[i], stream=s)
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(o[i], want) for i in range(20))


def test_growing_on_a_captured_stream_is_refused(kvb):
    P = Pool(kvb, 1, 2, 128, 64, 1, 70000, BF)  # few keys have no workspace
    P.fill([70000])
    q = P.rows(1, 16, 1)
    out = torch.empty_like(q)
    seqs = P.seqs([0, 1], [69999])
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        assert status_of(kvb, lambda: kvb.kvb_paged_attention(P.ctx, P.cache, seqs, q, out)) == UNSUPPORTED
        out.zero_()
    kvb.kvb_paged_attention(P.ctx, P.cache, seqs, q, out)
    kvb.kvb_ctx_check(P.ctx)
    check_attention(P, q, [0, 1], [69999], out, None)


# ------------------------------------------------------------------ refusals

def test_refusals(kvb):
    P = Pool(kvb, 2, 2, 64, 16, 1, 64, BF)
    P.fill([64])
    lib, h = kvb.load_library(), P.ctx.handle
    from cross_model_kv_gb300 import _binding as B
    k, q = P.rows(2, 2, 3), P.rows(2, 4, 3)
    out = torch.empty_like(q)
    rows = lambda x, **kw: B._pack_rows(kw.get("data", x.data_ptr()), *(kw.get(n, s) for n, s in zip("lht", x.stride()[:3])))
    s = P.seqs([0, 3], [0])

    def append(cache=P.cache.ref, seqs=s.ref, l=0, n=2, rk=rows(k), rv=rows(k), rq=None, ro=None, heads=0, T=3, turn=1):
        return lib.kvb_paged_append(h, cache, seqs, l, n, rk, rv, rq, ro, heads, T, turn, None)

    def attention(cache=P.cache.ref, seqs=s.ref, l=0, n=2, rq=rows(q), heads=4, T=3, scale=0.0, ro=rows(out), lse=None):
        return lib.kvb_paged_attention(h, cache, seqs, l, n, rq, heads, T, scale, ro, lse, None)

    def struct(**kw):
        c = B.kvb_paged_cache(P.cache.struct.dtype, 16, P.n_pages, P.cache.struct.k, P.cache.struct.v)
        for n, x in kw.items():
            setattr(c, n, x)
        return c

    assert append() == 0 and append(rq=rows(q), ro=rows(out), heads=4) == 0 and attention() == 0
    for call in (append, attention):
        assert call(cache=None) == 1 and call(seqs=None) == 1
        assert call(l=1) == 1 and call(l=-1) == 1 and call(n=-1) == 1 and call(T=-1) == 1 and call(T=2) == 1
        assert call(T=2 ** 31) == 3
        for kw, want in (({"dtype": 2}, 3), ({"page_tokens": 48}, 3), ({"n_pages": -1}, 1), ({"n_pages": 2 ** 31}, 1), ({"k": None}, 1),
                         ({"v": P.cache.k.data_ptr() + 8}, 1)):
            c = struct(**kw)
            assert call(cache=B.ctypes.addressof(c)) == want, kw
        assert call(n=0) == 0  # nothing to do
    for kw in ({"rk": None}, {"rv": None}, {"rk": rows(k, data=0)}, {"rk": rows(k, data=k.data_ptr() + 2)}, {"rk": rows(k, t=68)},
               {"rv": rows(k, h=-64)}, {"rk": rows(k, l=2 ** 62)}, {"rq": rows(q)}, {"ro": rows(out)}, {"turn": 2}, {"turn": -1},
               {"rq": rows(q), "ro": rows(out), "heads": 3}, {"rq": rows(q), "ro": rows(out), "heads": 0},
               {"rq": rows(q), "ro": rows(out), "heads": 4, "turn": 0},
               {"rq": rows(q), "ro": rows(out, t=0), "heads": 4},          # every token to one row
               {"rq": rows(q), "ro": rows(out, t=64, h=64), "heads": 4},   # heads over tokens
               {"rq": rows(q), "ro": rows(q, t=256, h=64), "heads": 4}):   # q's place, other strides
        assert append(**kw) == 1, kw
    for kw in ({"rq": None}, {"ro": None}, {"ro": rows(out, h=0)}, {"heads": 3}, {"heads": 0}, {"heads": -2}, {"scale": -1.0},
               {"scale": float("nan")}, {"scale": float("inf")}, {"scale": 1e300}, {"scale": 1e-300}, {"lse": out.data_ptr() + 2},
               {"ro": rows(out, data=out.data_ptr() + 8)}):
        assert attention(**kw) == 1, kw
    assert attention(heads=2 ** 31 - 2, n=1) == 3  # more query rows than a call takes
    torch.cuda.synchronize()
    kvb.kvb_ctx_check(P.ctx)
    # the binding's own
    for f in (lambda: kvb.kvb_paged_append(P.ctx, P.cache, s, k.float(), k.float()), lambda: kvb.kvb_paged_append(P.ctx, P.cache, s, k, k[:1]),
              lambda: kvb.kvb_paged_append(P.ctx, P.cache, s, k, k, q), lambda: kvb.kvb_paged_append(P.ctx, P.cache, s, k, k, q, out[:, :2]),
              lambda: kvb.kvb_paged_append(P.ctx, P.cache, s, k, k, q[:, :, :2], out[:, :, :2]),
              lambda: kvb.kvb_paged_append(P.ctx, P.cache, s, k.cpu(), k), lambda: kvb.kvb_paged_attention(P.ctx, P.cache, s, q.float(), out.float()),
              lambda: kvb.kvb_paged_attention(P.ctx, P.cache, s, q, out.transpose(2, 3)), lambda: kvb.kvb_paged_attention(P.ctx, P.cache, s, q, out, out),
              lambda: kvb.PagedCache(P.ctx, P.cache.k, P.cache.v[:1]), lambda: kvb.PagedCache(P.ctx, P.cache.k.half(), P.cache.v.half()),
              lambda: kvb.PagedCache(P.ctx, P.cache.k.transpose(1, 2), P.cache.v)):
        with pytest.raises(ValueError):
            f()
    other = kvb.kvb_ctx_create(spec(1, 2, 32, 1e4), spec(2, 2, 32, 1e4), 1, 64)
    with pytest.raises(ValueError, match="another context"):
        kvb.kvb_paged_attention(other, P.cache, s, q, out)
    with pytest.raises(ValueError, match="another context"):
        kvb.kvb_paged_append(other, P.cache, s, k, k)
