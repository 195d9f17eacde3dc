"""The paged 8-bit cache against its float64 oracle: codes and scales bit for
bit, reads exactly, attention within bounds derived from the formats.

Attention tolerance, per row, with spread A = sum p|v| and reach B = max_j
scale * sum_e |q_e k_je| (natural log units):
  * a score is d products summed in fp32, at most d/16 + 4 roundings of 2^-23
    relative to B with the scalings: |ds| <= (d/16 + 4) 2^-23 B;
  * the exponential adds 2^-21 to a weight's relative error, and numerator and
    denominator both carry the weights' errors: 2 (|ds| + 2^-21) A;
  * sums over kv keys in steps of 16, spread over four warps, and the joins:
    (kv/64 + 32) 2^-23 A;
  * weights as fp16 (bf16 calls): 2^-11 A; as fp16 pairs (fp32 calls): 2^-21 A;
    a weight below the least fp16 number: kv 2^-31 times the largest |v|, which
    is at most 2^-15 A' with A' = max |v|, covered by kv 2^-31 maxv;
  * the output's own rounding: 2^-8 |o| (bf16, a whole unit), 2^-23 |o| (fp32).
"""
import numpy as np
import pytest

from cases import spec, to_host64
from oracle import cache8 as C8

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
INVALID_ARG, UNSUPPORTED, NUMERIC = 1, 3, 5


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


class Pool:
    """A cache on the device and the oracle's, with sequences whose pages come in no order."""

    def __init__(self, kvb, L, H, d, page, n_seq, max_len, seed=0, spare=3, share=None):
        self.kvb, self.L, self.H, self.d, self.page = kvb, L, H, d, page
        self.ctx = kvb.kvb_ctx_create(spec(1, H, d, 1e6), spec(L, H, d, 1e6), 1, 64)
        cols = -(-max_len // page)
        self.rng = np.random.default_rng(seed)
        ids = self.rng.permutation(n_seq * cols + spare)[:n_seq * cols].reshape(n_seq, cols)
        if share:  # every sequence's first pages are sequence 0's
            ids[:, :share] = ids[0, :share]
        self.table = ids
        n_pages = n_seq * cols + spare
        self.cache = kvb.kvb_cache8_create(self.ctx, n_pages, page)
        # nothing is promised about unwritten slots: fill them with NaN codes and scales
        for t in (self.cache.k, self.cache.v):
            t.view(torch.uint8).fill_(0x7f)
        for t in (self.cache.k_scale, self.cache.v_scale):
            t.fill_(float("nan"))
        self.ref = C8.Cache8(L, n_pages, H, page, d)
        self.dtab = i32(ids)

    def seqs(self, off, pos, **kw):
        off, pos = np.asarray(off), np.asarray(pos)
        kw.setdefault("max_tokens", int(np.diff(off).max()) if len(off) > 1 else 0)
        return self.kvb.Seqs(self.dtab, i32(off), i32(pos), **kw)

    def write(self, off, pos, dtype, sigma=1.0, l_begin=0, n_layers=None, x=None, bump=None):
        n_layers = self.L if n_layers is None else n_layers
        T = int(off[-1])
        if x is None:
            s = np.exp(0.5 * self.rng.standard_normal((n_layers, self.H, 1, self.d)))
            x = [sigma * s * self.rng.standard_normal((n_layers, self.H, T, self.d)) for _ in range(2)]
            if bump is not None:
                x = [a * bump[:, None] for a in x]
        dx = [torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda() for a in x]
        self.kvb.kvb_cache8_write(self.ctx, self.cache, self.seqs(off, pos), dx[0], dx[1], l_begin=l_begin)
        for kv in range(2):
            self.ref.write(kv, to_host64(dx[kv]), self.table, off, pos, l_begin)
        return dx

    def fill(self, lens, dtype=BF, sigma=1.0):
        self.lens = np.asarray(lens)
        off = np.concatenate([[0], np.cumsum(self.lens)])
        self.write(off, np.zeros(len(lens), dtype=int), dtype, sigma)

    def check_codes(self, lens, layers=None):
        """Written slots and their blocks' scales equal the oracle's bit for bit; the others are untouched."""
        layers = range(self.L) if layers is None else layers
        for kv, (c, s) in enumerate(((self.cache.k, self.cache.k_scale), (self.cache.v, self.cache.v_scale))):
            got, gs = c.view(torch.uint8).cpu().numpy(), s.cpu().numpy()
            written = np.zeros(got.shape[1:4], dtype=bool)  # [pages][H][page]
            for q, n in enumerate(lens):
                for p in range(-(-int(n) // self.page)):
                    written[self.table[q, p], :, :min(self.page, int(n) - p * self.page)] = True
            touched = written.any(axis=2)
            for l in range(self.L):
                if l not in layers:
                    assert np.all(got[l] == 0x7f) and np.isnan(gs[l]).all()
                    continue
                assert np.array_equal(got[l][written], self.ref.codes[kv][l][written])
                assert np.all(got[l][~written] == 0x7f)
                assert np.array_equal(gs[l][touched], self.ref.scales[kv][l][touched])
                assert np.isnan(gs[l][~touched]).all()


def offsets(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(int)


# ------------------------------------------------------------------ write

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,page,H", [(16, 16, 1), (32, 128, 3), (64, 32, 2), (128, 64, 2), (128, 128, 1), (128, 16, 5)])
def test_write_bit_for_bit_growing_pages(kvb, d, page, H, dtype):
    # prompts, then a few tokens, then single tokens; later tokens are larger, so that
    # scales rise and earlier codes are rounded again, by a warp and by a CTA
    P = Pool(kvb, 2, H, d, page, 4, 5 * page + 40, seed=d + page)
    lens = np.zeros(4, dtype=int)
    for step, n in enumerate(([1, 0, page, 3 * page + 7], [5, page - 1, 1, 2 * page - 3], [1, 1, 1, 1], [17, 2, 30, 0],
                              [1, 1, 1, 1], [0, page + 20, 0, 1])):
        P.write(offsets(n), lens, dtype, sigma=1.7 ** step)
        lens = lens + np.asarray(n)
    kvb.kvb_ctx_check(P.ctx)
    P.check_codes(lens)


def test_write_starts_a_reused_page_afresh(kvb):
    P = Pool(kvb, 1, 2, 64, 32, 1, 64)
    P.write([0, 40], [0], BF, sigma=1e4)
    P.write([0, 33], [0], BF, sigma=1e-3)  # the same pages, from their first slots
    kvb.kvb_ctx_check(P.ctx)
    got = P.cache.k_scale.cpu().numpy()
    assert np.array_equal(got[:, P.table[0]], P.ref.scales[0][:, P.table[0]])
    assert got[:, P.table[0]].max() < 1e-3


def test_write_extremes(kvb):
    # zeros, the smallest and largest floats, ties, one value far above the rest
    P = Pool(kvb, 1, 1, 16, 16, 6, 16)
    x = np.zeros((1, 1, 6 * 16, 16), dtype=np.float32)
    f = x[0, 0].reshape(6, 16, 16)
    f[1] = np.float32(1e-45)
    f[2] = np.float32(3.4028235e38) * np.linspace(-1, 1, 256, dtype=np.float32).reshape(16, 16)
    f[3] = (np.arange(256).reshape(16, 16) + 0.5) * 1.75  # many ties
    f[4] = np.float32(1e-30)
    f[4, 3, 3] = 2.0
    f[5] = np.float32(2.0 ** -126) * np.arange(256, dtype=np.float32).reshape(16, 16)
    f[0, 0, 0] = -0.0
    P.write(offsets([16] * 6), np.zeros(6, dtype=int), F32, x=[x, -x])
    kvb.kvb_ctx_check(P.ctx)
    P.check_codes([16] * 6)
    out = [torch.full(x.shape, float("nan"), device="cuda") for _ in range(2)]
    kvb.kvb_cache8_read(P.ctx, P.cache, P.seqs(offsets([16] * 6), np.zeros(6, dtype=int)), *out)
    assert torch.isfinite(out[0]).all() and torch.isfinite(out[1]).all()


def test_write_of_values_that_are_not_finite(kvb):
    P = Pool(kvb, 1, 2, 128, 64, 2, 70)
    x = P.rng.standard_normal((1, 2, 90, 128))
    x[0, 0, 3, 5], x[0, 1, 64, 0], x[0, 1, 80, 127] = np.nan, np.inf, -np.inf
    P.write(offsets([65, 25]), [0, 0], BF, x=[x, x])
    with pytest.raises(kvb.KvbError) as e:
        kvb.kvb_ctx_check(P.ctx)
    assert e.value.status == NUMERIC
    kvb.kvb_ctx_check(P.ctx)  # reported once
    P.check_codes([65, 25])   # stored as 0; the blocks' other values as if those were 0


def test_write_and_read_of_some_layers(kvb):
    P = Pool(kvb, 5, 2, 64, 16, 2, 50)
    dx = P.write(offsets([20, 31]), [0, 0], BF, l_begin=1, n_layers=3)
    kvb.kvb_ctx_check(P.ctx)
    P.check_codes([20, 31], layers=(1, 2, 3))
    out = [torch.empty_like(dx[0][:2]) for _ in range(2)]
    kvb.kvb_cache8_read(P.ctx, P.cache, P.seqs(offsets([20, 31]), [0, 0]), *out, l_begin=2)
    for kv in range(2):
        assert np.array_equal(to_host64(out[kv]), P.ref.read(kv, P.table, offsets([20, 31]), [0, 0], 2, 2))


# ------------------------------------------------------------------ read

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,page", [(16, 16), (32, 64), (64, 128), (128, 32), (128, 64)])
def test_read_exactly(kvb, d, page, dtype):
    P = Pool(kvb, 2, 3, d, page, 4, 300, seed=page)
    P.fill([300, 1, page, 2 * page + 1])
    n, pos = [170, 1, 0, page + 1], [13, 0, 5, page]
    T = sum(n)
    out = [torch.full((2, 3, T, d), float("nan"), dtype=dtype, device="cuda") for _ in range(2)]
    kvb.kvb_cache8_read(P.ctx, P.cache, P.seqs(offsets(n), pos), *out)
    one = [torch.full((2, 3, 2, d), float("nan"), dtype=dtype, device="cuda") for _ in range(2)]
    kvb.kvb_cache8_read(P.ctx, P.cache, P.seqs([0, 1, 1, 1, 2], [299, 0, 0, 0]), *one)
    kvb.kvb_ctx_check(P.ctx)
    for kv in range(2):
        assert np.array_equal(to_host64(out[kv]), P.ref.read(kv, P.table, offsets(n), pos))
        assert np.array_equal(to_host64(one[kv]), P.ref.read(kv, P.table, [0, 1, 1, 1, 2], [299, 0, 0, 0]))


# ------------------------------------------------------------------ attention

def attend(P, q, off, pos, lse=True, l_begin=0, scale=0.0, **kw):
    out = torch.full(q.shape, float("nan"), dtype=q.dtype, device="cuda")
    z = torch.full(q.shape[:3], float("nan"), device="cuda") if lse else None
    P.kvb.kvb_cache8_attention(P.ctx, P.cache, P.seqs(off, pos, **kw), q, out, z, l_begin=l_begin, scale=scale)
    return out, z


def check_attention(P, q, off, pos, out, lse, kv_len=None, l_begin=0, scale=None):
    d, dtype = q.shape[3], q.dtype
    o, z, A, B = P.ref.attention(to_host64(q), P.table, off, pos, kv_len, l_begin, scale)
    kv = int(max(np.asarray(pos) + np.diff(off)) if kv_len is None else max(kv_len))
    maxv = max(np.abs(P.ref.read(1, P.table, offsets(P.lens), np.zeros(len(P.lens), dtype=int))).max(), 0.0)
    ds = (d / 16 + 4) * 2.0 ** -23 * B
    tol = A * (2 * (ds[..., None] + 2.0 ** -21) + (kv / 64 + 32) * 2.0 ** -23 + (2.0 ** -11 if dtype == BF else 2.0 ** -21))
    tol = tol + kv * 2.0 ** -31 * maxv + np.abs(o) * (2.0 ** -8 if dtype == BF else 2.0 ** -23)
    got = to_host64(out)
    assert np.isfinite(got).all()
    assert (np.abs(got - o) <= tol).all(), float((np.abs(got - o) / np.maximum(tol, 1e-300)).max())
    empty = np.isneginf(z)
    if lse is not None:
        gz = to_host64(lse)
        assert np.array_equal(np.isneginf(gz), empty)
        err = np.abs(np.where(empty, 0, gz) - np.where(empty, 0, z))
        assert (err <= ds + 2.0 ** -21 + (kv / 64 + 32) * 2.0 ** -23 + 2.0 ** -22 * np.abs(np.where(empty, 0, z))).all()
    assert np.all(got[empty] == 0)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,page,H,g", [(16, 16, 2, 1), (32, 32, 1, 3), (64, 128, 2, 4), (128, 64, 2, 8), (128, 16, 1, 5),
                                        (64, 16, 3, 16), (128, 128, 1, 12)])
def test_one_token_over_ragged_lengths(kvb, d, page, H, g, dtype):
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 250]
    P = Pool(kvb, 2, H, d, page, len(lens), 250, seed=g)
    P.fill(lens)
    q = torch.from_numpy(1.5 * P.rng.standard_normal((2, H * g, len(lens), d))).to(dtype).cuda()
    off, pos = np.arange(len(lens) + 1), np.asarray(lens) - 1
    out, lse = attend(P, q, off, pos)
    kvb.kvb_ctx_check(P.ctx)
    check_attention(P, q, off, pos, out, lse)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,g,n", [(128, 8, [3, 0, 20, 1, 130]), (64, 2, [8, 7, 33, 0, 64]), (32, 5, [1, 2, 40, 9, 0]),
                                   (128, 1, [200, 5, 0, 129, 64]), (16, 6, [11, 0, 3, 1, 50])])
def test_several_tokens_are_causal(kvb, d, g, n, dtype):
    lens = np.asarray([40, 9, 20, 300, 333])
    n = np.minimum(n, lens)
    P = Pool(kvb, 1, 2, d, 32, 5, 333, seed=d + g)
    P.fill(lens)
    q = torch.from_numpy(1.5 * P.rng.standard_normal((1, 2 * g, int(n.sum()), d))).to(dtype).cuda()
    out, lse = attend(P, q, offsets(n), lens - n)
    kvb.kvb_ctx_check(P.ctx)
    check_attention(P, q, offsets(n), lens - n, out, lse)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_long_cache_split_over_ctas_joins_and_repeats_bit_for_bit(kvb, dtype):
    P = Pool(kvb, 1, 1, 128, 64, 3, 9000, seed=5)
    P.fill([9000, 70, 4097])
    q = torch.from_numpy(2.0 * P.rng.standard_normal((1, 8, 3, 128))).to(dtype).cuda()
    off, pos = np.arange(4), np.asarray([8999, 69, 4096])
    out, lse = attend(P, q, off, pos)
    check_attention(P, q, off, pos, out, lse)
    for _ in range(5):
        o2, z2 = attend(P, q, off, pos)
        assert torch.equal(out, o2) and torch.equal(lse, z2)
    kvb.kvb_ctx_check(P.ctx)


def test_rows_that_see_nothing(kvb):
    # kv_len 0 and negative, queries before position 0, sequences without tokens
    P = Pool(kvb, 1, 2, 64, 16, 5, 100)
    P.fill([50, 50, 50, 50, 50])
    n, pos, kv_len = [2, 3, 0, 4, 1], [10, 20, 7, -2, -1], [0, -5, 50, 50, 50]
    q = torch.from_numpy(P.rng.standard_normal((1, 4, sum(n), 64))).to(BF).cuda()
    out, lse = attend(P, q, offsets(n), pos, kv_len=i32(kv_len))
    kvb.kvb_ctx_check(P.ctx)
    check_attention(P, q, offsets(n), pos, out, lse, kv_len=kv_len)
    seen = torch.isfinite(lse)[0, 0].cpu().numpy()
    assert np.array_equal(seen, [False] * 5 + [False, False, True, True] + [False])
    # nothing at all: no tokens, no sequences, no layers
    e = torch.empty((1, 4, 0, 64), dtype=BF, device="cuda")
    kvb.kvb_cache8_attention(P.ctx, P.cache, P.seqs([0] * 6, pos), e, e.clone())
    kvb.kvb_ctx_check(P.ctx)


def test_prefix_and_suffix_join_by_lse(kvb):
    # kv_len cuts the cache: attention over [0, 37) and over the rest, joined by their sums
    P = Pool(kvb, 1, 2, 128, 16, 1, 96)
    P.fill([96])
    q = torch.from_numpy(P.rng.standard_normal((1, 6, 1, 128))).to(F32).cuda()
    whole, z = attend(P, q, [0, 1], [95])
    a, za = attend(P, q, [0, 1], [95], kv_len=i32([37]))
    check_attention(P, q, [0, 1], [95], a, za, kv_len=[37])
    assert torch.all(za < z) and not torch.allclose(a, whole)


def test_shared_prefix_pages(kvb):
    P = Pool(kvb, 1, 2, 64, 32, 3, 150, share=3)
    P.lens = np.asarray([150, 150, 150])
    P.write([0, 96, 96, 96], [0, 0, 0], BF)           # the shared pages, once
    P.write(offsets([54, 54, 54]), [96, 96, 96], BF)  # each sequence's own
    q = torch.from_numpy(P.rng.standard_normal((1, 6, 3, 64))).to(BF).cuda()
    out, lse = attend(P, q, np.arange(4), [149, 120, 97])
    kvb.kvb_ctx_check(P.ctx)
    check_attention(P, q, np.arange(4), np.asarray([149, 120, 97]), out, lse)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [1, 40])
def test_page_scales_far_apart(kvb, dtype, n):
    # value blocks from 2^-90 to 2^90 and keys that decide which of them count: every
    # output is as exact relative to what it sums as with equal scales
    d, page, kv = 64, 16, 96
    P = Pool(kvb, 1, 1, d, page, 2, kv)
    P.lens = np.asarray([kv, kv])
    blocks = np.asarray([0, 90, -90, 5, 60, -60])
    x = P.rng.standard_normal((1, 1, kv, d))
    v = x * 2.0 ** np.repeat(blocks, page)[None, None, :, None]
    k = 0.02 * P.rng.standard_normal((1, 1, kv, d))
    k[0, 0, :, 0] += -4.0 * np.repeat(blocks, page) / 8  # large values get small weights, more or less
    two = lambda a: np.concatenate([a, a], axis=2)
    P.write([0, kv, 2 * kv], [0, 0], F32, x=[two(k), two(v)])
    q = P.rng.standard_normal((1, 4, 2 * n, d))
    q[..., 0] = np.linspace(-9, 9, 2 * n * 4).reshape(1, 4, 2 * n)
    q = torch.from_numpy(q).to(dtype).cuda()
    pos = np.asarray([kv - n, kv - n])
    out, lse = attend(P, q, [0, n, 2 * n], pos)
    kvb.kvb_ctx_check(P.ctx)
    o, z, A, B = P.ref.attention(to_host64(q), P.table, [0, n, 2 * n], pos)
    ds = (d / 16 + 4) * 2.0 ** -23 * B[..., None]
    # bf16: fp16 weights (2^-11) and the output's rounding; the scores' error covers both exponentials
    tol = A * (2 * (ds + 2.0 ** -21) + 40 * 2.0 ** -23 + (2.0 ** -11 if dtype == BF else 2.0 ** -21) + kv * 2.0 ** -31)
    tol = tol + np.abs(o) * (2.0 ** -8 if dtype == BF else 2.0 ** -23)
    assert (np.abs(to_host64(out) - o) <= tol).all()
    assert (np.abs(to_host64(lse) - z) <= ds[..., 0] + 2.0 ** -18 + 2.0 ** -22 * np.abs(z)).all()


def test_scores_that_rise_and_fall_over_the_tiles(kvb):
    # row maxima that rise by more than 2^8 several times, then stay below: references are raised, sums rescaled
    P = Pool(kvb, 1, 1, 128, 64, 2, 700)
    P.lens = np.asarray([700, 700])
    ramp = np.concatenate([np.linspace(0, 30, 500), np.linspace(30, -20, 200)])
    k = 0.3 * P.rng.standard_normal((1, 1, 1400, 128))
    k[0, 0, :, 0] += np.concatenate([ramp, ramp[::-1]])
    v = P.rng.standard_normal((1, 1, 1400, 128))
    P.write([0, 700, 1400], [0, 0], BF, x=[k, v])
    for dtype in (BF, F32):
        q = P.rng.standard_normal((1, 8, 2, 128))
        q[..., 0] = np.linspace(-20, 20, 16).reshape(1, 8, 2)
        q = torch.from_numpy(q).to(dtype).cuda()
        out, lse = attend(P, q, [0, 1, 2], [699, 640])
        check_attention(P, q, [0, 1, 2], np.asarray([699, 640]), out, lse)
    kvb.kvb_ctx_check(P.ctx)


def test_scale_layers_and_no_lse(kvb):
    P = Pool(kvb, 4, 2, 64, 32, 2, 60)
    P.fill([60, 33])
    q = torch.from_numpy(P.rng.standard_normal((2, 4, 2, 64))).to(BF).cuda()
    out, _ = attend(P, q, [0, 1, 2], [59, 32], lse=False, l_begin=2, scale=0.31)
    kvb.kvb_ctx_check(P.ctx)
    check_attention(P, q, [0, 1, 2], np.asarray([59, 32]), out, None, l_begin=2, scale=0.31)


def test_a_query_that_is_not_finite_stays_in_its_row(kvb):
    P = Pool(kvb, 1, 1, 128, 64, 1, 300)
    P.fill([300])
    q = torch.from_numpy(P.rng.standard_normal((1, 8, 2, 128))).to(BF).cuda()
    clean, zc = attend(P, q, [0, 2], [298])
    q2 = q.clone()
    q2[0, 3, 1, 7] = float("nan")
    out, z = attend(P, q2, [0, 2], [298])
    assert torch.isnan(out[0, 3, 1]).all() and torch.isnan(z[0, 3, 1])
    out[0, 3, 1], z[0, 3, 1] = clean[0, 3, 1], zc[0, 3, 1]
    assert torch.equal(out, clean) and torch.equal(z, zc)


def test_tiny_and_large_queries(kvb):
    P = Pool(kvb, 1, 1, 64, 16, 1, 40)
    P.fill([40])
    base = P.rng.standard_normal((1, 4, 1, 64))
    for f in (1e-30, 1e-3, 1e3):
        for dtype in (BF, F32):
            q = torch.from_numpy(base * f).to(dtype).cuda()
            out, lse = attend(P, q, [0, 1], [39])
            check_attention(P, q, [0, 1], np.asarray([39]), out, lse)


# ------------------------------------------------------------------ streams, capture, long offsets

def test_on_another_stream_and_captured_while_the_cache_grows(kvb):
    P = Pool(kvb, 1, 2, 128, 64, 2, 200)
    P.fill([100, 63])
    side = torch.cuda.Stream()
    off, pos = i32([0, 1, 2]), i32([100, 63])
    k, v = (torch.randn(1, 2, 2, 128, device="cuda").to(BF) for _ in range(2))
    q = torch.randn(1, 16, 2, 128, device="cuda").to(BF)
    out, lse = torch.empty_like(q), torch.empty(1, 16, 2, device="cuda")
    seqs = kvb.Seqs(P.dtab, off, pos, max_tokens=1, max_kv=200)

    def step():
        kvb.kvb_cache8_write(P.ctx, P.cache, seqs, k, v)
        kvb.kvb_cache8_attention(P.ctx, P.cache, seqs, q, out, lse)

    kvb.kvb_cache8_attention(P.ctx, P.cache, seqs, q, out, lse)  # sizes the workspace
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for i in range(5):
        with torch.cuda.stream(side):
            for t in (k, v, q):
                t.normal_()
            pos.copy_(i32([100 + i, 63 + i]))
            graph.replay()
        side.synchronize()
        for kv, x in enumerate((k, v)):
            P.ref.write(kv, to_host64(x), P.table, [0, 1, 2], [100 + i, 63 + i])
        P.lens = np.asarray([101 + i, 64 + i])
        check_attention(P, q, np.arange(3), P.lens - 1, out, lse)
    kvb.kvb_ctx_check(P.ctx)


def test_pages_beyond_four_gib(kvb):
    # a pool whose code offsets pass 2^32 bytes; the sequence lives at its far end
    n_pages, page, d, H = 70000, 64, 128, 8
    ctx = kvb.kvb_ctx_create(spec(1, H, d, 1e6), spec(1, H, d, 1e6), 1, 64)
    cache = kvb.kvb_cache8_create(ctx, n_pages, page)
    assert cache.k.numel() > 2 ** 32
    table = np.asarray([[n_pages - 1, 3, n_pages - 2]])
    seqs = lambda off, pos: kvb.Seqs(i32(table), i32(off), i32(pos), max_tokens=int(off[-1]))
    x = [torch.randn(1, H, 150, d, device="cuda").to(BF) for _ in range(2)]
    kvb.kvb_cache8_write(ctx, cache, seqs([0, 150], [0]), *x)
    back = [torch.empty_like(t) for t in x]
    kvb.kvb_cache8_read(ctx, cache, seqs([0, 150], [0]), *back)
    ref = C8.Cache8(1, 3, H, page, d)
    small = np.asarray([[2, 0, 1]])
    for kv in range(2):
        ref.write(kv, to_host64(x[kv]), small, [0, 150], [0])
        assert np.array_equal(to_host64(back[kv]), ref.read(kv, small, [0, 150], [0]))
    q = torch.randn(1, 2 * H, 1, d, device="cuda").to(BF)
    out, lse = torch.empty_like(q), torch.empty(1, 2 * H, 1, device="cuda")
    kvb.kvb_cache8_attention(ctx, cache, seqs([0, 1], [149]), q, out, lse)
    kvb.kvb_ctx_check(ctx)
    o, z, A, _ = ref.attention(to_host64(q), small, [0, 1], [149])
    assert (np.abs(to_host64(out) - o) <= 2.0 ** -8 * np.abs(o) + 2.0 ** -10 * A).all()


# ------------------------------------------------------------------ refusals

def status_of(kvb, f):
    with pytest.raises(kvb.KvbError) as e:
        f()
    return e.value.status


def test_kernels_report_sequences_and_pages_outside_the_call(kvb):
    P = Pool(kvb, 1, 1, 64, 16, 2, 64)
    P.fill([64, 64])
    q = torch.randn(1, 2, 4, 64, device="cuda").to(BF)
    good, _ = attend(P, q, [0, 2, 4], [62, 62])
    bits = lambda: (P.cache.k.view(torch.uint8).clone(), P.cache.k_scale.view(torch.int32).clone())
    before = bits()
    k = torch.randn(1, 1, 4, 64, device="cuda").to(BF)
    out, lse = torch.empty_like(q), torch.empty(1, 2, 4, device="cuda")
    rw = lambda s: (lambda: kvb.kvb_cache8_read(P.ctx, P.cache, s, k.clone(), k.clone()))
    at = lambda s: (lambda: kvb.kvb_cache8_attention(P.ctx, P.cache, s, q, out, lse))
    wr = lambda s: (lambda: kvb.kvb_cache8_write(P.ctx, P.cache, s, k, k))
    bad_page = P.dtab.clone()
    bad_page[1] = P.cache.n_pages
    neg_page = P.dtab.clone()
    neg_page[1] = -1
    cases = []
    for table in (bad_page, neg_page):
        s = kvb.Seqs(table, i32([0, 0, 4]), i32([0, 60]), max_tokens=4)
        cases += [rw(s), at(s), wr(s)]
    for off, pos in (([0, 5, 4], [0, 0]), ([0, 0, 9], [0, 0]), ([-1, 0, 0], [0, 0]), ([0, 0, 4], [0, 62]),
                     ([0, 0, 4], [0, 2 ** 31 - 2])):
        s = kvb.Seqs(P.dtab, i32(off), i32(pos), max_tokens=4)
        cases.append(at(s))
        if pos[1] < 2 ** 30 and pos != [0, 62]:
            cases += [rw(s), wr(s)]
    for f in cases:
        f()
        assert status_of(kvb, lambda: kvb.kvb_ctx_check(P.ctx)) == INVALID_ARG
        kvb.kvb_ctx_check(P.ctx)
    # a sequence whose pages are bad sees nothing; the other one is as before
    s = kvb.Seqs(bad_page, i32([0, 2, 4]), i32([62, 62]), max_tokens=2)
    kvb.kvb_cache8_attention(P.ctx, P.cache, s, q, out, lse)
    assert status_of(kvb, lambda: kvb.kvb_ctx_check(P.ctx)) == INVALID_ARG
    assert torch.equal(out[:, :, :2], good[:, :, :2]) and torch.all(out[:, :, 2:] == 0)
    # reading from bad pages gives zeros; writing to them writes nothing
    r = [torch.full((1, 1, 4, 64), 7.0, dtype=BF, device="cuda") for _ in range(2)]
    kvb.kvb_cache8_read(P.ctx, P.cache, kvb.Seqs(bad_page, i32([0, 0, 4]), i32([0, 60]), max_tokens=4), *r)
    assert status_of(kvb, lambda: kvb.kvb_ctx_check(P.ctx)) == INVALID_ARG
    assert torch.all(r[0] == 0) and torch.all(r[1] == 0)
    kvb.kvb_cache8_write(P.ctx, P.cache, kvb.Seqs(P.dtab, i32([0, 0, 4]), i32([0, -2]), max_tokens=4), k, k)
    assert status_of(kvb, lambda: kvb.kvb_ctx_check(P.ctx)) == INVALID_ARG
    assert all(torch.equal(a, b) for a, b in zip(bits(), before))


def test_the_next_call_reports_an_earlier_error(kvb):
    P = Pool(kvb, 1, 1, 64, 16, 1, 16)
    k = torch.full((1, 1, 1, 64), float("nan"), device="cuda")
    s = P.seqs([0, 1], [0])
    kvb.kvb_cache8_write(P.ctx, P.cache, s, k, k)
    torch.cuda.synchronize()
    assert status_of(kvb, lambda: kvb.kvb_cache8_write(P.ctx, P.cache, s, k, k)) == NUMERIC


def test_refusals(kvb):
    import ctypes
    P = Pool(kvb, 2, 2, 64, 16, 1, 32)
    lib = kvb.load_library()
    q = torch.zeros((2, 4, 1, 64), device="cuda")
    k = torch.zeros((2, 2, 1, 64), device="cuda")
    s = P.seqs([0, 1], [0])
    p = lambda t: ctypes.c_void_p(t.data_ptr())

    def att(cache=P.cache.ref, seqs=s.ref, l0=0, nl=2, dt=0, qp=p(q), hq=4, T=1, scale=0.0, out=p(q), lse=None):
        return lib.kvb_cache8_attention(P.ctx.handle, cache, seqs, l0, nl, dt, qp, hq, T, scale, out, lse, None)

    def struct(S, base, **kw):
        c = S.from_buffer_copy(base)
        for n, v in kw.items():
            setattr(c, n, v)
        return c

    B = __import__("cross_model_kv_gb300._binding", fromlist=["x"])
    cache = lambda **kw: struct(B.kvb_cache8, P.cache.struct, **kw)
    seqs = lambda **kw: struct(B.kvb_seqs, s.struct, **kw)
    ok = att()
    assert ok == 0
    keep = []

    def ref(c):
        keep.append(c)
        return ctypes.addressof(c)

    assert att(cache=None) == INVALID_ARG and att(seqs=None) == INVALID_ARG
    assert att(dt=2) == UNSUPPORTED and att(dt=-1) == UNSUPPORTED
    assert att(l0=1) == INVALID_ARG and att(l0=-1) == INVALID_ARG and att(nl=-1) == INVALID_ARG
    assert att(l0=2 ** 31 - 1, nl=2) == INVALID_ARG
    assert att(hq=3) == INVALID_ARG and att(hq=0) == INVALID_ARG
    assert att(T=-1) == INVALID_ARG and att(T=2 ** 31) == UNSUPPORTED and att(T=0) == INVALID_ARG  # max_tokens above T
    assert att(scale=-1.0) == INVALID_ARG and att(scale=float("nan")) == INVALID_ARG
    assert att(scale=float("inf")) == INVALID_ARG
    assert att(qp=None) == INVALID_ARG and att(out=None) == INVALID_ARG
    assert att(qp=ctypes.c_void_p(q.data_ptr() + 4)) == INVALID_ARG
    assert att(lse=ctypes.c_void_p(q.data_ptr() + 2)) == INVALID_ARG
    for kw in (dict(page_tokens=24), dict(page_tokens=0), dict(page_tokens=256)):
        assert att(cache=ref(cache(**kw))) == UNSUPPORTED
    for kw in (dict(k=None), dict(v=None), dict(k_scale=None), dict(v_scale=None), dict(n_pages=-1), dict(n_pages=2 ** 31),
               dict(k=P.cache.k.data_ptr() + 8)):
        assert att(cache=ref(cache(**kw))) == INVALID_ARG
    for kw in (dict(n_seq=-1), dict(max_pages=-1), dict(max_tokens=-1), dict(max_tokens=2), dict(max_kv=-1),
               dict(page_table=None), dict(seq_off=None), dict(seq_pos=None), dict(seq_pos=P.dtab.data_ptr() + 1)):
        assert att(seqs=ref(seqs(**kw))) == INVALID_ARG
    assert att(seqs=ref(seqs(max_pages=2 ** 31 - 1))) == UNSUPPORTED
    for f in (lib.kvb_cache8_write, lib.kvb_cache8_read):
        assert f(P.ctx.handle, P.cache.ref, s.ref, 0, 2, 0, None, p(k), 1, None) == INVALID_ARG
        assert f(P.ctx.handle, P.cache.ref, s.ref, 0, 3, 0, p(k), p(k), 1, None) == INVALID_ARG
        assert f(P.ctx.handle, P.cache.ref, ref(seqs(n_seq=2 ** 31 - 1)), 0, 2, 0, p(k), p(k), 1, None) == UNSUPPORTED
    assert att(seqs=ref(seqs(n_seq=2 ** 31 - 1))) == UNSUPPORTED  # sequences x layers x heads above 2^31-1
    bad_d = kvb.kvb_ctx_create(spec(1, 1, 96, 1e6), spec(1, 1, 96, 1e6), 1, 64)
    assert lib.kvb_cache8_write(bad_d.handle, P.cache.ref, s.ref, 0, 1, 0, p(k), p(k), 1, None) == UNSUPPORTED
    # the binding's own
    with pytest.raises(ValueError):
        kvb.kvb_cache8_attention(P.ctx, P.cache, s, q, q[:, :, :, :32].contiguous())
    with pytest.raises(ValueError):
        kvb.kvb_cache8_attention(P.ctx, P.cache, s, q, q.clone(), lse=torch.zeros(3, device="cuda"))
    with pytest.raises(ValueError):
        kvb.kvb_cache8_write(P.ctx, P.cache, s, k.transpose(0, 1), k.transpose(0, 1))
    with pytest.raises(ValueError):
        kvb.kvb_cache8_write(P.ctx, P.cache, s, k, k.to(BF))
    with pytest.raises(ValueError):
        kvb.kvb_cache8_write(P.ctx, P.cache, s, k.half(), k.half())
    with pytest.raises(ValueError):
        kvb.Cache8(P.ctx, P.cache.k, P.cache.v[:, :2], P.cache.k_scale, P.cache.v_scale)
    with pytest.raises(ValueError):
        kvb.Seqs(P.dtab, i32([0, 1]).long(), i32([0]), max_tokens=1)
    kvb.kvb_ctx_check(P.ctx)


# ------------------------------------------------------------------ many rows on the tensor cores

@pytest.mark.parametrize("page,H,g,n,lens", [(64, 1, 8, [100, 33, 0], [1500, 40, 10]), (16, 2, 4, [257, 64, 1], [900, 64, 300]),
                                             (128, 1, 16, [70, 20, 16], [700, 129, 16]), (32, 2, 1, [513, 128, 65], [513, 640, 65])])
def test_prompt_over_a_cached_prefix(kvb, page, H, g, n, lens):
    P = Pool(kvb, 1, H, 128, page, 3, max(lens), seed=page + g)
    P.fill(lens)
    q = torch.from_numpy(1.5 * P.rng.standard_normal((1, H * g, sum(n), 128))).to(BF).cuda()
    pos = np.asarray(lens) - n
    out, lse = attend(P, q, offsets(n), pos)
    kvb.kvb_ctx_check(P.ctx)
    check_attention(P, q, offsets(n), pos, out, lse)
    o2, z2 = attend(P, q, offsets(n), pos)
    assert torch.equal(out, o2) and torch.equal(lse, z2)


def test_prompt_with_rising_maxima_and_rows_that_see_nothing(kvb):
    P = Pool(kvb, 1, 1, 128, 32, 2, 1200)
    P.lens = np.asarray([1200, 1200])
    ramp = np.concatenate([np.linspace(0, 30, 800), np.linspace(30, -20, 400)])
    k = 0.3 * P.rng.standard_normal((1, 1, 2400, 128))
    k[0, 0, :, 0] += np.concatenate([ramp, ramp[::-1]])
    P.write([0, 1200, 2400], [0, 0], BF, x=[k, P.rng.standard_normal((1, 1, 2400, 128))])
    q = P.rng.standard_normal((1, 2, 160, 128))
    q[..., 0] = np.linspace(-20, 20, 320).reshape(1, 2, 160)
    q = torch.from_numpy(q).to(BF).cuda()
    for pos, kv_len in (([1100, 1120], None), ([-30, 0], None), ([1100, 900], [1000, 0])):
        out, lse = attend(P, q, [0, 80, 160], pos, kv_len=None if kv_len is None else i32(kv_len))
        kvb.kvb_ctx_check(P.ctx)
        check_attention(P, q, [0, 80, 160], np.asarray(pos), out, lse, kv_len=kv_len)


def test_prompt_with_page_scales_far_apart(kvb):
    # as test_page_scales_far_apart, on the tensor-core kernel: 160 rows of head_dim 128
    d, page, kv, n = 128, 16, 288, 80
    P = Pool(kvb, 1, 1, d, page, 1, kv)
    blocks = P.rng.permutation(np.repeat([0, 90, -90, 5, 60, -60, 1, -1, 3], 2))
    v = P.rng.standard_normal((1, 1, kv, d)) * 2.0 ** np.repeat(blocks, page)[None, None, :, None]
    k = 0.02 * P.rng.standard_normal((1, 1, kv, d))
    k[0, 0, :, 0] += -4.0 * np.repeat(blocks, page) / 8
    P.write([0, kv], [0], F32, x=[k, v])
    q = P.rng.standard_normal((1, 2, n, d))
    q[..., 0] = np.linspace(-12, 12, 2 * n).reshape(1, 2, n)
    q = torch.from_numpy(q).to(BF).cuda()
    out, lse = attend(P, q, [0, n], [kv - n])
    kvb.kvb_ctx_check(P.ctx)
    o, z, A, B = P.ref.attention(to_host64(q), P.table, [0, n], [kv - n])
    ds = (d / 16 + 4) * 2.0 ** -23 * B[..., None]
    tol = A * (2 * (ds + 2.0 ** -21) + 40 * 2.0 ** -23 + 2.0 ** -11 + kv * 2.0 ** -31) + np.abs(o) * 2.0 ** -8
    assert (np.abs(to_host64(out) - o) <= tol).all()
    assert (np.abs(to_host64(lse) - z) <= ds[..., 0] + 2.0 ** -18 + 2.0 ** -22 * np.abs(z)).all()


def test_prompt_over_bad_pages_reports_and_sees_the_others(kvb):
    P = Pool(kvb, 1, 2, 128, 64, 2, 500)
    P.fill([500, 500])
    q = torch.from_numpy(P.rng.standard_normal((1, 8, 60, 128))).to(BF).cuda()
    good, _ = attend(P, q, [0, 30, 60], [470, 470])
    kvb.kvb_ctx_check(P.ctx)
    bad = P.dtab.clone()
    bad[1, 2] = P.cache.n_pages + 5
    bad[1, 5] = -7
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    s = kvb.Seqs(bad, i32([0, 30, 60]), i32([470, 470]), max_tokens=30)
    kvb.kvb_cache8_attention(P.ctx, P.cache, s, q, out, lse)
    assert status_of(kvb, lambda: kvb.kvb_ctx_check(P.ctx)) == INVALID_ARG
    assert torch.equal(out[:, :, :30], good[:, :, :30])
    # the same pages as if their keys were not there: a sequence without those positions
    keep = [p for p in range(8) if p not in (2, 5)]
    few = i32(np.stack([P.table[1][keep]]))
    o2, z2 = torch.empty_like(q[:, :, 30:].contiguous()), torch.empty((1, 8, 30), device="cuda")
    s2 = kvb.Seqs(few, i32([0, 30]), i32([470 - 128]), max_tokens=30)
    kvb.kvb_cache8_attention(P.ctx, P.cache, s2, q[:, :, 30:].contiguous(), o2, z2)
    kvb.kvb_ctx_check(P.ctx)
    assert torch.allclose(out[:, :, 30:].float(), o2.float(), rtol=2.0 ** -7, atol=2.0 ** -9)
    assert torch.allclose(lse[:, :, 30:], z2, rtol=0, atol=2.0 ** -16)


@pytest.mark.parametrize("page,H,g,n,lens", [(64, 1, 8, [100, 33, 0], [1500, 40, 10]), (16, 2, 4, [257, 64, 1], [900, 64, 300]),
                                             (128, 1, 16, [70, 20, 16], [700, 129, 16]), (32, 2, 1, [513, 128, 65], [513, 640, 65])])
def test_prompt_of_head_dim_64(kvb, page, H, g, n, lens):
    P = Pool(kvb, 2, H, 64, page, 3, max(lens), seed=page + g + 1)
    P.fill(lens)
    q = torch.from_numpy(1.5 * P.rng.standard_normal((2, H * g, sum(n), 64))).to(BF).cuda()
    pos = np.asarray(lens) - n
    out, lse = attend(P, q, offsets(n), pos)
    kvb.kvb_ctx_check(P.ctx)
    check_attention(P, q, offsets(n), pos, out, lse)
    o2, z2 = attend(P, q, offsets(n), pos)
    assert torch.equal(out, o2) and torch.equal(lse, z2)
