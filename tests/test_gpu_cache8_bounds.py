"""The 8-bit cache at the edges of what its calls accept: how the buffers are
aligned, positions up to the last that a call may name, caches of other sizes."""
import numpy as np
import pytest

from cases import spec, to_host64
from oracle import cache8 as C8
from test_gpu_cache8 import BF, F32, Pool, i32, kvb, offsets  # noqa: F401  (kvb: the fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def moved(t, at):
    """t's bytes in a buffer that starts `at` bytes past a 32-byte boundary."""
    pool = torch.empty(t.numel() + 64, dtype=torch.uint8, device="cuda")
    first = -pool.data_ptr() % 32 + at
    view = pool[first:first + t.numel()].view(t.shape)
    view.copy_(t.view(torch.uint8))
    assert view.data_ptr() % 32 == at
    return view


# ------------------------------------------------------------------ alignment

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [16, 32, 64, 128])
@pytest.mark.parametrize("g,n", [(8, 1), (8, 2), (5, 9)])
def test_codes_aligned_to_16_bytes(kvb, d, g, n, dtype):  # noqa: F811
    # buffers that start 16 bytes past a 32-byte boundary hold the same codes: every result is
    # the same bit for bit (a few rows over few and over many keys, rows of the prompt kernel)
    P = Pool(kvb, 1, 2, d, 16, 3, 700, seed=d + g)
    P.fill([700, 33, 258])
    near = P.cache
    far = kvb.Cache8(P.ctx, moved(near.k, 16), moved(near.v, 16), near.k_scale.clone(), near.v_scale.clone())
    for reps in (1, 40):  # 40 times the three sequences: more keys than the few-key form takes
        table = i32(np.tile(P.table, (reps, 1)))
        lens = np.tile([700, 33, 258], reps)
        q = torch.from_numpy(P.rng.standard_normal((1, 2 * g, n * len(lens), d))).to(dtype).cuda()
        seqs = kvb.Seqs(table, i32(offsets([n] * len(lens))), i32(lens - n), max_tokens=n)
        got = []
        for cache in (near, far):
            out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
            kvb.kvb_cache8_attention(P.ctx, cache, seqs, q, out, lse)
            got.append((out, lse))
        kvb.kvb_ctx_check(P.ctx)
        assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
        assert torch.isfinite(got[0][0]).all()
    # tokens written there and read back
    x = [torch.randn(1, 2, 20, d, device="cuda").to(dtype) for _ in range(2)]
    at = P.seqs([0, 0, 20, 20], [0, 33, 0])
    back = []
    for cache in (near, far):
        kvb.kvb_cache8_write(P.ctx, cache, at, *x)
        y = [torch.empty_like(t) for t in x]
        kvb.kvb_cache8_read(P.ctx, cache, at, *y)
        back.append(y)
    kvb.kvb_ctx_check(P.ctx)
    assert all(torch.equal(a, b) for a, b in zip(*back))
    assert torch.equal(near.k.view(torch.uint8), far.k) and torch.equal(near.v.view(torch.uint8), far.v)


# ------------------------------------------------------------------ positions up to 2^31

@pytest.mark.parametrize("d,g,dtype", [(16, 1, BF), (64, 2, F32), (128, 8, BF), (64, 50, BF)])
def test_the_last_positions_that_a_call_may_name(kvb, d, g, dtype):  # noqa: F811
    # 2^31 - 1024 positions, the most that is accepted, on three pages that repeat: a list of
    # pages that is asked for from near the end would pass 2^31.  Every key counts as often as its page comes.
    # Tolerance: each CTA adds the keys of its share one after another in fp32, 16 (bf16 prompt
    # kernel, 152 CTAs) or 32 (152 CTAs at least, 4 warps) at a time: steps of 2^-23 each, in
    # numerator and denominator; then the formats' 2^-11 for weights and 2^-8 for the output.
    page, kv = 128, 0x7ffffc00
    P = Pool(kvb, 1, 1, d, page, 1, 3 * page, spare=0)
    P.fill([3 * page])
    table = i32(P.table[0])[torch.arange(kv // page, device="cuda") % 3][None].contiguous()
    q = torch.from_numpy(4.0 * P.rng.standard_normal((1, g, 1, d))).to(dtype).cuda()  # few keys decide
    out, lse = torch.empty_like(q), torch.empty((1, g, 1), device="cuda")
    seqs = kvb.Seqs(table, i32([0, 1]), i32([kv - 1]), max_tokens=1)
    kvb.kvb_cache8_attention(P.ctx, P.cache, seqs, q, out, lse)
    kvb.kvb_ctx_check(P.ctx)
    k, v = (P.ref.sequence(x, P.table[0], 3 * page, 0, 0) for x in (0, 1))
    times = np.repeat([kv // page - 2 * (kv // page // 3) - (kv // page % 3 > 1), 0, kv // page // 3], page)
    times[page:2 * page] = kv // page - times[0] - times[-1]
    s = to_host64(q)[0, :, 0] @ k.T / np.sqrt(d)
    w = np.exp(s - s.max(axis=1, keepdims=True)) * times
    z = s.max(axis=1) + np.log(w.sum(axis=1))
    w /= w.sum(axis=1, keepdims=True)
    steps = kv / 152 / 16
    tol = (w @ np.abs(v)) * (2 * steps * 2.0 ** -23 + 2.0 ** -10) + np.abs(w @ v) * 2.0 ** -8
    assert (np.abs(to_host64(out)[0, :, 0] - w @ v) <= tol).all()
    assert (np.abs(to_host64(lse)[0, :, 0] - z) <= steps * 2.0 ** -23 + 2.0 ** -10).all()


def test_more_positions_are_refused(kvb):  # noqa: F811
    P = Pool(kvb, 1, 1, 64, 128, 1, 128)
    P.fill([5])
    q = torch.zeros((1, 1, 1, 64), device="cuda")
    lib = kvb.load_library()

    def status(call, max_pages, max_kv):  # the sequence itself stays at its five positions
        s = P.seqs([0, 1], [4])
        s.struct.max_pages, s.struct.max_kv = max_pages, max_kv
        if call == "attention":
            return lib.kvb_cache8_attention(P.ctx.handle, P.cache.ref, s.ref, 0, 1, 0, q.data_ptr(), 1, 1, 0.0, q.data_ptr(),
                                            None, None)
        return getattr(lib, "kvb_cache8_" + call)(P.ctx.handle, P.cache.ref, s.ref, 0, 1, 0, q.data_ptr(), q.data_ptr(), 1, None)

    most = 0x7ffffc00 // 128
    for call in ("write", "read", "attention"):
        assert status(call, most, 0) == 0 and status(call, most + 1, 0x7ffffc00) == 0
        for max_kv in (0, 0x7ffffc01, 0x7fffffff):
            assert status(call, most + 1, max_kv) == 3
    kvb.kvb_ctx_check(P.ctx)


# ------------------------------------------------------------------ one cache, several contexts

def test_a_cache_of_another_context_s_sizes_is_refused(kvb):  # noqa: F811
    # the library sees bare pointers: only the binding can tell that a cache has other sizes than
    # the context that a call is made with
    def tensors(L, H, d):
        k = torch.zeros((L, H, 1, d), dtype=BF, device="cuda")
        return k, torch.zeros_like(k)

    def calls(ctx, cache, L, H, d):
        k, v = tensors(L, H, d)
        s = kvb.Seqs(i32([[0]]), i32([0, 1]), i32([0]), max_tokens=1)
        return (lambda: kvb.kvb_cache8_write(ctx, cache, s, k, v), lambda: kvb.kvb_cache8_read(ctx, cache, s, k, v),
                lambda: kvb.kvb_cache8_attention(ctx, cache, s, k, v))

    make = lambda L, H, d: kvb.kvb_ctx_create(spec(1, H, d, 1e6), spec(L, H, d, 1e6), 1, 64)
    cache = kvb.kvb_cache8_create(make(2, 2, 64), 1, 16)
    for L, H, d in ((3, 2, 64), (1, 2, 64), (2, 4, 64), (2, 1, 64), (2, 2, 128), (2, 2, 32)):
        for f in calls(make(L, H, d), cache, L, H, d):
            with pytest.raises(ValueError, match="another context"):
                f()
    twin = make(2, 2, 64)  # of the same sizes: as good as its own
    for f in calls(twin, cache, 2, 2, 64):
        f()
    kvb.kvb_ctx_check(twin)


# ------------------------------------------------------------------ no time to wait

@pytest.mark.parametrize("d", [64, 128])
def test_a_limit_of_no_time_runs_out_every_time(kvb, d, monkeypatch):  # noqa: F811
    # the prompt kernel over one key and over many, again and again: never a matter of which warp is first
    P = Pool(kvb, 1, 1, d, 16, 1, 2000)
    P.fill([2000])
    q = torch.randn(1, 60, 1, d, device="cuda").to(BF)
    out = torch.empty_like(q)
    monkeypatch.setenv("KVB_WAIT_TIMEOUT_MS", "0")
    ctx0 = kvb.kvb_ctx_create(spec(1, 1, d, 1e6), spec(1, 1, d, 1e6), 1, 64)
    monkeypatch.delenv("KVB_WAIT_TIMEOUT_MS")
    for pos in [0, 1999] * 25:
        kvb.kvb_cache8_attention(ctx0, P.cache, P.seqs([0, 1], [pos]), q, out)
        with pytest.raises(kvb.KvbError) as e:
            kvb.kvb_ctx_check(ctx0)
        assert e.value.status == 7
    kvb.kvb_cache8_attention(P.ctx, P.cache, P.seqs([0, 1], [0]), q, out)
    kvb.kvb_ctx_check(P.ctx)
    v = torch.from_numpy(P.ref.sequence(1, P.table[0], 1, 0, 0)).to(BF).cuda()  # one key: its value
    assert torch.equal(out[0, :, 0], v.expand(60, d))


# ------------------------------------------------------------------ products past the range of fp32

@pytest.mark.parametrize("d,n,dtype", [(64, 1, BF), (128, 1, F32), (128, 9, BF), (64, 60, BF), (128, 60, BF)])
def test_scores_of_zero_between_values_past_the_range_of_fp32(kvb, d, n, dtype):  # noqa: F811
    # queries of 2^100 in the first dims, keys of 2^70 in the others: every product is 0, although
    # the query's and the keys' scales together pass fp32.  The output is the mean of the values.
    P = Pool(kvb, 1, 1, d, 16, 1, 200)
    P.lens = np.asarray([200])
    k = 2.0 ** 70 * P.rng.standard_normal((1, 1, 200, d))
    k[..., :8] = 0
    P.write([0, 200], [0], BF, x=[k, P.rng.standard_normal((1, 1, 200, d))])
    q = np.zeros((1, 1, n, d))
    q[..., :8] = 2.0 ** 100 * P.rng.standard_normal((1, 1, n, 8))
    q = torch.from_numpy(q).to(dtype).cuda()
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    kvb.kvb_cache8_attention(P.ctx, P.cache, P.seqs([0, n], [200 - n]), q, out, lse)
    kvb.kvb_ctx_check(P.ctx)
    v = P.ref.sequence(1, P.table[0], 200, 0, 0)
    for i in range(n):
        see = v[:200 - n + i + 1]
        tol = 2.0 ** -8 * np.abs(see.mean(axis=0)) + 2.0 ** -10 * np.abs(see).mean(axis=0)
        assert (np.abs(to_host64(out)[0, 0, i] - see.mean(axis=0)) <= tol).all()
        assert abs(float(lse[0, 0, i]) - np.log(len(see))) <= 2.0 ** -16


# ------------------------------------------------------------------ a page begun in its middle

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,page,pos,n", [(64, 32, 13, 5), (128, 64, 63, 1), (128, 16, 7, 40), (16, 128, 100, 20)])
def test_a_sequence_that_begins_inside_a_page(kvb, d, page, pos, n, dtype):  # noqa: F811
    # a new cache holds no older scale: its first tokens decide, wherever in the page they lie, although
    # the memory that it gets was another's
    ctx = kvb.kvb_ctx_create(spec(1, 2, d, 1e6), spec(1, 2, d, 1e6), 1, 64)
    old = kvb.kvb_cache8_create(ctx, 4, page)
    for t in (old.k_scale, old.v_scale):
        t.fill_(float("nan"))
    del old, t
    cache = kvb.kvb_cache8_create(ctx, 4, page)
    ref = C8.Cache8(1, 4, 2, page, d)
    for t in ref.scales:
        t[:] = 2.0 ** -117
    table = [[2, 0, 3, 1]]
    s = kvb.Seqs(i32(table), i32([0, n]), i32([pos]), max_tokens=n)
    x = [torch.randn(1, 2, n, d, device="cuda").to(dtype) for _ in range(2)]
    kvb.kvb_cache8_write(ctx, cache, s, *x)
    y = [torch.empty_like(t) for t in x]
    kvb.kvb_cache8_read(ctx, cache, s, *y)
    kvb.kvb_ctx_check(ctx)
    for kv in range(2):
        ref.write(kv, to_host64(x[kv]), table, [0, n], [pos])
        assert np.array_equal(to_host64(y[kv]), ref.read(kv, table, [0, n], [pos]))
