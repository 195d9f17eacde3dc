"""Pages whose offsets pass 2^32, in every kernel that reads or writes them."""
import numpy as np
import pytest

from cases import spec, to_host64
from oracle import cache8 as C8
from oracle import paged as PG

from test_gpu_paged import BF, THETA, UNSUPPORTED, i32, kvb, offsets, status_of  # noqa: F401  (kvb: the fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

PAGES, PAGE, D, H = 70000, 64, 128, 8  # 4.59e9 elements
LEN = 150
NEAR = np.array([[2, 0, 1]])  # the oracle's pages: 0 is page 3 of the pool, 1 and 2 the last but one and the last
FAR = [PAGES - 1, 3, PAGES - 2]


def table(cols=3):
    return torch.nn.functional.pad(i32([FAR]), (0, cols - 3), value=-1)


@pytest.fixture(scope="module")
def pool(kvb):  # noqa: F811
    torch.cuda.empty_cache()
    ctx = kvb.kvb_ctx_create(spec(1, H, D, 1e6), spec(1, H, D, THETA), 1, 256)
    cache = kvb.kvb_paged_create(ctx, PAGES, PAGE)
    assert cache.k.numel() > 2 ** 32
    torch.manual_seed(1)
    k, v = (torch.randn(1, H, LEN, D, device="cuda").to(BF) for _ in range(2))
    kvb.kvb_paged_append(ctx, cache, kvb.Seqs(table(), i32([0, LEN]), i32([0]), max_tokens=LEN), k, v, rotate=False)
    ref = PG.Paged(1, 3, H, PAGE, D)
    for kv, x in enumerate((k, v)):
        ref.append(kv, to_host64(x), NEAR, [0, LEN], [0])
    yield ctx, cache, ref
    torch.cuda.empty_cache()


# query heads of a KV head, tokens; what takes the call, by rows and by the keys that the page table has room for
@pytest.mark.parametrize("g,n,cols,kernel", [(2, 1, 3, "paged_attention"), (8, 1, 4096, "paged_attention"), (2, 4, 4096, "paged_attention"),
                                             (4, 5, 4096, "paged_attention_tcgen05"), (8, 5, 4096, "paged_attention_tcgen05"),
                                             (8, 8, 4096, "paged_attention_tcgen05")])
def test_attention_over_pages_beyond_four_gib(kvb, pool, g, n, cols, kernel):  # noqa: F811
    """In clusters, in the line and on tcgen05; then with a last value that is infinite, which is read again at its page."""
    ctx, cache, ref = pool
    q = torch.randn(1, H * g, n, D, device="cuda").to(BF)
    seqs = kvb.Seqs(table(cols), i32([0, n]), i32([LEN - n]), max_tokens=n)
    out, lse = torch.empty_like(q), torch.empty(1, H * g, n, device="cuda")
    if cols > 3:  # the line, or tcgen05: a workspace
        fresh = kvb.kvb_ctx_create(spec(1, H, D, 1e6), spec(1, H, D, THETA), 1, 256)
        with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=torch.cuda.Stream()):
            assert status_of(kvb, lambda: kvb.kvb_paged_attention(fresh, cache, seqs, q, out, lse)) == UNSUPPORTED
            out.zero_()
    kvb.kvb_profile_enable(ctx)
    kvb.kvb_profile_read(ctx)
    kvb.kvb_paged_attention(ctx, cache, seqs, q, out, lse)
    kvb.kvb_ctx_check(ctx)
    assert list(kvb.kvb_profile_read(ctx)) == [kernel]
    o, z, A, _ = ref.attention(to_host64(q), NEAR, [0, n], [LEN - n])
    # the output's rounding; 2^-12 of the spread is far above what products and weights lose over 150 keys
    assert (np.abs(to_host64(out) - o) <= 2.0 ** -8 * np.abs(o) + 2.0 ** -12 * A).all()
    assert np.abs(to_host64(lse) - z).max() <= 2.0 ** -12
    if n == 1:
        return
    page, slot = FAR[(LEN - 1) // PAGE], (LEN - 1) % PAGE
    was = cache.v[0, page, :, slot, 5].clone()
    cache.v[0, page, :, slot, 5] = float("inf")
    again = torch.empty_like(q)
    kvb.kvb_paged_attention(ctx, cache, seqs, q, again)
    cache.v[0, page, :, slot, 5] = was
    kvb.kvb_ctx_check(ctx)
    # only the last token sees it: infinite or NaN there
    assert torch.equal(again[:, :, :-1], out[:, :, :-1])
    assert not torch.isfinite(again[:, :, -1, 5]).any()
    rest = torch.arange(D, device="cuda") != 5
    assert torch.equal(again[:, :, -1, rest], out[:, :, -1, rest])


def test_append8_beyond_four_gib(kvb):  # noqa: F811
    """Codes and scales at the far end, written in two calls that share a block; what lies next to them stays."""
    torch.cuda.empty_cache()
    ctx = kvb.kvb_ctx_create(spec(1, H, D, 1e6), spec(1, H, D, THETA), 1, 256)
    cache = kvb.kvb_cache8_create(ctx, PAGES, PAGE)
    assert cache.k.numel() > 2 ** 32
    for t in (cache.k, cache.v):
        t.view(torch.uint8)[0, [0, 2, 4, PAGES - 3]] = 0x55
    ref = C8.Cache8(1, 3, H, PAGE, D)
    cos, sin = PG.table(THETA, D, 256)
    for at, n, sigma in ((0, 100, 1.0), (100, LEN - 100, 9.0)):
        k, v, q = (sigma * torch.randn(1, h, n, D, device="cuda") for h in (H, H, 2 * H))
        turned = torch.empty_like(q)
        kvb.kvb_cache8_append(ctx, cache, kvb.Seqs(table(), i32([0, n]), i32([at]), max_tokens=n), k, v, q, turned)
        pos = at + np.arange(n)
        assert np.array_equal(turned.cpu().numpy(), PG.rotate32(q.cpu().numpy(), pos, cos, sin))
        ref.write(0, PG.rotate32(k.cpu().numpy(), pos, cos, sin).astype(np.float64), NEAR, [0, n], [at])
        ref.write(1, to_host64(v), NEAR, [0, n], [at])
    kvb.kvb_ctx_check(ctx)
    for kv, (codes, scales) in enumerate(((cache.k, cache.k_scale), (cache.v, cache.v_scale))):
        for p, (far, near) in enumerate(zip(FAR, NEAR[0])):
            m = min(PAGE, LEN - p * PAGE)
            assert np.array_equal(scales[0, far].cpu().numpy(), ref.scales[kv][0, near])
            assert np.array_equal(codes.view(torch.uint8)[0, far, :, :m].cpu().numpy(), ref.codes[kv][0, near, :, :m])
        for far in (0, 2, 4, PAGES - 3):
            assert torch.all(codes.view(torch.uint8)[0, far] == 0x55) and torch.all(scales[0, far] == 0)
    # and read back by the 8-bit cache's own call, whose numbers are exact
    back = [torch.empty(1, H, LEN, D, device="cuda") for _ in range(2)]
    kvb.kvb_cache8_read(ctx, cache, kvb.Seqs(table(), i32([0, LEN]), i32([0]), max_tokens=LEN), *back)
    kvb.kvb_ctx_check(ctx)
    for kv, x in enumerate(back):
        assert np.array_equal(to_host64(x), ref.read(kv, NEAR, [0, LEN], [0]))
