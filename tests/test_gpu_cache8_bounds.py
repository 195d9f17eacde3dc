"""The 8-bit cache at the edges of what its calls accept: how the buffers are aligned."""
import numpy as np
import pytest

from test_gpu_cache8 import BF, F32, Pool, attend, i32, kvb, offsets  # noqa: F401  (kvb: the fixture)

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
