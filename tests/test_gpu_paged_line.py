"""Many sequences in the line of tiles: a CTA's place among up to 128 row blocks is found by every warp for itself,
four of them a lane, and among more by all of its threads."""
import numpy as np
import pytest

from test_gpu_paged import BF, F32, THETA, UNSUPPORTED, Pool, check_attention, i32, kvb, status_of  # noqa: F401  (kvb: the fixture)
from test_gpu_paged_long import widen

from cases import spec

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

COUNTS = (31, 32, 33, 64, 65, 96, 97, 127, 128, 129, 256, 257, 384, 385, 600)  # around the warps and threads that look


@pytest.mark.parametrize("dtype,d,g,n", [(BF, 128, 8, 1), (F32, 64, 4, 1), (BF, 64, 40, 1), (BF, 64, 64, 1), (BF, 64, 4, 3), (BF, 64, 20, 3)])
def test_many_sequences_find_their_places_in_the_line(kvb, dtype, d, g, n):  # noqa: F811
    """Lengths from 0 (a sequence that owns no token, one that sees no key) to 100, in the order of no kernel."""
    most = max(COUNTS)
    P = Pool(kvb, 1, 1, d, 16, most, 100, dtype)
    P.fill([100] * most)
    widen(P)
    lens = P.rng.integers(n, 100, most)
    tokens = np.where(np.arange(most) % 7 == 3, 0, P.rng.integers(1, n + 1, most))
    seen = np.where(np.arange(most) % 5 == 1, 0, lens)  # kv_len
    tcgen05 = dtype == BF and g * n > 16
    for m in COUNTS:
        off = np.concatenate([[0], np.cumsum(tokens[:m])])
        pos = lens[:m] - tokens[:m]
        q = P.rows(1, g, int(off[-1]))
        seqs = kvb.Seqs(P.dtab[:m].contiguous(), i32(off), i32(pos), max_tokens=n, kv_len=i32(seen[:m]))
        out, lse = torch.full_like(q, float("nan")), torch.full(q.shape[:3], float("nan"), device="cuda")
        if m == COUNTS[0]:  # neither clusters nor CTAs of their own take the call: those have no workspace that would grow
            fresh = kvb.kvb_ctx_create(spec(1, 1, d, 1e4), spec(1, 1, d, THETA), 1, 64)
            with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=torch.cuda.Stream()):
                assert status_of(kvb, lambda: kvb.kvb_paged_attention(fresh, P.cache, seqs, q, out, lse)) == UNSUPPORTED
                out.fill_(float("nan"))
            kvb.kvb_profile_enable(P.ctx)
        kvb.kvb_paged_attention(P.ctx, P.cache, seqs, q, out, lse)
        kvb.kvb_ctx_check(P.ctx)
        assert list(kvb.kvb_profile_read(P.ctx)) == ["paged_attention_tcgen05" if tcgen05 else "paged_attention"]
        check_attention(P, q, off, pos, out, lse, kv_len=seen[:m])
