"""Sequences of an 8-bit attention call around the number, 32, up to which every warp finds a CTA's place in the line
by itself, and around the threads that look for it among more."""
import numpy as np
import pytest

from test_gpu_cache8 import BF, F32, Pool, attend, check_attention, kvb  # noqa: F401  (kvb: the fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

COUNTS = (31, 32, 33, 64, 96, 127, 128, 129, 257)


@pytest.mark.parametrize("dtype,d,g,n,kernel", [(BF, 128, 8, 1, "cache8_attention"), (F32, 64, 4, 2, "cache8_attention"),
                                                (BF, 128, 8, 40, "cache8_attention_tcgen05"), (BF, 64, 4, 80, "cache8_attention_tcgen05")])
def test_sequences_around_what_a_warp_places(kvb, dtype, d, g, n, kernel):  # noqa: F811
    most = max(COUNTS) if n < 3 else 65
    P = Pool(kvb, 1, 1, d, 16, most, 120, seed=d + n)
    P.fill([120] * most, dtype)
    lens = P.rng.integers(n, 120, most)
    tokens = np.where(np.arange(most) % 7 == 3, 0, P.rng.integers(1, n + 1, most))
    kvb.kvb_profile_enable(P.ctx)
    kvb.kvb_profile_read(P.ctx)
    for m in (c for c in COUNTS if c <= most):
        off, pos = np.concatenate([[0], np.cumsum(tokens[:m])]), lens[:m] - tokens[:m]
        q = torch.from_numpy(P.rng.standard_normal((1, g, int(off[-1]), d))).to(dtype).cuda()
        whole = P.table, P.dtab, P.lens
        P.table, P.dtab, P.lens = P.table[:m], P.dtab[:m].contiguous(), P.lens[:m]
        out, lse = attend(P, q, off, pos, max_tokens=n)
        kvb.kvb_ctx_check(P.ctx)
        assert list(kvb.kvb_profile_read(P.ctx)) == [kernel]
        check_attention(P, q, off, pos, out, lse)
        P.table, P.dtab, P.lens = whole
