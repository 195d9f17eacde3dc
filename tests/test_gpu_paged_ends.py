"""The ends of the paged attention on tcgen05 whose waits give up: a CTA leaves no load behind in shared memory that
the next kernel's CTAs take over, and waits only for what it asked for."""
import numpy as np
import pytest

from cases import spec

from test_gpu_paged import BF, THETA, Pool, attend, check_attention, kvb, offsets, status_of  # noqa: F401  (kvb: the fixture)
from test_gpu_paged_long import widen

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TIMEOUT = 7


@pytest.mark.parametrize("d,g,longest", [(64, 20, 500), (128, 40, 250), (128, 64, 250), (64, 32, 3000), (128, 20, 3000)])
def test_a_call_that_gives_up_leaves_no_load_behind(kvb, d, g, longest, monkeypatch):  # noqa: F811
    """Up to 500 or 250 keys a CTA's tiles all fit its rings, so that no wait of its loads is there to give up.

    What a load that is still in flight would overwrite is the shared memory of the call that follows, on as many
    CTAs.  A wait for a barrier that no load was asked for would run for 12.5 ms at least."""
    n = 76
    P = Pool(kvb, 1, 2, d, 16, n, longest, BF)
    widen(P)
    lens = P.rng.integers(longest // 2, longest, n)
    P.fill(lens)
    off, pos = offsets([1] * n), lens - 1
    q, one = P.rows(1, 2 * g, n), P.rows(1, 4, n)
    good, z = attend(P, q, off, pos)
    alone, _ = attend(P, one, off, pos)
    check_attention(P, q, off, pos, good, z)
    monkeypatch.setenv("KVB_WAIT_TIMEOUT_MS", "0")
    ctx0 = kvb.kvb_ctx_create(spec(1, 2, d, 1e4), spec(1, 2, d, THETA), 1, 64)
    monkeypatch.delenv("KVB_WAIT_TIMEOUT_MS")
    kvb.kvb_profile_enable(ctx0)
    seqs, out, rest = P.seqs(off, pos), torch.empty_like(q), torch.empty_like(one)
    times = []
    for _ in range(40):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        kvb.kvb_paged_attention(ctx0, P.cache, seqs, q, out)
        b.record()
        kvb.kvb_paged_attention(P.ctx, P.cache, seqs, one, rest)
        assert status_of(kvb, lambda: kvb.kvb_ctx_check(ctx0)) == TIMEOUT
        assert torch.equal(rest, alone)
        times.append(a.elapsed_time(b))
    assert list(kvb.kvb_profile_read(ctx0)) == ["paged_attention_tcgen05"]
    assert min(times) < 12.5, times
    kvb.kvb_ctx_check(P.ctx)
    out, lse = attend(P, q, off, pos)
    kvb.kvb_ctx_check(P.ctx)
    assert torch.equal(out, good) and torch.equal(lse, z)
