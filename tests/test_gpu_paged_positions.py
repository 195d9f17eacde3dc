"""Positions outside the context's table, and sequences that begin before position 0, in both appends."""
import numpy as np
import pytest

from test_gpu_paged import BF, F32, INVALID_ARG, Pool, check_codes, kvb, status_of  # noqa: F401  (kvb: the fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("eight", [False, True])
def test_without_rotation_the_page_table_alone_bounds_positions(kvb, eight, dtype):  # noqa: F811
    # a table of 50 positions; rows at 40 .. 99 are stored as they are, and nothing is recorded
    P = Pool(kvb, 2, 2, 64, 16, 2, 100, dtype, max_pos=50, eight=eight)
    P.append([0, 40, 80], [0, 0], "token", rotate=False)
    P.append([0, 60, 61], [40, 40], "spaced", rotate=False)
    kvb.kvb_ctx_check(P.ctx)
    check_codes(P, [100, 41]) if eight else P.check_pages()


@pytest.mark.parametrize("rotate", [True, False])
@pytest.mark.parametrize("eight", [False, True])
def test_a_sequence_that_begins_before_position_0(kvb, eight, rotate):  # noqa: F811
    """Recorded.  Its tokens from position 0 on are stored in pages of the model's type; the 8-bit cache, whose blocks
    are rounded as a whole, takes none of them.  Queries at positions below 0 become 0."""
    P = Pool(kvb, 1, 2, 64, 16, 2, 64, BF, eight=eight)
    k, v = P.rows(1, 2, 4), P.rows(1, 2, 4)
    q = P.rows(1, 4, 4) if rotate else None
    out = torch.full_like(q, 7.0) if rotate else None
    raw = lambda: [t.view(torch.uint8).clone() for t in (P.cache.k, P.cache.v)]
    if eight:
        P.cache.k.view(torch.uint8).fill_(0x7f), P.cache.v.view(torch.uint8).fill_(0x7f)
    before = raw()
    call = kvb.kvb_cache8_append if eight else kvb.kvb_paged_append
    call(P.ctx, P.cache, P.seqs([0, 0, 4], [0, -2]), k, v, q, out, rotate=rotate)
    assert status_of(kvb, lambda: kvb.kvb_ctx_check(P.ctx)) == INVALID_ARG
    kvb.kvb_ctx_check(P.ctx)
    if rotate:
        want = torch.from_numpy(P.turned(q, [0, 0, 4], [0, -2])).to(BF)
        assert torch.equal(out.cpu(), want) and torch.all(out[:, :, :2] == 0) and torch.any(out[:, :, 2:] != 0)
    if eight:
        assert all(torch.equal(a, b) for a, b in zip(raw(), before))
        assert torch.all(P.cache.k_scale == 0) and torch.all(P.cache.v_scale == 0)
        return
    rk = torch.from_numpy(P.turned(k, [0, 0, 4], [0, -2])).to(BF) if rotate else k.cpu()
    for t, x in ((P.cache.k, rk), (P.cache.v, v.cpu())):
        page = t[:, P.table[1, 0]].cpu()
        assert torch.equal(page[:, :, :2], x[:, :, 2:])
        assert torch.isnan(page[:, :, 2:]).all()
