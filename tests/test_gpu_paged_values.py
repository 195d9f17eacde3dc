"""Attention over large values and of broadcast rows; appends of broadcast rows."""
import numpy as np
import pytest

from cases import to_host64

from test_gpu_paged import BF, F32, Pool, attend, check_attention, check_codes, kvb, offsets  # noqa: F401  (kvb: the fixture)
from test_gpu_paged_long import widen

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("dtype,d,g", [(BF, 128, 8), (BF, 64, 40), (F32, 64, 4)])
def test_values_that_sums_can_hold(kvb, dtype, d, g, wide):  # noqa: F811
    # weights are at most 2^8 before the division: 2^8 times 3000 keys times 6 sigma of 2^105 is below 2^128
    P = Pool(kvb, 1, 2, d, 32, 3, 3000, dtype)
    lens = np.array([3000, 77, 1])
    P.lens = lens
    k, v = P.rows(1, 2, int(lens.sum())), P.rows(1, 2, int(lens.sum()), sigma=2.0 ** 105)
    off = offsets(lens)
    kvb.kvb_paged_append(P.ctx, P.cache, P.seqs(off, [0, 0, 0]), k, v, rotate=False)
    for kv, x in enumerate((k, v)):
        P.ref.append(kv, to_host64(x), P.table, off, [0, 0, 0])
    if wide:
        widen(P)
    q = P.rows(1, 2 * g, 3)
    out, lse = attend(P, q, offsets([1] * 3), lens - 1)
    kvb.kvb_ctx_check(P.ctx)
    check_attention(P, q, offsets([1] * 3), lens - 1, out, lse)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_broadcast_rows(kvb, dtype):  # noqa: F811
    """Inputs with strides of 0: one head's rows for every head, one layer's for every layer, one token's for all."""
    P = Pool(kvb, 3, 2, 64, 16, 1, 40, dtype)
    E = Pool(kvb, 3, 2, 64, 16, 1, 40, dtype, eight=True)
    for axis in range(3):
        def rows(heads):
            own = [1 if i == axis else n for i, n in enumerate((3, heads, 40))]
            return P.rows(*own).expand(3, heads, 40, 64)

        k, v, q = rows(2), rows(2), rows(8)
        assert 0 in k.stride() and 0 in q.stride()
        off, pos = [0, 40], [0]
        rk = P.turned(k, off, pos)
        for pool, call in ((P, kvb.kvb_paged_append), (E, kvb.kvb_cache8_append)):
            out = torch.full(q.shape, 7.0, dtype=dtype, device="cuda")
            call(pool.ctx, pool.cache, pool.seqs(off, pos), k, v, q, out)
            kvb.kvb_ctx_check(pool.ctx)
            assert torch.equal(out.cpu(), torch.from_numpy(P.turned(q, off, pos)).to(dtype))
        P.ref.append(0, torch.from_numpy(rk).to(dtype).double().numpy(), P.table, off, pos)
        P.ref.append(1, to_host64(v), P.table, off, pos)
        E.ref.write(0, rk.astype(np.float64), E.table, off, pos)
        E.ref.write(1, to_host64(v), E.table, off, pos)
        P.check_pages()
        check_codes(E, [40])
        a, b = (torch.empty(q.shape, dtype=dtype, device="cuda") for _ in range(2))
        kvb.kvb_paged_attention(P.ctx, P.cache, P.seqs(off, pos), q, a)
        kvb.kvb_paged_attention(P.ctx, P.cache, P.seqs(off, pos), q.contiguous(), b)
        kvb.kvb_ctx_check(P.ctx)
        assert torch.equal(a, b)
