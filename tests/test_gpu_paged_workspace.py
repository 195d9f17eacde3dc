"""Captured attention calls whose workspace later calls outgrow: both its parts, the counters and the partial results,
for the line of tiles and for tcgen05."""
import numpy as np
import pytest

from test_gpu_paged import BF, UNSUPPORTED, Pool, check_attention, i32, kvb, status_of  # noqa: F401  (kvb: the fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

KEYS = 70000  # that a sequence may have: enough for the line, and for tcgen05


def refused_while_captured(kvb, call, out):  # noqa: F811
    """Whether the workspace would have to grow for the call: a captured stream refuses that."""
    with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=torch.cuda.Stream()):
        try:
            call()
            grows = False
        except kvb.KvbError as e:
            assert e.status == UNSUPPORTED
            grows = True
        out.zero_()
    return grows


def test_captured_calls_of_both_kernels_outlive_what_they_were_captured_with(kvb):  # noqa: F811
    P = Pool(kvb, 1, 2, 128, 64, 2, KEYS, BF)
    P.fill([KEYS, 3000])
    side, kinds = torch.cuda.Stream(), []

    def make(g, lens):
        q = P.rows(1, 2 * g, len(lens))
        out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
        table = P.dtab[:2] if len(lens) == 2 else P.dtab[:1].repeat(len(lens), 1)
        seqs = kvb.Seqs(table, i32(np.arange(len(lens) + 1)), i32(np.asarray(lens) - 1), max_tokens=1, max_kv=KEYS)
        return q, out, lse, lambda: kvb.kvb_paged_attention(P.ctx, P.cache, seqs, q, out, lse), seqs

    def replayed():
        for _ in range(2):
            for graph, out, lse, want, *_ in kinds:
                out.zero_(), lse.zero_()
                torch.cuda.synchronize()
                graph.replay()
                torch.cuda.synchronize()
                assert torch.equal(out, want[0]) and torch.equal(lse, want[1])

    # 8 rows: the line; 40: tcgen05 in blocks of 48
    for g, lens in ((8, [KEYS, 3000]), (40, [3000, 2000])):
        q, out, lse, call, seqs = make(g, lens)
        call()
        check_attention(P, q, [0, 1, 2], np.asarray(lens) - 1, out, lse)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call()
        kinds.append((graph, out, lse, (out.clone(), lse.clone()), q, seqs))
        assert not refused_while_captured(kvb, call, out)
    replayed()
    # 64 rows on as many CTAs: partial results a third larger, and a quarter more was allocated; then units for more
    # than the 16384 counters that there are at first
    for g, n in ((64, 4), (4, 8400)):
        q, out, lse, call, seqs = make(g, [1000] * n)
        assert refused_while_captured(kvb, call, out)
        call()
        kvb.kvb_ctx_check(P.ctx)
        few = [0, n // 2, n - 1]
        own, P.table = P.table, np.repeat(P.table[:1], 3, axis=0)
        check_attention(P, q[:, :, few], np.arange(4), [999] * 3, out[:, :, few], lse[:, :, few])
        P.table = own
        assert torch.isfinite(out).all() and torch.isfinite(lse).all()
        replayed()
        assert not refused_while_captured(kvb, call, out)
    kvb.kvb_ctx_check(P.ctx)
