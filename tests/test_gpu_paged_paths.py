"""The paged cache's attention where it can be left halfway: waits that run out, workspaces that
are outgrown while graphs hold them; and all its tests on the checked build, whose kernels look at
every index before they use it."""
import os
import subprocess
import sys

import numpy as np
import pytest

from cases import spec

from test_gpu_paged import BF, F32, THETA, Pool, attend, check_attention, i32, kvb, offsets, status_of  # noqa: F401  (kvb: the fixture)
from test_gpu_paged_long import widen

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TIMEOUT = 7


@pytest.mark.parametrize("d,g", [(64, 20), (128, 40), (128, 64)])
def test_a_limit_of_no_time_runs_out_every_time(kvb, d, g, monkeypatch):  # noqa: F811
    # every role gives up, what it holds is released, and the units' counters are left as the next call needs them
    P = Pool(kvb, 1, 2, d, 16, 3, 9000, BF)
    widen(P)  # rows over keys that may be many: the kernel that waits
    lens = np.array([9000, 1, 700])
    P.fill(lens)
    q, one = P.rows(1, 2 * g, 3), P.rows(1, 4, 3)
    good, z = attend(P, q, offsets([1] * 3), lens - 1)
    alone, _ = attend(P, one, offsets([1] * 3), lens - 1)
    monkeypatch.setenv("KVB_WAIT_TIMEOUT_MS", "0")
    ctx0 = kvb.kvb_ctx_create(spec(1, 2, d, 1e4), spec(1, 2, d, THETA), 1, 64)
    monkeypatch.delenv("KVB_WAIT_TIMEOUT_MS")
    long, short = P.seqs([0, 1, 2, 3], lens - 1), P.seqs([0, 1, 1, 1], [0, 0, 0])
    for i in range(20):
        kvb.kvb_paged_attention(ctx0, P.cache, short if i % 4 == 3 else long, q, torch.empty_like(q))
        assert status_of(kvb, lambda: kvb.kvb_ctx_check(ctx0)) == TIMEOUT
        kvb.kvb_ctx_check(ctx0)  # reported once, then cleared
        # a call without waits on the same context and workspace
        out = torch.empty_like(one)
        kvb.kvb_paged_attention(ctx0, P.cache, long, one, out)
        kvb.kvb_ctx_check(ctx0)
        assert torch.equal(out, alone)
    out, lse = attend(P, q, offsets([1] * 3), lens - 1)
    kvb.kvb_ctx_check(P.ctx)
    assert torch.equal(out, good) and torch.equal(lse, z)


def test_a_captured_call_outlives_larger_ones(kvb):  # noqa: F811
    """Graphs of both kernels hold workspaces that later, larger calls outgrow; replayed in turn they are right."""
    P = Pool(kvb, 1, 2, 128, 64, 2, 70000, BF)
    P.fill([70000, 3000])
    side = torch.cuda.Stream()
    kinds = []
    for g, lens in ((8, [70000, 3000]), (40, [3000, 3000])):
        q = P.rows(1, 2 * g, 2)
        out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
        seqs = P.seqs([0, 1, 2], np.asarray(lens) - 1, max_kv=70000)
        kvb.kvb_paged_attention(P.ctx, P.cache, seqs, q, out, lse)
        torch.cuda.synchronize()
        want = out.clone(), lse.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            kvb.kvb_paged_attention(P.ctx, P.cache, seqs, q, out, lse)
        kinds.append((graph, out, lse, want, seqs, q))
    for n_seq, g in ((600, 8), (300, 48)):  # more units, and more rows of them
        table = P.dtab[:1].repeat(n_seq, 1)
        q = P.rows(1, 2 * g, n_seq)
        seqs = kvb.Seqs(table, i32(np.arange(n_seq + 1)), i32([999] * n_seq), max_tokens=1, max_kv=1000)
        kvb.kvb_paged_attention(P.ctx, P.cache, seqs, q, torch.empty_like(q))
        for _ in range(2):
            for graph, out, lse, want, *_ in kinds:
                out.zero_(), lse.zero_()
                torch.cuda.synchronize()
                graph.replay()
                torch.cuda.synchronize()
                assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    kvb.kvb_ctx_check(P.ctx)


@pytest.mark.parametrize("dtype,g", [(BF, 8), (BF, 40), (F32, 4)])
def test_many_sequences_of_every_length(kvb, dtype, g):  # noqa: F811
    # more sequences than a warp, and than every warp together, places in the line; a page table of one page each
    n = 700
    P = Pool(kvb, 1, 1, 64, 16, n, 16, dtype)
    lens = np.arange(n) % 16 + 1
    P.fill(lens)
    for m in (90, n):
        q = P.rows(1, g, m)
        seqs = kvb.Seqs(P.dtab[:m].contiguous(), i32(np.arange(m + 1)), i32(lens[:m] - 1), max_tokens=1)
        out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
        kvb.kvb_paged_attention(P.ctx, P.cache, seqs, q, out, lse)
        kvb.kvb_ctx_check(P.ctx)
        check_attention(P, q, np.arange(m + 1), lens[:m] - 1, out, lse)


def test_example_decodes_from_pages_of_the_models_type(kvb):  # noqa: F811
    # the cache holds what the plain one does but for the sums and table that torch rounds otherwise: a key's
    # element differs by a bf16 step, 2^-8 of it, now and then, and moves an output less than 2^-6 rad; cos 0.999 is 0.045
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import decode_mapped_cache as ex
    finally:
        sys.path.pop(0)
    r = ex.main(["--cache", "model", "--layers-src", "5", "--layers-tgt", "3", "--kv-heads", "2", "--q-heads", "8", "--prefix", "700",
                 "--tokens", "9", "--page", "32"])
    assert r["cos_min"] > 0.999 and torch.isfinite(r["out"]).all()


@pytest.mark.parametrize("d,g", [(64, 10), (128, 20), (64, 32)])
def test_sequences_without_keys_among_others(kvb, d, g):  # noqa: F811
    # several units of a CTA, of which some see nothing: the next one's rows are still its own
    n = 300
    P = Pool(kvb, 1, 2, d, 16, n, 100, BF)
    widen(P)
    P.fill([100] * n)
    q = P.rows(1, 2 * g, 2 * n)
    off, pos = offsets([2] * n), P.rng.integers(0, 98, n)
    for empty in (2, 3, 1):
        lens = np.where(np.arange(n) % 4 < empty, 0, P.rng.integers(1, 100, n))
        out, lse = attend(P, q, off, pos, kv_len=i32(lens))
        kvb.kvb_ctx_check(P.ctx)
        check_attention(P, q, off, pos, out, lse, kv_len=lens)
        for _ in range(5):
            again, z = attend(P, q, off, pos, kv_len=i32(lens))
            assert torch.equal(out, again) and torch.equal(lse, z)


def test_outputs_in_the_place_of_the_queries_are_refused(kvb):  # noqa: F811
    P = Pool(kvb, 1, 1, 64, 16, 1, 20, BF)
    P.fill([20])
    q = P.rows(1, 2, 1)
    assert status_of(kvb, lambda: kvb.kvb_paged_attention(P.ctx, P.cache, P.seqs([0, 1], [19]), q, q)) == 1


def test_everything_on_the_checked_build():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from cross_model_kv_gb300 import build
    build.build(checked=True)
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", "tests/test_gpu_paged.py",
                        "tests/test_gpu_paged_long.py", "tests/test_gpu_paged_paths.py", "-k", "not checked_build"],
                       cwd=ROOT, env=dict(os.environ, KVB_LIBRARY="checked"), capture_output=True, text=True, timeout=900)
    if r.returncode != 0 or " passed" not in r.stdout:
        pytest.fail(r.stdout[-6000:] + r.stderr[-2000:])
