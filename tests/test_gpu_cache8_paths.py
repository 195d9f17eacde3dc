"""The 8-bit cache in use: the example from a mapped cache to decoded tokens, the
operators' parity on the checked build, and a wait that runs out."""
import os
import subprocess
import sys

import numpy as np
import pytest

from cases import spec

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def kvb():
    from cross_model_kv_gb300 import build
    build.build()
    import cross_model_kv_gb300 as m
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return m


def test_example_decodes_from_a_mapped_cache(kvb):
    # a code is off by at most 2^-4 of its value and by 2^-4 / sqrt(3) in the mean square, so
    # values alone turn an output by about 0.036 rad at most; keys move the scores likewise.
    # cos 0.99 is 0.14 rad.
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import decode_mapped_cache as ex
    finally:
        sys.path.pop(0)
    r = ex.main(["--layers-src", "5", "--layers-tgt", "3", "--kv-heads", "2", "--q-heads", "8", "--prefix", "700",
                 "--tokens", "9", "--page", "32"])
    assert r["cos_mean"] > 0.99 and r["cos_min"] > 0.9
    assert torch.isfinite(r["out"]).all()


def test_parity_on_the_checked_build(kvb):
    from cross_model_kv_gb300 import build
    build.build(checked=True)
    env = dict(os.environ, KVB_LIBRARY="checked")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
                        "tests/test_gpu_cache8.py"], cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, (r.stdout[-4000:], r.stderr[-2000:])
    assert " passed" in r.stdout


def test_wait_limit_runs_out_status_reported_and_device_usable(kvb, monkeypatch):
    # with no time to wait the tensor-core kernel's roles give up, release what they hold and
    # report; the next call, on a context with the default limit, is right
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")
    T, H, g, n = 8192, 2, 8, 256
    x = [torch.randn(1, H, T, 128, device="cuda").to(torch.bfloat16) for _ in range(2)]
    q = torch.randn(1, H * g, n, 128, device="cuda").to(torch.bfloat16)
    table = torch.arange(T // 64, dtype=torch.int32, device="cuda")[None]
    s = spec(1, H, 128, 1e6)
    mk = lambda: kvb.kvb_ctx_create(s, s, 1, 64)
    ctx = mk()
    cache = kvb.kvb_cache8_create(ctx, T // 64, 64)
    kvb.kvb_cache8_write(ctx, cache, kvb.Seqs(table, i32([0, T]), i32([0]), max_tokens=T), *x)
    seqs = kvb.Seqs(table, i32([0, n]), i32([T - n]), max_tokens=n)
    good = torch.empty_like(q)
    kvb.kvb_cache8_attention(ctx, cache, seqs, q, good)
    kvb.kvb_ctx_check(ctx)
    monkeypatch.setenv("KVB_WAIT_TIMEOUT_MS", "0")
    ctx0 = mk()
    kvb.kvb_cache8_attention(ctx0, cache, seqs, q, torch.empty_like(q))
    with pytest.raises(kvb.KvbError) as e:
        kvb.kvb_ctx_check(ctx0)
    assert e.value.status == 7
    kvb.kvb_ctx_check(ctx0)  # reported once, then cleared
    monkeypatch.delenv("KVB_WAIT_TIMEOUT_MS")
    out = torch.empty_like(q)
    kvb.kvb_cache8_attention(ctx, cache, seqs, q, out)
    kvb.kvb_ctx_check(ctx)
    assert torch.equal(out, good)
