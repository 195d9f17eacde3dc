"""smoke() runs the kernels that it names."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_smoke_reaches_both_kernels_of_paged_attention(monkeypatch):
    sys.path.insert(0, ROOT)
    try:
        import __graft_entry__ as entry
    finally:
        sys.path.pop(0)
    entry.build()
    import cross_model_kv_gb300 as kvb
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    call, names = kvb.kvb_paged_attention, []

    def attention(ctx, *args, **kw):
        kvb.kvb_profile_enable(ctx)
        kvb.kvb_profile_read(ctx)
        call(ctx, *args, **kw)
        names.extend(kvb.kvb_profile_read(ctx))
        call(ctx, *args, **kw)  # for smoke()'s own reading

    monkeypatch.setattr(kvb, "kvb_paged_attention", attention)
    entry.smoke()
    assert names == ["paged_attention", "paged_attention_tcgen05"]
