"""Pins of the paged cache's oracle, and refusals of its calls that need no GPU."""
import ctypes
import types

import numpy as np
import pytest

from oracle import kvb_oracle as O
from oracle import paged as PG


def test_rotation_in_32_bits_is_the_rotation():
    rng = np.random.default_rng(0)
    d, theta, pos = 64, 1e6, np.array([0, 1, 7, 500, 32767])
    x = rng.standard_normal((3, 5, d)).astype(np.float32)
    cos, sin = PG.table(theta, d, 32768)
    got, want = PG.rotate32(x, pos, cos, sin), O.rope(x, pos, theta)
    # table, products and sum: one half-step of 2^-24 each, relative to the pair's magnitudes
    mag = np.abs(np.concatenate([x[..., :32], x[..., 32:]], -1)) + np.abs(np.concatenate([x[..., 32:], x[..., :32]], -1))
    assert (np.abs(got - want) <= 3 * 2.0 ** -24 * mag).all()
    assert np.array_equal(got[:, 0], x[:, 0])  # position 0 turns nothing
    back = O.rope(got.astype(np.float64), pos, theta, -1)
    assert (np.abs(back - x) <= 6 * 2.0 ** -24 * mag).all()


def test_rotation_is_a_complex_product():
    d, theta, p = 16, 1e4, 123
    x = np.random.default_rng(1).standard_normal((1, d))
    z = (x[:, :8] + 1j * x[:, 8:]) * np.exp(1j * p * theta ** (-2.0 * np.arange(8) / d))
    assert np.allclose(O.rope(x, [p], theta), np.concatenate([z.real, z.imag], -1), rtol=0, atol=1e-12)


def test_positions_outside_the_table_give_zeros():
    cos, sin = PG.table(1e4, 16, 10)
    got = PG.rotate32(np.ones((1, 3, 16)), np.array([-1, 9, 10]), cos, sin)
    assert np.all(got[0, 0] == 0) and np.all(got[0, 2] == 0) and np.any(got[0, 1] != 0)


def test_appended_pages_and_their_attention():
    rng = np.random.default_rng(2)
    P = PG.Paged(1, 4, 2, 16, 16)
    tab = np.array([[3, 1], [0, 2]])
    x = [rng.standard_normal((1, 2, 25, 16)) for _ in range(2)]
    for kv in range(2):
        P.append(kv, x[kv], tab, [0, 20, 25], [0, 3])
        assert np.array_equal(P.sequence(kv, tab[0], 20, 0, 1), x[kv][0, 1, :20])
    q = rng.standard_normal((1, 4, 1, 16))
    out, lse, _, _ = P.attention(q, tab[:1], [0, 1], [19])
    s = q[0, 3, 0] @ x[0][0, 1, :20].T / 4
    w = np.exp(s)
    assert np.allclose(out[0, 3, 0], (w / w.sum()) @ x[1][0, 1, :20]) and np.isclose(lse[0, 3, 0], np.log(w.sum()))


# ------------------------------------------------------------------ the calls, without a GPU

@pytest.fixture(scope="module")
def lib():
    from cross_model_kv_gb300 import build
    build.build()
    import cross_model_kv_gb300 as kvb
    return kvb.load_library()


def test_a_null_context_is_refused(lib):
    for name, args in (("kvb_paged_append", [None, None, 0, 1, None, None, None, None, 0, 1, 1, None]),
                       ("kvb_cache8_append", [None, None, 0, 1, 1, None, None, None, None, 0, 1, 1, None]),
                       ("kvb_paged_attention", [None, None, 0, 1, None, 1, 1, 0.0, None, None, None])):
        assert getattr(lib, name)(None, *args) == 1
        assert b"ctx is NULL" in lib.kvb_last_error()


def test_rows_are_described_by_their_strides_and_checked():
    torch = pytest.importorskip("torch")
    from cross_model_kv_gb300 import _binding as B
    here = types.SimpleNamespace(device=-1)  # where CPU tensors are
    x = torch.zeros(3, 10, 7, 16)  # [layer][token][head][dim]
    v = x[:, :, 2:4].transpose(1, 2)
    data, l, h, t = B._pack_rows.__self__.unpack(B._rows(here, "k", v, (3, 2, 10, 16), torch.float32))
    assert (data, l, h, t) == (x.data_ptr() + 2 * 16 * 4, 10 * 7 * 16, 16, 7 * 16)
    with pytest.raises(ValueError, match="k must be"):
        B._rows(here, "k", v, (3, 2, 9, 16), torch.float32)
    with pytest.raises(ValueError, match="k must be"):
        B._rows(here, "k", v, (3, 2, 10, 16), torch.bfloat16)
    with pytest.raises(ValueError, match="next to each other"):
        B._rows(here, "k", torch.zeros(3, 16, 10, 2).transpose(1, 3), (3, 2, 10, 16), torch.float32)
    with pytest.raises(ValueError, match="context's device"):
        B._rows(types.SimpleNamespace(device=0), "k", v, (3, 2, 10, 16), torch.float32)


def test_struct_layouts_match_the_header(tmp_path):
    import os
    import subprocess
    from cross_model_kv_gb300 import _binding as B
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "kvb.h"\nint main(void) { printf("%zu %zu %zu %zu %zu %zu %zu", '
                   "sizeof(kvb_rows), offsetof(kvb_rows, layer), offsetof(kvb_rows, token), sizeof(kvb_paged_cache), "
                   "offsetof(kvb_paged_cache, page_tokens), offsetof(kvb_paged_cache, n_pages), offsetof(kvb_paged_cache, v)); return 0; }\n")
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(src), "-o", str(tmp_path / "s")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "s")], capture_output=True, text=True, check=True).stdout.split()]
    p = B.kvb_paged_cache
    assert got == [B._pack_rows.__self__.size, 8, 24, ctypes.sizeof(p), p.page_tokens.offset, p.n_pages.offset, p.v.offset]
