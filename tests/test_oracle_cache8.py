"""Pins of the 8-bit cache's oracle, and of the calls' host-side refusals (no GPU)."""
import ctypes
import os

import numpy as np
import pytest

from oracle import cache8 as C8


def test_e4m3_values_and_rounding():
    v = C8.e4m3_values()
    assert v[0x7e] == 448 and v[0x38] == 1 and v[0x01] == 2.0 ** -9 and v[0x08] == 2.0 ** -6 and v[0xb8] == -1
    assert np.isnan(v[0x7f]) and np.isnan(v[0xff])
    finite = np.r_[0:127, 128:255]
    assert np.array_equal(C8.e4m3_encode(v[finite]), finite)          # every number is its own rounding
    mid = (v[0:126] + v[1:127]) / 2                                   # ties go to the even byte
    assert np.array_equal(C8.e4m3_encode(mid), np.arange(126) + np.arange(126) % 2)
    assert C8.e4m3_encode(1e9) == 0x7e and C8.e4m3_encode(-460.0) == 0xfe


def test_e4m3_agrees_with_torch():
    torch = pytest.importorskip("torch")
    x = np.random.default_rng(0).standard_normal(20000) * np.exp2(np.random.default_rng(1).uniform(-12, 8, 20000))
    x = np.clip(x, -448, 448).astype(np.float32)
    t = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(C8.e4m3_encode(x), t)


def test_block_exponent_is_the_least():
    for amax, e in ((448.0, 0), (448.0001, 1), (224.0, -1), (1.0, -8), (1.75, -8), (1.76, -7), (0.0, -117),
                    (1e-45, -117), (3.4e38, 119)):
        assert C8.block_exponent(amax) == e


def test_growing_a_page_equals_writing_it_at_once_above_the_subnormals():
    # codes rounded under a small scale and lowered to a larger one are what the larger
    # scale would have given, except for values that are subnormal there
    rng = np.random.default_rng(2)
    x = rng.standard_normal((1, 1, 16, 16)) + np.where(rng.random((1, 1, 16, 16)) < 0.5, 3, -3)
    x[0, 0, 10:] *= 20
    one, two = (C8.Cache8(1, 1, 1, 16, 16) for _ in range(2))
    one.write(0, x, [[0]], [0, 16], [0])
    two.write(0, x[:, :, :7], [[0]], [0, 7], [0])
    two.write(0, x[:, :, 7:], [[0]], [0, 9], [7])
    assert np.array_equal(one.scales[0], two.scales[0]) and np.array_equal(one.codes[0], two.codes[0])
    got = two.read(0, [[0]], [0, 16], [0])
    assert np.abs(got / x - 1).max() <= 2.0 ** -4


def test_attention_of_one_visible_key_is_its_value():
    rng = np.random.default_rng(3)
    c = C8.Cache8(1, 2, 2, 16, 16)
    for kv in (0, 1):
        c.write(kv, rng.standard_normal((1, 2, 20, 16)), [[1, 0]], [0, 20], [0])
    q = rng.standard_normal((1, 4, 20, 16))
    out, lse, _, _ = c.attention(q, [[1, 0]], [0, 20], [0])
    v = c.read(1, [[1, 0]], [0, 20], [0])
    assert np.allclose(out[0, :, 0], np.repeat(v[0, :, 0], 2, axis=0))
    k = c.read(0, [[1, 0]], [0, 20], [0])
    assert np.allclose(lse[0, 3, 0], q[0, 3, 0] @ k[0, 1, 0] / 4)
    out, lse, _, _ = c.attention(q, [[1, 0]], [0, 20], [-3])
    assert np.all(out[:, :, :3] == 0) and np.all(np.isneginf(lse[:, :, :3])) and np.all(out[:, :, 3] != 0)


@pytest.fixture(scope="module")
def lib():
    from cross_model_kv_gb300 import build
    build.build()
    import cross_model_kv_gb300 as kvb
    return kvb.load_library()


def test_null_context_is_rejected(lib):
    assert lib.kvb_cache8_write(None, None, None, 0, 1, 1, None, None, 1, None) == 1
    assert lib.kvb_cache8_read(None, None, None, 0, 1, 1, None, None, 1, None) == 1
    assert lib.kvb_cache8_attention(None, None, None, 0, 1, 1, None, 8, 1, 0.0, None, None, None) == 1
    assert b"ctx" in lib.kvb_last_error()


def test_struct_layout_matches_the_header(tmp_path, lib):
    # sizes and offsets as a C compiler lays out include/kvb.h
    import shutil
    import subprocess
    from cross_model_kv_gb300 import _binding as B
    cc = shutil.which("gcc")
    if not cc:
        pytest.skip("no C compiler")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    prints = []
    want = []
    for S in (B.kvb_cache8, B.kvb_seqs):
        n = S.__name__
        prints.append(f'printf("%zu\\n", sizeof({n}));')
        want.append(ctypes.sizeof(S))
        for f, _ in S._fields_:
            prints.append(f'printf("%zu\\n", offsetof({n}, {f}));')
            want.append(getattr(S, f).offset)
    src = tmp_path / "l.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "kvb.h"\nint main(void){%s return 0;}' % "".join(prints))
    exe = tmp_path / "l"
    subprocess.run([cc, "-I", os.path.join(root, "include"), str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()
    assert [int(x) for x in out] == want
