"""The e4m3 block codec that the GPU tests compare with, on the CPU: against the type of torch and by hand; sizes of such pools."""

import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import e4m3_cases as e8                                                                  # noqa: E402
from quantized_kv_cache_gb300 import KVQError, _lib, build, paged                        # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return _lib.load()


def test_values_and_codes_are_torchs():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, e8.VALUES, equal_nan=True)
    x = np.concatenate([np.linspace(-448, 448, 20001), np.random.default_rng(0).standard_normal(20000) * 2.0 ** np.arange(-12, 8).repeat(1000)])
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(e8.encode(x), want)
    mid = (e8.VALUES[:126] + e8.VALUES[1:127]) / 2                       # ties
    assert np.array_equal(e8.encode(mid), torch.from_numpy(mid).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    assert list(e8.encode([np.nan, np.inf, 0.0, -0.0])) == [127, 127, 0, 128]


@pytest.mark.parametrize("amax,e", [(0.0, -126), (448.0, 0), (448.5, 1), (224.0, -1), (1.75, -8), (1.7500001, -7), (1.0, -8), (2.0, -7),
                                    (1e-40, -126), (57344.0, 7), (57345.0, 8), (3.3895e38, 120)])
def test_powers(amax, e):
    assert e8.power(amax) == e
    assert e == -126 or 448 * 2.0 ** (e - 1) < amax <= 448 * 2.0 ** e


@pytest.mark.parametrize("ps,pad", [(16, 32), (32, 32), (128, 32), (256, 64)])
def test_pool_bytes(ps, pad):
    c = paged.paged_config(3, 5, 64, 10, ps, 7, "e4m3")
    pool, ws = _lib.kv_paged_required_bytes(c, 4, 10)
    assert pool == 256 + 6 * (-(-35 * (64 * ps + pad) // 256) * 256) and ws > 0


@pytest.mark.parametrize("k,v", [("e4m3", "q4_0"), ("e4m3", "f16"), ("q8_0", "e4m3"), ("f16", "e4m3")])
def test_formats_of_keys_and_values_go_together(k, v):
    with pytest.raises(KVQError):
        _lib.kv_paged_required_bytes(paged.paged_config(1, 2, 64, 2, 16, 4, k, v), 1)


def test_other_caches_do_not_take_the_format():
    c = _lib.kvq_config()
    c.n_layers, c.n_kv_heads, c.head_dim, c.n_q_heads, c.max_seqs, c.max_ctx = 1, 2, 128, 4, 1, 1024
    c.journal = c.tail_fmt = _lib.F16
    c.tail, c.ring_capacity = 128, 256
    c.k_body = c.v_body = _lib.Q8_0
    _lib.kv_required_bytes(c)
    c.k_body = c.v_body = _lib.PAGED_E4M3
    with pytest.raises(KVQError):
        _lib.kv_required_bytes(c)


def test_null_handle_refused(lib):
    assert lib.kv_paged_append(None, 0, 0, 1, 16, 1, 1, 16, None, 1, 16, 256, 16, 256, None) == 1
