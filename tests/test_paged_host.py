"""The paged cache on the host: sizes, and what is refused before a GPU is needed (CPU only)."""

import ctypes

import pytest

from quantized_kv_cache_gb300 import _lib, build


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return _lib.load()


def config(**kw):
    c = _lib.kvq_paged_config()
    base = dict(n_layers=3, n_kv_heads=8, head_dim=128, n_q_heads=40, page_size=64, n_pages=100, k_fmt=_lib.Q8_0,
                v_fmt=_lib.Q4_0, softmax_scale=0.0)
    base.update(kw)
    for k, v in base.items():
        setattr(c, k, v)
    return c


@pytest.mark.parametrize("k,v,per_row", [("f16", "f16", 512), ("bf16", "bf16", 512), ("q8_0", "q8_0", 272),
                                         ("q8_0", "q4_0", 208), ("q4_0", "q4_0", 144)])
@pytest.mark.parametrize("ps,pages", [(16, 1), (64, 100), (256, 7)])
def test_pool_bytes(k, v, per_row, ps, pages):
    """The page's rows at the formats' sizes (34 B per 32 values for q8_0, 18 B for q4_0), each area padded to 256 B."""
    c = config(k_fmt=_lib.FMT_NAMES[k], v_fmt=_lib.FMT_NAMES[v], page_size=ps, n_pages=pages)
    pool, ws = _lib.kv_paged_required_bytes(c, 4, 100)
    rows = ps * pages * 8
    kb = {"f16": 256, "bf16": 256, "q8_0": 136, "q4_0": 72}
    areas = sum(-(-rows * kb[f] // 256) * 256 for f in (k, v))
    assert kb[k] + kb[v] == per_row
    assert pool == 256 + 3 * areas
    assert ws % 4 == 0 and ws > 0


def test_workspace_grows_with_the_batch():
    a, b = (_lib.kv_paged_required_bytes(config(), n, 0)[1] for n in (1, 1000))
    assert b > a


@pytest.mark.parametrize("kw", [dict(n_layers=0), dict(n_kv_heads=0), dict(head_dim=96), dict(head_dim=512),
                                dict(n_q_heads=41), dict(n_q_heads=8 * 17), dict(n_q_heads=0), dict(page_size=8),
                                dict(page_size=48), dict(page_size=512), dict(n_pages=0), dict(n_pages=1 << 26),
                                dict(k_fmt=_lib.TBQ4), dict(k_fmt=_lib.F16, v_fmt=_lib.BF16),
                                dict(k_fmt=_lib.Q4_0, v_fmt=_lib.Q8_0), dict(v_fmt=_lib.F16), dict(k_fmt=99),
                                dict(softmax_scale=-1.0), dict(softmax_scale=float("nan")),
                                dict(softmax_scale=float("inf")), dict(n_kv_heads=1 << 30, n_q_heads=1 << 30)])
def test_bad_configs_refused(kw):
    with pytest.raises(_lib.KVQError) as e:
        _lib.kv_paged_required_bytes(config(**kw), 1)
    assert e.value.code == 1


@pytest.mark.parametrize("seqs,tokens", [(-1, 0), (1, -1), (1, 1 << 31)])
def test_bad_batch_sizes_refused(seqs, tokens):
    with pytest.raises(_lib.KVQError):
        _lib.kv_paged_required_bytes(config(), seqs, tokens)


def test_null_arguments_refused(lib):
    h = ctypes.c_void_p()
    c = config()
    assert lib.kv_paged_required_bytes(None, 1, 0, None, None) == 1
    assert lib.kv_paged_required_bytes(ctypes.byref(c), 1, 0, None, None) == 0
    assert lib.kv_paged_create(ctypes.byref(c), None, 1 << 40, 0, ctypes.byref(h)) == 1
    assert lib.kv_paged_create(None, 256, 1 << 40, 0, ctypes.byref(h)) == 1
    assert lib.kv_paged_create(ctypes.byref(c), 256, 1, 0, ctypes.byref(h)) == 1            # pool too small
    assert lib.kv_paged_create(ctypes.byref(c), 256 + 16, 1 << 40, 0, ctypes.byref(h)) == 1  # pool misaligned
    assert lib.kv_paged_destroy(None) == 1
    assert lib.kv_paged_get_status(None, None) == 1
    assert lib.kv_paged_write(None, 0, 0, 1, 16, 1024, 16, 1024, 16, None) == 1
    assert lib.kv_paged_read(None, 0, 0, 1, 16, 1, 1, 16, None, 1, 16, 16, None) == 1
    assert lib.kv_paged_decode_attn(None, 0, 0, 1, 16, 5120, 16, 1, 1, 16, 16, None, 16, 1 << 30, None) == 1
    assert lib.kv_paged_prefill_attn(None, 0, 0, 1, 1, 1, 16, 5120, 16, 16, 1, 1, 16, 16, None, 16, 1 << 30, None) == 1
    assert lib.kv_qk_norm_rope(None, None) == 1


def norm_args(**kw):
    a = _lib.kvq_norm_rope_args()
    base = dict(dtype=_lib.F16, n_tok=4, n_q_heads=8, n_k_heads=2, head_dim=128, rot_dim=128, max_pos=100, eps=1e-6,
                q=4096, k=8192, cos_sin=4096, positions=4096, q_out=16384, k_out=32768, q_stride=1024, k_stride=256,
                q_out_stride=1024, k_out_stride=256)
    base.update(kw)
    for k, v in base.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw", [dict(dtype=_lib.Q8_0), dict(n_tok=-1), dict(n_q_heads=-1), dict(n_q_heads=0, n_k_heads=0),
                                dict(n_q_heads=1 << 21, q_stride=1 << 40), dict(head_dim=96), dict(rot_dim=24),
                                dict(rot_dim=144), dict(rot_dim=-16), dict(head_dim=512, rot_dim=16),
                                dict(eps=-1.0), dict(eps=float("nan")), dict(cos_sin=None), dict(positions=None),
                                dict(max_pos=0), dict(cos_sin=4100), dict(q=None), dict(k_out=None), dict(q=4104),
                                dict(q_stride=1000), dict(q_stride=1028), dict(k_weight=24), dict(positions=4097),
                                dict(q_out=4096, q_out_stride=2048)])
def test_norm_rope_refusals(kw):
    """Refused on the host: the pointers here are never followed."""
    with pytest.raises(_lib.KVQError) as e:
        _lib.kv_qk_norm_rope(ctypes.byref(norm_args(**kw)))
    assert e.value.code == 1


def test_norm_rope_no_tokens():
    _lib.kv_qk_norm_rope(ctypes.byref(norm_args(n_tok=0)))
