"""The plain model of the calls on page tables, by hand, and what those calls refuse on the host (CPU only)."""

import ctypes
import random

import pytest

from pages_model import Tables
from quantized_kv_cache_gb300 import _lib, build


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return _lib.load()


def test_model_by_hand():
    t = Tables(4, 4, 8, 16)
    assert t.extend([20, 0, 0, 3]) and t.table[0][:2] == [0, 1] and t.table[3][0] == 2 and t.lens == [20, 0, 0, 3]
    assert not t.fork([0, 0], [1, 2]) and t.refs[:3] == [3, 3, 1]
    assert t.extend([1, 1, 1, 13])                       # all holders of page 1 go on: row 0 keeps it
    assert t.moved == [(1, 3), (1, 4)] and [r[1] for r in t.table[:3]] == [1, 3, 4] and t.table[3] == [2, -1, -1, -1]
    t.check()
    t.free([1, 1, 0], [0, 5, 16])
    assert t.lens == [16, 0, 21, 16] and t.table[0] == [0, -1, -1, -1] and t.refs == [2, 0, 1, 0, 1, 0, 0, 0]
    assert t.compact() == [0, -1, 2, -1, 1, -1, -1, -1] and t.table[2][:2] == [0, 1] and t.moved == [(4, 1)]
    t.check()
    assert t.fork([2, 2, 2], [1, 2, 3]) and t.lens[1] == 0               # 2 is a child too: a parent of none
    assert t.fork([2, 2, 2], [1, 1, 3]) and t.lens == [16, 21, 21, 16]     # 1 once; 3 holds positions
    t.check()


def test_model_keeps_its_counts():
    rng = random.Random(0)
    t = Tables(12, 9, 60, 16)
    failed = 0
    for _ in range(400):
        k = rng.randrange(4)
        if k == 0:
            kids = [r for r in range(12) if t.lens[r] == 0 and rng.random() < 0.5]
            up = [r for r in range(12) if t.lens[r]]
            if kids and up:
                t.fork([rng.choice(up) for _ in kids], kids)
        elif k == 1:
            failed += not t.extend([rng.choice([0, 1, 20]) for _ in range(12)])
        elif k == 2:
            rows = [rng.randrange(12) for _ in range(3)]
            t.free(rows, [rng.choice([0, rng.randrange(100)]) for _ in rows])
        else:
            t.compact()
        t.check()
    assert failed


def tables(**kw):
    t = _lib.kvq_page_tables(4, 8, 8, 4096, 8192, 16384)
    for k, v in kw.items():
        setattr(t, k, v)
    return t


def test_null_handles_refused(lib):
    t = ctypes.byref(tables())
    assert lib.kv_pages_copy(None, 1, 16, 32, None) == 1
    assert lib.kv_pages_fork(None, t, 1, 16, 32, None) == 1
    assert lib.kv_pages_extend(None, t, 16, 4096, 1 << 40, None) == 1
    assert lib.kv_pages_free(None, t, 1, 16, None, None) == 1
    assert lib.kv_pages_compact(None, t, 16, 4096, 1 << 40, None) == 1
    assert lib.kv_pages_required_bytes(None, None) == 1


def test_workspace_bytes(lib):
    c = _lib.kvq_paged_config()
    for k, v in dict(n_layers=3, n_kv_heads=8, head_dim=128, n_q_heads=40, page_size=64, n_pages=100, k_fmt=_lib.Q8_0, v_fmt=_lib.Q4_0).items():
        setattr(c, k, v)
    assert _lib.kv_pages_required_bytes(c) == 4 * (16 + 500)
    assert lib.kv_pages_required_bytes(ctypes.byref(c), None) == 1
    c.n_pages = 0
    with pytest.raises(_lib.KVQError):
        _lib.kv_pages_required_bytes(c)
