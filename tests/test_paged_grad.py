"""The paged calls and autograd on the host: what is refused, and what counts as changed (CPU only)."""

import pytest

torch = pytest.importorskip("torch")

from quantized_kv_cache_gb300 import paged                                               # noqa: E402


def test_tensors_that_require_a_gradient_are_refused_where_autograd_records():
    x, leaf = torch.zeros(3), torch.zeros(3, requires_grad=True)
    paged._no_grad(x, None, leaf.detach())
    for bad in (leaf, leaf * 2):
        with pytest.raises(ValueError, match="no_grad"):
            paged._no_grad(x, None, bad)
        with torch.no_grad():
            paged._no_grad(bad)
        with torch.inference_mode():
            paged._no_grad(bad)


def test_written_tensors_count_as_changed():
    base = torch.zeros(8)
    v = base._version
    paged._changed((base[:4], base[4:]))
    assert base._version == v + 2
    with torch.inference_mode():
        paged._changed([torch.zeros(3)])
