"""The paged cache on the GPU at the edges of what its calls allow: odd partials, NaN among what a query sees, chunks longer
than max_q, the largest windows, scales and queries, weights far below the largest, and the status word beside other streams.
"""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import paged_cases as pc                                                                 # noqa: E402
from paged_cases import DT, HALF_ULP, Pages                                              # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def ints(x, dev="cuda:0"):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def steps_of(n):
    return n / 16 + 64


def normal(shape, seed, dtype="f16", scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn(shape, generator=g, device="cuda")).to(DT[dtype])


# ------------------------------------------------------------------------------------------------ split chunks
@pytest.mark.parametrize("H,G,qlens", [(5, 3, [2, 1]), (3, 3, [1] * 7), (1, 1, [1])])
@pytest.mark.parametrize("fmt,dtype", [(("f16", "f16"), "f16"), (("bf16", "bf16"), "bf16"), (("q8_0", "q4_0"), "bf16")])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_split_chunk_with_odd_counts(H, G, qlens, fmt, dtype, D):
    """Heads, rows and (where the SMs allow it: 15 and 7 on 152 of them) splits all odd, over 700 positions."""
    n, T = 700, sum(qlens)
    p = Pages(H, D, 32, len(qlens) * 22 + 1, *fmt, Hq=H * G, max_seqs=len(qlens), max_tokens=T)
    table, ks, vs = pc.fill(p, 0, [n] * len(qlens), 3, dtype)
    q = normal((T, H * G, D), 4, dtype)
    out, lse = torch.empty_like(q), torch.empty((T, H * G), device="cuda")
    cu = [0] + [int(x) for x in np.cumsum(qlens)]
    p.cache.prefill_attn(0, q, ints(cu), max(qlens), table, ints([n] * len(qlens)), out, lse=lse)
    assert p.cache.status() == 0
    for b, m in enumerate(qlens):
        r = slice(cu[b], cu[b + 1])
        want = pc.attention64(q[r].double(), ks[b], vs[b], torch.arange(n - m, n, device="cuda"), 1 / math.sqrt(D))
        pc.check_attention(out[r], lse[r], want, dtype, HALF_ULP["bf16" if fmt[0] == "bf16" else "f16"], steps_of(n))
