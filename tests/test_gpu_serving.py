"""The calls around the paged cache as a serving loop makes them: pages taken, prompts attended to and stored, drafted tokens looked at and
partly taken back, a request forked, the pool brought together, a last step. Against 64 bits over what the pages hold."""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import paged_cases as pc                                                                 # noqa: E402
from paged_cases import DT, HALF_ULP                                                     # noqa: E402
from quantized_kv_cache_gb300 import (PagedKVCache, paged_config, prompt_attn, prompt_status, prompt_workspace,  # noqa: E402
                                      qk_norm_rope)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Server:
    """Three table rows over e4m3 pages; the rows of K and V that each sequence was given, beside."""

    def __init__(self, dtype, D):
        self.H, self.G, self.D, self.dtype, self.rows = 2, 3, D, dtype, 3
        self.c = PagedKVCache(paged_config(1, 2, D, 6, 16, 60, "e4m3"), 0, 3, 400)
        self.table, self.lens, self.refs = torch.full((3, 20), -1, dtype=torch.int32, device="cuda"), ints([0] * 3), ints([0] * 60)
        ang = torch.rand((300, D // 2), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
        self.cs, self.w = torch.cat((ang.cos(), ang.sin()), 1), torch.ones(D, device="cuda").to(DT[dtype])
        self.sections = (D // 8, D // 8, D // 4)
        self.ws = prompt_workspace(400, 6, D)
        self.given = [[], [], []]

    def project(self, n, seed):
        """Rotated q, k and v of n[r] new tokens of each row, and their bounds."""
        T, at = sum(n), self.lens.tolist()
        x = torch.randn((T, 10, self.D), generator=torch.Generator().manual_seed(seed)).to(DT[self.dtype]).cuda()
        pos = np.concatenate([np.arange(a, a + k) for a, k in zip(at, n)])
        q, k, v = x[:, :6], x[:, 6:8], x[:, 8:]
        qk_norm_rope(q, k, self.w, self.w, self.cs, ints(np.stack([pos, pos // 7, pos % 7]).tolist()), sections=self.sections, cyclic=True,
                     stream=self.st())
        return q, k, v, [0] + np.cumsum(n).tolist()

    def st(self):
        return torch.cuda.current_stream().cuda_stream

    def put(self, n, seed):
        """The new tokens of a step: pages for them, their rows stored. Returns q, k, v and the bounds."""
        q, k, v, cu = self.project(n, seed)
        start = self.lens.clone()
        self.c.extend(self.table, self.lens, self.refs, ints(n), stream=self.st())
        self.c.append(0, k, v, self.table, ints(cu), start, stream=self.st())
        for r in range(self.rows):
            self.given[r] += [(k[i], v[i]) for i in range(cu[r], cu[r + 1])]
        return q, k, v, cu

    def held(self):
        """K and V of each row as the attentions take them, after a look at them: each within its code's rounding of what was given."""
        lens = self.lens.tolist()
        assert lens == [len(g) for g in self.given]
        back = [torch.empty((sum(lens), self.H, self.D), device="cuda") for _ in range(2)]
        self.c.read(0, self.table, ints([0] + np.cumsum(lens).tolist()), *back, stream=self.st())
        out, at = [], 0
        for g in self.given:
            rows = [x[at:at + len(g)].half().double() for x in back]
            at += len(g)
            if g:
                for w in range(2):
                    # half a step of three bits of the value or of the smallest code (2^-9) under the block's power (2^-6 at most, for
                    # values up to 7), for each of the at most three roundings that a row gets as its block grows
                    mine = torch.stack([x[w] for x in g]).double()
                    assert mine.abs().max() < 7 and ((rows[w] - mine).abs() <= 3 * (2.0 ** -4 * mine.abs() + 2.0 ** -16)).all()
            out.append(rows)
        return out

    def check(self, q, out, lse, n):
        at = 0
        for r, (k, v) in enumerate(self.held()):
            rows = slice(at, at + n[r])
            at += n[r]
            if n[r]:
                pos = torch.arange(len(k) - n[r], len(k), device="cuda")
                want = pc.attention64(q[rows].double(), k, v, pos, 1 / math.sqrt(self.D))
                pc.check_attention(out[rows], lse[rows], want, self.dtype, 2.0 ** -11, len(k) / 16 + 64)


@pytest.mark.parametrize("dtype,D", [("f16", 128), ("bf16", 64), ("bf16", 256)])
def test_a_serving_loop(dtype, D):
    s = Server(dtype, D)
    n = [70, 33, 0]
    q, k, v, cu = s.put(n, 0)                                    # prompts: attended to by their own rows
    out, lse = torch.empty((103, 6, D), dtype=DT[dtype], device="cuda"), torch.empty((103, 6), device="cuda")
    prompt_attn(q, k, v, ints(cu), 70, out, s.ws, lse=lse, stream=s.st())
    for b in range(2):
        r = slice(cu[b], cu[b + 1])
        want = pc.attention64(q[r].double(), k[r].double(), v[r].double(), torch.arange(n[b], device="cuda"), 1 / math.sqrt(D))
        pc.check_attention(out[r], lse[r], want, dtype, HALF_ULP[dtype], 70)
    s.held()
    for step, (n, kept) in enumerate((([4, 4, 0], [1, 3]), ([5, 2, 0], [5, 0]), ([40, 3, 0], [40, 1]))):
        before = [len(g) for g in s.given]
        q, _, _, cu = s.put(n, 10 + step)                        # drafted tokens (or a further piece), some of them taken back
        out, lse = torch.empty((sum(n), 6, D), dtype=DT[dtype], device="cuda"), torch.empty((sum(n), 6), device="cuda")
        s.c.prefill_attn(0, q, ints(cu), max(n), s.table, s.lens, out, lse=lse, stream=s.st())
        s.check(q, out, lse, n)
        keep = [a + b for a, b in zip(before, kept)]
        s.c.free(s.table, s.lens, s.refs, ints([0, 1]), ints(keep), stream=s.st())
        for r in range(2):
            del s.given[r][keep[r]:]
    s.c.fork(s.table, s.lens, s.refs, ints([0]), ints([2]), stream=s.st())
    s.given[2] = list(s.given[0])
    for step in range(3):                                        # the fork goes its own way
        n = [1, 1, 1]
        q, _, _, cu = s.put(n, 20 + step)
        out, lse = torch.empty((3, 6, D), dtype=DT[dtype], device="cuda"), torch.empty((3, 6), device="cuda")
        s.c.decode_attn(0, q, s.table, s.lens, out, lse=lse, stream=s.st())
        s.check(q, out, lse, n)
    s.c.free(s.table, s.lens, s.refs, ints([0]), stream=s.st())
    s.given[0] = []
    s.c.compact(s.table, s.lens, s.refs, ints([0] * 60), stream=s.st())
    used = int((s.refs > 0).sum())
    assert (s.refs[:used] > 0).all() and int(s.refs.sum()) == sum(-(-len(g) // 16) for g in s.given)
    q, _, _, cu = s.put([0, 1, 1], 30)
    out, lse = torch.empty((2, 6, D), dtype=DT[dtype], device="cuda"), torch.empty((2, 6), device="cuda")
    s.c.prefill_attn(0, q, ints(cu), 1, s.table, s.lens, out, lse=lse, stream=s.st())
    s.check(q, out, lse, [0, 1, 1])
    assert s.c.status() == 0 and prompt_status(s.ws) == 0
