"""The paged cache on the GPU at the edges of what its calls allow: odd partials, NaN among what a query sees, chunks longer
than max_q, the largest windows, scales and queries, weights far below the largest, and the status word beside other streams.
"""

import math
import os
import subprocess
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import paged_cases as pc                                                                 # noqa: E402
from paged_cases import DT, HALF_ULP, Pages                                              # noqa: E402
from quantized_kv_cache_gb300 import KVQError, PagedKVCache, _lib, qk_norm_rope          # noqa: E402
from test_gpu_paged import decode_case, prefill_case                                     # noqa: E402

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


# ------------------------------------------------------------------------------------------------ NaN
def nan_case(fmt, dtype, what, how):
    """(out, lse, rows that see a NaN) of 3 queries over 700 positions, the second query NaN, or the keys of positions 0-255;
    in one split call, in a call that is not split (160 equal sequences), or as a decode step each."""
    H, G, D, ps, n, m = 1, 2, 64, 32, 700, 3
    p = Pages(H, D, ps, 23, *fmt, Hq=H * G, max_seqs=160, max_tokens=160 * m)
    table, _, _ = pc.fill(p, 0, [n], 3, dtype)
    q = normal((m, H * G, D), 4, dtype)
    bad = torch.zeros(m, dtype=torch.bool, device="cuda")
    if what == "query":
        q[1], bad[1] = float("nan"), True
    else:
        k = torch.full((256, H, D), float("nan"), dtype=DT[dtype], device="cuda")
        v = normal((256, H, D), 5, dtype)
        tab = table[0].cpu().numpy()
        p.cache.write(0, k, v, ints([int(tab[i // ps]) * ps + i % ps for i in range(256)]))
        bad[:] = True
    p.cache.status()
    copies = 160 if how == "whole" else 1
    many = q.repeat(copies, 1, 1)
    out, lse = torch.full_like(many, 7.0), torch.full((m * copies, H * G), 7.0, device="cuda")
    if how == "decode":
        p.cache.decode_attn(0, many, table.repeat(m, 1), ints([n] * m), out, lse=lse)
    else:
        p.cache.prefill_attn(0, many, ints([m * i for i in range(copies + 1)]), m, table.repeat(copies, 1), ints([n] * copies),
                             out, lse=lse)
    assert p.cache.status() == 0
    return out, lse, bad.repeat(copies)


@pytest.mark.parametrize("fmt,dtype", [(("f16", "f16"), "f16"), (("bf16", "bf16"), "bf16"), (("q8_0", "q4_0"), "bf16")])
@pytest.mark.parametrize("what", ["query", "keys"])
@pytest.mark.parametrize("how", ["split", "whole", "decode"])
def test_nan_among_what_a_query_sees_gives_nan(fmt, dtype, what, how):
    out, lse, bad = nan_case(fmt, dtype, what, how)
    assert torch.isnan(out[bad]).all() and torch.isfinite(out[~bad]).all()


@pytest.mark.parametrize("fmt,dtype", [(("f16", "f16"), "f16"), (("bf16", "bf16"), "bf16"), (("q8_0", "q4_0"), "bf16")])
@pytest.mark.parametrize("what", ["query", "keys"])
@pytest.mark.parametrize("how", ["split", "whole", "decode"])
def test_log_sum_exp_of_nan_scores_is_nan(fmt, dtype, what, how):
    """-inf is kept for queries that see nothing."""
    out, lse, bad = nan_case(fmt, dtype, what, how)
    assert torch.isnan(lse[bad]).all() and torch.isfinite(lse[~bad]).all()


@pytest.mark.parametrize("what", ["query", "keys"])
def test_log_sum_exp_of_nan_scores_inside_one_run(what):
    """Short sequences: a head's partials are joined inside one CTA."""
    p = Pages(2, 128, 16, 8, "f16", "f16", Hq=4, max_seqs=3)
    table, _, _ = pc.fill(p, 0, [20, 0, 33], 3)
    q = normal((3, 4, 128), 4)
    if what == "query":
        q[0, 1] = float("nan")
    else:
        nan = torch.full((20, 2, 128), float("nan"), dtype=torch.float16, device="cuda")
        p.cache.write(0, nan, nan, ints([int(table[0, i // 16]) * 16 + i % 16 for i in range(20)]))
    out, lse = torch.empty_like(q), torch.empty((3, 4), device="cuda")
    p.cache.decode_attn(0, q, table, ints([20, 0, 33]), out, lse=lse)
    bad = torch.isnan(out).all(-1)
    assert torch.equal(bad[0], torch.tensor([what == "keys", True, what == "keys", what == "keys"], device="cuda"))
    assert torch.equal(torch.isnan(lse), bad) and (lse[1] == -math.inf).all() and not out[1].any() and not bad[1:].any()


# ------------------------------------------------------------------------------------------------ lengths
@pytest.mark.parametrize("window", [(1 << 31) - 1, (1 << 31) - 3, 65, 64])
@pytest.mark.parametrize("prefix", [None, [3]])
@pytest.mark.parametrize("copies", [1, 160])
def test_window_as_wide_as_the_table_changes_nothing(window, prefix, copies):
    """A chunk longer than its sequence, so that positions start below zero, and windows up to the largest number."""
    p = Pages(1, 64, 16, 4, "f16", "f16", Hq=2, max_seqs=160, max_tokens=160 * 40)
    table, ks, vs = pc.fill(p, 0, [33], 1)
    table = table.repeat(copies, 1)
    q = normal((40, 2, 64), 2).repeat(copies, 1, 1)
    cu, lens = ints([40 * i for i in range(copies + 1)]), ints([33] * copies)
    pre = None if prefix is None else ints(prefix * copies)
    got = []
    for w in (0, window):
        out, lse = torch.full_like(q, 7.0), torch.full((40 * copies, 2), 7.0, device="cuda")
        p.cache.prefill_attn(0, q, cu, 40, table, lens, out, lse=lse, window=w, prefix=pre)
        got += [out, lse]
    assert torch.equal(got[0], got[2]) and torch.equal(got[1], got[3])
    assert torch.isfinite(got[3].view(copies, 40, 2)[:, 7:]).all() and (got[3].view(copies, 40, 2)[:, :7] == -math.inf).all()
    one = [torch.empty((copies, 2, 64), dtype=torch.float16, device="cuda") for _ in range(2)]
    for w, o in zip((0, window), one):
        p.cache.decode_attn(0, q.view(copies, 40, 2, 64)[:, 39], table, lens, o, window=w, prefix=pre)
    assert torch.equal(*one)


@pytest.mark.parametrize("H,G,D,seqs", [(1, 4, 128, 1), (2, 3, 256, 1), (16, 1, 128, 6), (16, 2, 256, 6)])
@pytest.mark.parametrize("max_q", [1, 100, 130])
def test_chunk_longer_than_max_q_leaves_the_rest(H, G, D, seqs, max_q):
    """Chunks of 300 tokens (several row tiles), split and not: the first max_q rows of each are what they should be, the
    rows behind stay as they were, and the status says so."""
    n, m = 333, 300
    p = Pages(H, D, 32, seqs * 11 + 1, "f16", "f16", Hq=H * G, max_seqs=seqs, max_tokens=seqs * m)
    table, ks, vs = pc.fill(p, 0, [n] * seqs, 3)
    q = normal((seqs * m, H * G, D), 4)
    out, lse = torch.full_like(q, 7.0), torch.full((seqs * m, H * G), 7.0, device="cuda")
    p.cache.ws.fill_(0xff)                               # what the workspace holds is not read before it is written
    p.cache.prefill_attn(0, q, ints([m * i for i in range(seqs + 1)]), max_q, table, ints([n] * seqs), out, lse=lse)
    assert p.cache.status() == _lib.PAGED_BAD_LENGTH
    for b in range(seqs):
        r, rest = slice(b * m, b * m + max_q), slice(b * m + max_q, b * m + m)
        assert (out[rest] == 7).all() and (lse[rest] == 7).all()
        want = pc.attention64(q[r].double(), ks[b], vs[b], torch.arange(n - m, n - m + max_q, device="cuda"), 1 / math.sqrt(D))
        pc.check_attention(out[r], lse[r], want, "f16", HALF_ULP["f16"], steps_of(n))


def test_tables_of_nearly_2_31_positions_refused():
    """Positions are counted in 32 bits, a tile beyond the last one too: refused on the host, the pointers are never followed."""
    p = Pages(1, 64, 16, 4, "f16", "f16")
    x = torch.zeros((1, 1, 64), dtype=torch.float16, device="cuda")
    t = ints([[0]])
    for pages in ((1 << 27) - 1, (1 << 27) - 15):
        for call, extra in ((_lib.kv_paged_decode_attn, ()), (_lib.kv_paged_prefill_attn, (1, 1))):
            args = [p.cache.h, 0, _lib.F16, 1, *extra, x.data_ptr(), 64] + ([t.data_ptr()] if extra else [])
            args += [t.data_ptr(), pages, pages, t.data_ptr(), x.data_ptr(), None, p.cache.ws.data_ptr(), p.cache.ws_bytes]
            with pytest.raises(KVQError) as e:
                call(*args)
            assert e.value.code == 1


# ------------------------------------------------------------------------------------------------ small weights
@pytest.mark.parametrize("fmt", [("f16", "f16"), ("q8_0", "q8_0"), ("q4_0", "q4_0")])
@pytest.mark.parametrize("gap", [22.3, 24.4, 25.1, 28.3])
@pytest.mark.parametrize("where", [0, 29999])
@pytest.mark.parametrize("how", ["decode", "chunk"])
def test_weights_far_below_the_largest_keep_their_share(fmt, gap, where, how):
    """One position 2^gap above 29,999 others, its value row zero, so that the output is the others'. Sequences enough
    that none is split (they read the same pages)."""
    n, D, ps = 30000, 64, 256
    B = 1216 if how == "decode" else 160
    p = Pages(1, D, ps, 118, *fmt, Hq=2, max_seqs=B, max_tokens=B)
    k, v = torch.zeros((n, 1, D), dtype=torch.float16, device="cuda"), 100 + 10 * normal((n, 1, D), 1)
    k[:, :, 0] = -gap * math.log(2)
    k[where], v[where] = 0, 0
    p.cache.write(0, k, v, torch.arange(n, dtype=torch.int32, device="cuda"))
    table = torch.arange(118, dtype=torch.int32, device="cuda").repeat(B, 1)
    rows = [torch.empty((n, 1, D), device="cuda") for _ in range(2)]
    p.cache.read(0, table[:1], ints([0, n]), *rows)
    kk, vv = (r.half().double() for r in rows)
    q = torch.zeros((B, 2, D), dtype=torch.float16, device="cuda")
    q[:, :, 0] = 8
    out, lse = torch.empty_like(q), torch.empty((B, 2), device="cuda")
    if how == "decode":
        p.cache.decode_attn(0, q, table, ints([n] * B), out, lse=lse)
    else:
        p.cache.prefill_attn(0, q, ints(range(B + 1)), 1, table, ints([n] * B), out, lse=lse)
    want, lse64, wabs, ds = pc.attention64(q[:1].double(), kk, vv, torch.tensor([n - 1], device="cuda"), 1 / 8)
    # a weight is rounded to fp16 2^15 (decode: above the warp's largest) or at least 2^11 (chunk: above the largest met) times
    # itself: half a step is 2^-11 of it, or 2^-25 where that is subnormal. Then the scores, the fp32 sums and the output.
    floor = 2.0 ** -(40 if how == "decode" else 36)
    rel = HALF_ULP["f16"] + 4 * ds[..., None] + steps_of(n) * 2.0 ** -23
    tol = HALF_ULP["f16"] * want.abs() + (1 + HALF_ULP["f16"]) * (rel * wabs + n * floor * vv.abs().max()) + 2.0 ** -25
    err = (out.double() - want).abs()
    assert (err <= tol).all(), f"{float((err / tol).max()):.3g} of the tolerance"
    assert ((lse.double() - lse64).abs() <= 2 * ds + 2.0 ** -21 * (lse64.abs() + 1) + steps_of(n) * 2.0 ** -24).all()


# ------------------------------------------------------------------------------------------------ the status word
def test_status_waits_for_every_stream():
    """A call still running on a stream of its own: its bit is in the word that is read next, and in no later one."""
    p = Pages(1, 64, 16, 4, "f16", "f16")
    x, slots = torch.ones((1, 1, 64), dtype=torch.float16, device="cuda"), ints([64])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    p.cache.write(0, x, x, slots, stream=side.cuda_stream)
    assert p.cache.status() == _lib.PAGED_BAD_INDEX
    torch.cuda.synchronize()
    assert p.cache.status() == 0


def test_creation_has_cleared_the_status_word_when_it_returns():
    """Created beside a busy default stream, used on another one at once: the bit that a first call sets stays."""
    p = Pages(1, 64, 16, 4, "f16", "f16")
    x, slots = torch.ones((1, 1, 64), dtype=torch.float16, device="cuda"), ints([64])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    with torch.cuda.stream(side):
        cache = PagedKVCache(p.cfg, 0, pool=p.pool)
        cache.write(0, x, x, slots, stream=side.cuda_stream)
    torch.cuda.synchronize()
    assert cache.status() == _lib.PAGED_BAD_INDEX


# ------------------------------------------------------------------------------------------------ ranges
LARGEST = {"q8_0": 515.5, "q4_0": 9352.0}          # 127 or 7 times it is the largest fp16 that is no infinity, or less


def taken(p, w, table, n):
    """Rows [n, H, D] (fp64) of a side's pages as the attention takes them: scales cut at LARGEST, code x scale as fp16."""
    raw, fmt, out = p.host(), p.fmt[w], []
    tab = table.cpu().numpy()
    for j in range(n):
        page, row = int(tab[j // p.ps]), j % p.ps
        y = p.get(raw, 0, w, page, row).astype(np.float64).reshape(p.H, -1, 32)
        at = p.ps * pc.row_bytes(fmt, p.D) + row * (p.D // 16)
        d = np.stack([np.ascontiguousarray(p.unit(raw, 0, w, page, h)[at:at + p.D // 16]).view(np.float16) for h in range(p.H)])
        d = d.astype(np.float64)[..., None]
        code = np.rint(y / np.where(d > 0, d, 1.0))
        out.append((code * np.minimum(d, LARGEST[fmt])).reshape(p.H, p.D))
    return torch.from_numpy(np.stack(out)).cuda().half().double()


@pytest.mark.parametrize("fmt", [("q8_0", "q8_0"), ("q8_0", "q4_0"), ("q4_0", "q4_0")])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_blocks_beyond_fp16_stay_finite_and_are_reported(fmt, dtype, D):
    """Blocks whose largest value is fp16's, or (bf16 rows) far beyond it: read back as they are stored; the attention takes
    their scales cut to what keeps code x scale finite, and the write has said so."""
    H, G, ps, n = 2, 3, 32, 150
    p = Pages(H, D, ps, 6, *fmt, Hq=H * G, max_seqs=2, max_tokens=20)
    x = [normal((n, H, D), s, dtype) for s in (1, 2)]
    table = torch.randperm(6, generator=torch.Generator().manual_seed(0)).to(torch.int32).cuda()[None, :5].contiguous()
    slots = ints([int(table[0, j // ps]) * ps + j % ps for j in range(n)])
    p.cache.write(0, *x, slots)
    assert p.cache.status() == 0
    for y in x:
        y[7, 0, 5] = 65504.0 if dtype == "f16" else 65280.0
        y[70:75, 1, 33:37] = -65504.0 if dtype == "f16" else 4.0e5
    p.cache.write(0, *x, slots)
    assert p.cache.status() == _lib.PAGED_RANGE
    back = [torch.empty((n, H, D), device="cuda") for _ in range(2)]
    p.cache.read(0, table, ints([0, n]), *back)
    for y, z in zip(x, back):
        big = y.float().abs() > 6e4
        assert ((z[big] - y.float()[big]).abs() <= y.float()[big].abs() * 2.0 ** -10).all()
    kk, vv = (taken(p, w, table[0], n) for w in range(2))
    assert torch.isfinite(kk).all() and torch.isfinite(vv).all()
    q = normal((20, H * G, D), 4, dtype, 1e-4)
    out, lse = torch.empty_like(q), torch.empty((20, H * G), device="cuda")
    p.cache.prefill_attn(0, q, ints([0, 20]), 20, table, ints([n]), out, lse=lse)
    want = pc.attention64(q.double(), kk, vv, torch.arange(n - 20, n, device="cuda"), 1 / math.sqrt(D))
    pc.check_attention(out, lse, want, dtype, HALF_ULP["f16"], steps_of(n))
    one, one_lse = torch.empty_like(q[:1]), torch.empty_like(lse[:1])
    p.cache.decode_attn(0, q[19:], table, ints([n]), one, lse=one_lse)
    pc.check_attention(one, one_lse, tuple(y[19:] for y in want), dtype, HALF_ULP["f16"], steps_of(n))
    assert p.cache.status() == 0


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_non_finite_blocks_still_give_nan(bad):
    """A block with a scale that is no number is not cut: what sees it is NaN."""
    p = Pages(1, 64, 16, 4, "q8_0", "q8_0", Hq=2, max_tokens=8)
    x = normal((40, 1, 64), 1)
    x[20, 0, 40] = bad
    p.cache.write(0, x, x, ints(range(40)))
    assert p.cache.status() == _lib.PAGED_NONFINITE
    q = normal((8, 2, 64), 2)
    out = torch.empty_like(q)
    p.cache.prefill_attn(0, q, ints([0, 8]), 8, ints([[0, 1, 2]]), ints([40]), out)
    one = torch.empty_like(q[:1])
    p.cache.decode_attn(0, q[:1], ints([[0, 1, 2]]), ints([40]), one)
    assert torch.isnan(out).all() and torch.isnan(one).all()


@pytest.mark.parametrize("big", [2.0 ** 118, 2.0 ** 126, 2.0 ** -126])
@pytest.mark.parametrize("softcap", [0.0, 1e-30, 1e38])
@pytest.mark.parametrize("how", ["decode", "chunk"])
def test_bf16_queries_of_any_size_over_codes(big, softcap, how):
    """Query rows at the ends of bf16's range, keys of zeros but for one position: no product and no factor of a score leaves
    fp32's range, so that one position takes all (a large query), or all weigh the same (a tiny one, or a tiny cap)."""
    n, D = 200, 64
    p = Pages(1, D, 16, 13, "q8_0", "q8_0", Hq=2, max_tokens=4)
    k, v = torch.zeros((n, 1, D), dtype=torch.bfloat16, device="cuda"), normal((n, 1, D), 1, "bf16")
    k[5] = 2.0 ** -10
    p.cache.write(0, k, v, ints(range(n)))
    table = ints([list(range(13))])
    rows = torch.empty((n, 1, D), dtype=torch.float32, device="cuda")
    p.cache.read(0, table, ints([0, n]), None, rows)
    vv = rows.half().double()[:, 0]
    q = torch.full((1, 2, D), big, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.empty_like(q), torch.empty((1, 2), device="cuda")
    if how == "decode":
        p.cache.decode_attn(0, q, table, ints([n]), out, lse=lse, softcap=softcap)
    else:
        p.cache.prefill_attn(0, q, ints([0, 1]), 1, table, ints([n]), out, lse=lse, softcap=softcap)
    if big > 1 and softcap != 1e-30:
        want, mag = vv[5], vv[5].abs()
    else:
        want, mag = vv.mean(0), vv.abs().mean(0)
        assert ((lse - math.log(n)).abs() < 2.0 ** -19 * 8).all()
    assert (torch.isfinite(lse)).all()
    tol = HALF_ULP["bf16"] * want.abs() + (HALF_ULP["f16"] + n * 2.0 ** -23) * mag
    assert ((out.double() - want).abs() <= tol).all()


def test_caps_beyond_fp32_in_units_of_log2_refused():
    p = Pages(1, 64, 16, 4, "f16", "f16", max_tokens=1)
    x = torch.zeros((1, 1, 64), dtype=torch.float16, device="cuda")
    out = torch.empty_like(x)
    for f in (lambda: p.cache.decode_attn(0, x, ints([[0]]), ints([1]), out, softcap=3e38),
              lambda: p.cache.prefill_attn(0, x, ints([0, 1]), 1, ints([[0]]), ints([1]), out, softcap=3e38)):
        with pytest.raises(KVQError) as e:
            f()
        assert e.value.code == 1


# ------------------------------------------------------------------------------------------------ autograd
def test_calls_without_a_gradient_say_so():
    """Tensors that require a gradient are refused while autograd records, and a value saved for a backward pass that a call
    writes over is found out."""
    p = Pages(1, 64, 16, 4, "f16", "f16", Hq=2, max_tokens=2)
    x, w = normal((2, 3, 64), 1).requires_grad_(), normal((64,), 2).requires_grad_()
    y = x * 1
    q, k, v = y[:, :2], y[:, :1], y[:, 2:]
    one, lens, table, cu = normal((64,), 2), ints([2]), ints([[0, 1]]), ints([0, 2])
    out = torch.empty((2, 2, 64), dtype=torch.float16, device="cuda")
    rows = torch.empty((2, 1, 64), device="cuda")
    calls = [lambda: qk_norm_rope(q, k, one, one, None, None), lambda: qk_norm_rope(q.detach(), None, w, None, None, None, out),
             lambda: p.cache.write(0, k, v, ints([0, 1])), lambda: p.cache.decode_attn(0, q[:1], table, lens, out[:1]),
             lambda: p.cache.prefill_attn(0, q, cu, 2, table, lens, out),
             lambda: p.cache.read(0, table, cu, rows.clone().requires_grad_())]
    before = y.detach().clone()
    for f in calls:
        with pytest.raises(ValueError, match="gradient"):
            f()
    assert torch.equal(y, before)
    with torch.no_grad():
        for f in calls:
            f()
    assert p.cache.status() == 0 and torch.isfinite(out).all()
    for over in (lambda t: qk_norm_rope(t, None, one, None, None, None),
                 lambda t: p.cache.prefill_attn(0, out, cu, 2, table, lens, t),
                 lambda t: p.cache.decode_attn(0, out[:1], table, lens, t[:1])):
        z = x[:, :2] * 2
        loss = (z * z).sum()                              # saves z
        with torch.no_grad():
            over(z)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()


# ------------------------------------------------------------------------------------------------ wide groups, wide heads
@pytest.mark.parametrize("fmt,dtype", [(("f16", "f16"), "f16"), (("bf16", "bf16"), "bf16"), (("q8_0", "q8_0"), "bf16"),
                                       (("q8_0", "q4_0"), "f16"), (("q4_0", "q4_0"), "bf16")])
@pytest.mark.parametrize("H,G,ps", [(1, 16, 256), (2, 9, 128), (3, 1, 64)])
def test_heads_of_256(fmt, dtype, H, G, ps):
    """Groups of 9 and 16 query heads, and pages longer than a tile, at the widest head."""
    lens, opts = [1, 0, 600, 257, 64], dict(window=200, prefix=ints([1, 1, 70, 1, 0]))
    decode_case(fmt, dtype, H, G, 256, ps, lens, {})
    decode_case(fmt, dtype, H, G, 256, ps, lens, opts)
    prefill_case(fmt, dtype, H, G, 256, ps, lens, [1, 0, 33, 257, 5], {})
    prefill_case(fmt, dtype, H, G, 256, ps, lens, [1, 0, 33, 257, 5], opts)


# ------------------------------------------------------------------------------------------------ calls together
FIRST_CALL = """
import torch, math
from quantized_kv_cache_gb300 import PagedKVCache, paged_config, qk_norm_rope
def ints(x): return torch.tensor(x, dtype=torch.int32, device="cuda")
c = PagedKVCache(paged_config(1, 2, 128, 8, 16, 8, "{fmt}"), 0, max_seqs=1, max_tokens=40)
x = torch.randn((40, 12, 128), device="cuda").{dtype}()
w, cs = torch.ones(128, device="cuda").{dtype}(), torch.rand((64, 128), device="cuda")
q, k, v = x[:, :8], x[:, 8:10], x[:, 10:]
pos, cu, lens, table = ints(range(40)), ints([0, 40]), ints([40]), ints([list(range(3))])
qo, ko = torch.empty((40, 8, 128), dtype=x.dtype, device="cuda"), torch.empty((40, 2, 128), dtype=x.dtype, device="cuda")
out, one, rows = torch.zeros_like(qo), torch.zeros_like(qo[:1]), torch.zeros((40, 2, 128), device="cuda")
def step():
    s = torch.cuda.current_stream().cuda_stream
    qk_norm_rope(q, k, w, w, cs, pos, qo, ko, stream=s)
    c.write(0, ko, v, pos, stream=s)
    c.read(0, table, cu, rows, stream=s)
    c.prefill_attn(0, qo, cu, 40, table, lens, out, stream=s)
    c.decode_attn(0, qo[39:], table, lens, one, stream=s)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    step()
g.replay()
torch.cuda.synchronize()
got = [t.clone() for t in (qo, ko, rows, out, one)]
step()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, (qo, ko, rows, out, one))) and got[3].abs().sum() > 0
assert (got[3][39].float() - got[4][0].float()).abs().max() < 0.05 and c.status() == 0
print("same")
"""


@pytest.mark.parametrize("fmt,dtype", [("bf16", "bfloat16"), ("q8_0", "half")])
def test_a_process_may_begin_with_a_captured_call(fmt, dtype):
    """No call comes before the capture that could have loaded a kernel or asked for its occupancy."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL.format(fmt=fmt, dtype=dtype)], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and r.stdout.split()[-1:] == ["same"], r.stderr[-2000:]


@pytest.mark.parametrize("fmt,dtype", [(("f16", "f16"), "f16"), (("q8_0", "q4_0"), "bf16")])
def test_chunks_on_two_streams_repeat_themselves(fmt, dtype):
    """Split and unsplit chunks and decode steps side by side, each with a workspace of its own: bit for bit the same every
    time."""
    p = Pages(2, 128, 32, 70, *fmt, Hq=8, max_seqs=4, max_tokens=900)
    table, _, _ = pc.fill(p, 0, [900, 300, 0, 77], 4, dtype)
    lens, q = ints([900, 300, 0, 77]), normal((900, 8, 128), 5, dtype)
    cus = [ints([0, 5, 8, 8, 12]), ints([0, 600, 850, 850, 900])]
    want = [torch.zeros_like(q) for _ in cus] + [torch.zeros_like(q[:4])]
    for cu, o in zip(cus, want):
        p.cache.prefill_attn(0, q[:int(cu[-1])], cu, 600, table, lens, o[:int(cu[-1])])
    p.cache.decode_attn(0, q[:4], table, lens, want[2])
    streams, ws = [torch.cuda.Stream() for _ in range(3)], [p.cache.new_workspace() for _ in range(3)]
    got = [[torch.zeros_like(w) for w in want] for _ in range(6)]
    n = [int(cu[-1]) for cu in cus]
    torch.cuda.synchronize()
    for outs in got:
        for i, s in enumerate(streams):
            if i < 2:
                p.cache.prefill_attn(0, q[:n[i]], cus[i], 600, table, lens, outs[i][:n[i]], ws=ws[i], stream=s.cuda_stream)
            else:
                p.cache.decode_attn(0, q[:4], table, lens, outs[2], ws=ws[2], stream=s.cuda_stream)
    torch.cuda.synchronize()
    assert p.cache.status() == 0
    for outs in got:
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_lengths_that_a_kernel_moves_between_calls():
    """Lengths advanced on the device between steps, nothing waited for: each step sees its own."""
    p = Pages(2, 64, 16, 200, "f16", "f16", Hq=4, max_seqs=2)
    table, ks, vs = pc.fill(p, 0, [1500, 900], 4)
    q, lens = normal((2, 4, 64), 5), ints([1000, 3])
    outs = [torch.empty_like(q) for _ in range(40)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for o in outs:
            lens.add_(1)
            p.cache.decode_attn(0, q, table, lens, o, stream=side.cuda_stream)
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        want = torch.empty_like(o)
        p.cache.decode_attn(0, q, table, ints([1001 + i, 4 + i]), want)
        assert torch.equal(o, want)
