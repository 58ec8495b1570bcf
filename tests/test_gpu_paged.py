"""The paged cache on the GPU: rows written, read back and attended to, and the norm and rotation before.

Stored bytes are compared with the oracle's codecs byte for byte, rows read back bit for bit, attention
and the norm with 64-bit restatements within bounds that add up the roundings the kernels make.
"""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import paged_cases as pc                                                                 # noqa: E402
from paged_cases import DT, HALF_ULP, Pages                                              # noqa: E402
from quantized_kv_cache_gb300 import KVQError, PagedKVCache, _lib, qk_norm_rope          # noqa: E402

pytestmark = pytest.mark.gpu

FORMATS = [("f16", "f16"), ("bf16", "bf16"), ("q8_0", "q8_0"), ("q8_0", "q4_0"), ("q4_0", "q4_0")]


@pytest.fixture(autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def ints(x, dev="cuda:0"):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def stream():
    return torch.cuda.current_stream().cuda_stream


# ------------------------------------------------------------------------------------------------ write
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("H,D,ps", [(1, 64, 16), (3, 128, 32), (2, 256, 256)])
def test_write_stores_the_codecs_bytes(fmt, dtype, H, D, ps):
    """Strided rows, skipped tokens, several layers: the written rows' bytes are the oracle's, every other byte of
    the pool is what it was."""
    p = Pages(H, D, ps, 5, *fmt, layers=2)
    before = p.host()
    g = torch.Generator().manual_seed(1)
    T = 2 * ps + 3
    kv = torch.randn((T, 2 * H + 1, D), generator=g)
    kv[0] = 0.0                              # zero blocks
    kv[1, :, :32] = 1e-6                     # scales that underflow
    kv[2] *= 3000.0
    kv[3, :, ::2] = 0.5                      # ties of the codes
    kv = kv.to(DT[dtype]).cuda()
    k, v = kv[:, :H], kv[:, H:2 * H]
    slots = np.random.default_rng(2).permutation(5 * ps)[:T].astype(np.int32)
    slots[5] = -1
    slots[T - 1] = -3
    p.cache.write(1, k, v, ints(slots))
    torch.cuda.synchronize()
    want = before
    for w, x in ((0, k), (1, v)):
        x = x.float().cpu().numpy()
        for i, s in enumerate(slots):
            if s >= 0:
                p.put(want, 1, w, s // ps, s % ps, x[i])
    got = p.host()
    assert np.array_equal(got, np.concatenate([np.zeros(256, np.uint8), want[256:]]))
    assert p.cache.status() == 0


def test_write_flags_bad_slots_and_non_finite_scales():
    p = Pages(2, 64, 16, 4, "q8_0", "q8_0")
    before = p.host()
    x = torch.ones((3, 2, 64), dtype=torch.float16, device="cuda")
    p.cache.write(0, x, x, ints([64, 1 << 30, -5]))
    assert p.cache.status() == _lib.PAGED_BAD_INDEX
    assert np.array_equal(p.host()[256:], before[256:])
    x[1, 0, 40] = float("inf")
    p.cache.write(0, x, x, ints([0, 1, 2]))
    assert p.cache.status() == _lib.PAGED_NONFINITE
    x[1, 0, 40] = float("nan")
    p.cache.write(0, x, x, ints([0, 1, 2]))
    assert p.cache.status() == _lib.PAGED_NONFINITE
    assert p.cache.status() == 0


def test_write_no_tokens():
    p = Pages(1, 64, 16, 2, "f16", "f16")
    x = torch.ones((0, 1, 64), dtype=torch.float16, device="cuda")
    p.cache.write(0, x, x, ints([]))
    assert p.cache.status() == 0


# ------------------------------------------------------------------------------------------------ read
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("out", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("H,D,ps", [(2, 64, 16), (3, 128, 64), (1, 256, 128)])
def test_read_gives_the_stored_values(fmt, out, H, D, ps):
    p = Pages(H, D, ps, 9, *fmt)
    table, _, _ = pc.fill(p, 0, [2 * ps + 1, 0, ps, 5], 3)
    raw, tab = p.host(), table.cpu().numpy()
    start = [1, 0, ps - 1, 0]
    n = [2 * ps, 0, 1, 5]
    cu = np.concatenate([[2], 2 + np.cumsum(n)])
    rows = int(cu[-1]) + 3
    outs = [torch.full((rows, H, D), 7.0, dtype=DT[out], device="cuda") for _ in range(2)]
    p.cache.read(0, table, ints(cu), outs[0], outs[1], start=ints(start))
    torch.cuda.synchronize()
    for w in range(2):
        want = torch.full((rows, H, D), 7.0, dtype=DT[out])
        for b in range(4):
            for i in range(n[b]):
                at = start[b] + i
                want[cu[b] + i] = torch.from_numpy(p.get(raw, 0, w, tab[b, at // ps], at % ps)).to(DT[out])
        assert torch.equal(outs[w].cpu(), want)
    # either side alone
    one = torch.zeros_like(outs[1])
    p.cache.read(0, table, ints(cu), None, one, start=ints(start))
    assert torch.equal(one[2:cu[-1]], outs[1][2:cu[-1]])
    one.zero_()
    p.cache.read(0, table, ints(cu), one, None, start=ints(start))
    assert torch.equal(one[2:cu[-1]], outs[0][2:cu[-1]])
    assert p.cache.status() == 0


def test_read_reports_bad_pages_and_lengths():
    p = Pages(1, 64, 16, 4, "f16", "f16")
    table, k, v = pc.fill(p, 0, [20], 3, spare=0)
    out = torch.full((40, 1, 64), 7.0, dtype=torch.float32, device="cuda")
    bad = table.clone()
    bad[0, 1] = 4
    p.cache.read(0, bad, ints([0, 20]), out)
    assert p.cache.status() == _lib.PAGED_BAD_INDEX
    assert torch.equal(out[:16].double(), k[0][:16]) and not out[16:20].any() and (out[20:] == 7).all()
    p.cache.read(0, table, ints([0, 33]), out)               # one row more than the table holds
    assert p.cache.status() == _lib.PAGED_BAD_LENGTH and not out[32].any() and (out[33:] == 7).all()
    p.cache.read(0, table, ints([0, 50]), out[:8])           # rows beyond the buffer are left out
    assert p.cache.status() == _lib.PAGED_BAD_LENGTH and (out[33:] == 7).all()


# ------------------------------------------------------------------------------------------------ decode
def steps_of(n):
    return n / 16 + 64


def decode_case(fmt, dtype, H, G, D, ps, lens, opts, seed=0, q_scale=1.0, pages=None):
    p = Pages(H, D, ps, pages or sum(-(-n // ps) for n in lens) + 1, *fmt, Hq=H * G, max_seqs=len(lens), seed=seed)
    table, ks, vs = pc.fill(p, 0, lens, seed, dtype)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    wide = torch.randn((len(lens), H * G + 2 * H, D), generator=g, device="cuda")
    q = (q_scale * wide).to(DT[dtype])[:, :H * G]                       # a slice of a wider projection
    out = torch.full((len(lens), H * G, D), float("nan"), dtype=DT[dtype], device="cuda")
    lse = torch.full((len(lens), H * G), float("nan"), device="cuda")
    p.cache.decode_attn(0, q, table, ints(lens), out, lse=lse, **opts)
    torch.cuda.synchronize()
    assert p.cache.status() == 0
    # the weights of bf16 pages go in as two bf16 parts (2^-16 of them), those of the others as fp16
    p_half = 2.0 ** -16 if fmt[0] == "bf16" else HALF_ULP["f16"]
    for b, n in enumerate(lens):
        pre = int(opts["prefix"][b]) if "prefix" in opts else 0
        want = pc.attention64(q[b:b + 1].double(), ks[b], vs[b], torch.tensor([n - 1], device="cuda"),
                              1 / math.sqrt(D), opts.get("softcap", 0.0), opts.get("window", 0), opts.get("slopes"), pre)
        pc.check_attention(out[b:b + 1], lse[b:b + 1], want, dtype, p_half, steps_of(n))
    return p, table, q, out, lse


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("H,G,D,ps", [(2, 1, 64, 16), (1, 16, 128, 32), (3, 5, 128, 64), (2, 6, 256, 16), (1, 9, 64, 256)])
def test_decode_matches_64_bits(fmt, dtype, H, G, D, ps):
    if fmt[0] in DT and fmt[0] != dtype:
        pytest.skip("16-bit pages take queries of their own type")
    decode_case(fmt, dtype, H, G, D, ps, [1, 0, 16, 17, 500, 1291, 15], {})


@pytest.mark.parametrize("fmt", [("f16", "f16"), ("bf16", "bf16"), ("q8_0", "q4_0")])
@pytest.mark.parametrize("opts", [dict(softcap=5.0), dict(window=1), dict(window=33), dict(window=10000),
                                  dict(slopes=True), dict(prefix=[0, 3, 40, 700, -2]), dict(window=20, prefix=[5, 16, 33, 640, 0]),
                                  dict(softcap=30.0, slopes=True, window=64, prefix=[1, 1, 1, 1, 1])])
def test_decode_options(fmt, opts):
    opts = dict(opts)
    if "slopes" in opts:
        opts["slopes"] = 2.0 ** -torch.arange(1, 9, device="cuda", dtype=torch.float32)
    if "prefix" in opts:
        opts["prefix"] = ints(opts["prefix"])
    decode_case(fmt, "bf16" if fmt[0] == "bf16" else "f16", 2, 4, 128, 32, [1, 16, 47, 650, 2049], opts)


def test_decode_sharp_scores_and_large_queries():
    """One position far above the others, and bf16 queries beyond fp16's range on quantised pages."""
    decode_case(("f16", "f16"), "f16", 2, 4, 128, 16, [300, 5], {}, q_scale=20.0)
    decode_case(("q8_0", "q8_0"), "bf16", 2, 4, 64, 16, [300, 5], dict(softcap=1.0), q_scale=1e6)
    decode_case(("q8_0", "q8_0"), "bf16", 2, 4, 64, 16, [300, 5], {}, q_scale=1e-9)


def test_decode_ignores_what_no_query_sees():
    """NaN and infinities behind the last position of a page, before the window, and in unused pages: outputs
    are bit for bit those of zeros there."""
    for fmt, dtype in ((("f16", "f16"), "f16"), (("bf16", "bf16"), "bf16"), (("q8_0", "q4_0"), "f16")):
        p = Pages(1, 128, 32, 8, *fmt, Hq=4, max_seqs=2)
        lens, res = [70, 33], []
        for junk in (0x00, 0xff, 0x7c):
            p.pool[256:] = junk
            table, _, _ = pc.fill(p, 0, lens, 5, dtype)
            nan = torch.full((20, 1, 128), float("nan"), dtype=DT[dtype], device="cuda")
            page0 = int(table[0, 0])
            p.cache.write(0, nan, nan, ints([page0 * 32 + i for i in range(20)]))        # before the window of 40
            q = torch.randn((2, 4, 128), generator=torch.Generator().manual_seed(1)).to(DT[dtype]).cuda()
            out = torch.empty_like(q)
            p.cache.decode_attn(0, q, table, ints(lens), out, window=40)
            res.append(out)
        assert torch.isfinite(res[0]).all()
        assert torch.equal(res[0], res[1]) and torch.equal(res[0], res[2])


def test_decode_many_sequences_and_one_long():
    decode_case(("bf16", "bf16"), "bf16", 1, 2, 64, 16, [(7 * i) % 61 for i in range(300)], {})
    # more heads than a launch has CTAs, some of them cut by a CTA's run, some empty
    decode_case(("q8_0", "q8_0"), "bf16", 4, 2, 64, 16, [0] + [(37 * i) % 400 if i % 5 else 0 for i in range(600)] + [9000, 0], {})
    decode_case(("q8_0", "q8_0"), "f16", 1, 4, 128, 64, [30001], {})


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 34, 64])
@pytest.mark.parametrize("opts", [{}, dict(window=300)])
def test_decode_heads_cut_by_runs_at_any_number_of_sequences(n, opts):
    """Every count of sequences around a warp's width, with empty ones first, between and last, and heads in several runs."""
    lens = [(977 * (i + 1)) % 3001 if i % 4 != 1 else 0 for i in range(n)]
    lens[-1] = 0 if n == 34 else 4000
    if n == 33:
        lens[0] = 0
    decode_case(("f16", "f16"), "f16", 3, 2, 64, 32, lens, opts)


@pytest.mark.parametrize("n", [5, 40])
def test_captured_decodes_back_to_back_follow_their_lengths(n):
    """Two captured calls in a row over one workspace, replayed with other lengths: what the calls give outside a graph."""
    lens = [700, 0, 33, 1500, 1] + [(91 * i) % 900 for i in range(n - 5)]
    p, table, q, out, lse = decode_case(("f16", "f16"), "f16", 2, 4, 64, 16, lens, {})
    now, out2 = ints(lens), torch.empty_like(out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side = torch.cuda.current_stream().cuda_stream
        p.cache.decode_attn(0, q, table, now, out, stream=side)
        p.cache.decode_attn(0, q, table, now, out2, window=50, stream=side)
    for shift in (0, 1, 2):
        turned = ints([min(lens[i], (i + 1) * 97 * shift) if shift else lens[i] for i in range(n)])
        now.copy_(turned)
        graph.replay()
        got, got2 = out.clone(), out2.clone()
        a, b = torch.empty_like(out), torch.empty_like(out)
        p.cache.decode_attn(0, q, table, turned, a)
        p.cache.decode_attn(0, q, table, turned, b, window=50)
        assert torch.equal(got, a) and torch.equal(got2, b)


def test_decode_reports_bad_pages_and_lengths():
    p, table, q, out, _ = decode_case(("f16", "f16"), "f16", 1, 2, 64, 16, [40, 20], {})
    bad = table.clone()
    bad[0, 1] = 1 << 20
    p.cache.decode_attn(0, q, bad, ints([40, 20]), out)
    assert p.cache.status() == _lib.PAGED_BAD_INDEX
    p.cache.decode_attn(0, q, table[:, :2], ints([33, -4]), out)
    assert p.cache.status() == _lib.PAGED_BAD_LENGTH
    assert not out[1].any()


def test_decode_far_pages():
    """Pages beyond 4 GB of the pool: byte offsets past 32 bits."""
    p = pc.Pages.__new__(Pages)
    p.H, p.D, p.ps, p.fmt, p.n_pages, p.layers = 8, 128, 256, ("f16", "f16"), 12000, 1
    p.cfg = pc.paged_config(1, 8, 128, 16, 256, 12000, "f16")
    p.dev = torch.device("cuda", 0)
    p.cache = PagedKVCache(p.cfg, 0, 1, 0, pool=torch.empty(256 + 2 * 12000 * 8 * 256 * 256, dtype=torch.uint8, device="cuda"))
    n = 600
    g = torch.Generator(device="cuda").manual_seed(0)
    k, v = (torch.randn((n, 8, 128), generator=g, device="cuda").half() for _ in range(2))
    pages = [11999, 3, 11998]
    p.cache.write(0, k, v, ints([pages[i // 256] * 256 + i % 256 for i in range(n)]))
    q = torch.randn((1, 16, 128), generator=g, device="cuda").half()
    out = torch.empty_like(q)
    p.cache.decode_attn(0, q, ints([pages]), ints([n]), out)
    want = pc.attention64(q.double(), k.double(), v.double(), torch.tensor([n - 1], device="cuda"), 1 / math.sqrt(128))
    pc.check_attention(out, None, want, "f16", HALF_ULP["f16"], steps_of(n))
    back = torch.empty_like(k)
    p.cache.read(0, ints([pages]), ints([0, n]), back)
    assert torch.equal(back, k)
    out2 = torch.empty_like(q)
    p.cache.prefill_attn(0, q, ints([0, 1]), 1, ints([pages]), ints([n]), out2)
    pc.check_attention(out2, None, want, "f16", HALF_ULP["f16"], steps_of(n))


# ------------------------------------------------------------------------------------------------ prefill
def prefill_case(fmt, dtype, H, G, D, ps, lens, qlens, opts, seed=0, gap=0, q_scale=1.0):
    p = Pages(H, D, ps, sum(-(-n // ps) for n in lens) + 1, *fmt, Hq=H * G, max_seqs=len(lens),
              max_tokens=sum(qlens) + 2 * gap, seed=seed)
    table, ks, vs = pc.fill(p, 0, lens, seed, dtype)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    T = sum(qlens) + 2 * gap
    wide = torch.randn((T, H * G + 2 * H, D), generator=g, device="cuda")
    q = (q_scale * wide).to(DT[dtype])[:, :H * G]
    out = torch.full((T, H * G, D), 7.0, dtype=DT[dtype], device="cuda")
    lse = torch.full((T, H * G), 7.0, device="cuda")
    cu = [gap] + [gap + int(x) for x in np.cumsum(qlens)]
    p.cache.prefill_attn(0, q, ints(cu), max(qlens), table, ints(lens), out, lse=lse, **opts)
    torch.cuda.synchronize()
    assert p.cache.status() == 0
    for x in (out, lse):
        assert (x[:gap] == 7).all() and (x[T - gap:] == 7).all()
    p_half = HALF_ULP["bf16" if fmt[0] == "bf16" else "f16"]
    for b, n in enumerate(lens):
        pre = int(opts["prefix"][b]) if "prefix" in opts else 0
        r = slice(cu[b], cu[b + 1])
        pos = torch.arange(n - qlens[b], n, device="cuda")
        want = pc.attention64(q[r].double(), ks[b], vs[b], pos, 1 / math.sqrt(D), opts.get("softcap", 0.0),
                              opts.get("window", 0), opts.get("slopes"), pre)
        pc.check_attention(out[r], lse[r], want, dtype, p_half, steps_of(n))
    return p, table, q, out


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("H,G,D,ps", [(2, 1, 64, 16), (1, 16, 128, 32), (2, 5, 128, 64), (2, 6, 256, 16), (1, 9, 64, 256)])
def test_prefill_matches_64_bits(fmt, dtype, H, G, D, ps):
    if fmt[0] in DT and fmt[0] != dtype:
        pytest.skip("16-bit pages take queries of their own type")
    prefill_case(fmt, dtype, H, G, D, ps, [1, 0, 16, 130, 500, 300, 257], [1, 0, 16, 129, 1, 300, 0], {}, gap=3)


@pytest.mark.parametrize("fmt", [("f16", "f16"), ("bf16", "bf16"), ("q8_0", "q4_0")])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("opts", [dict(softcap=5.0), dict(window=1), dict(window=33), dict(window=10000), dict(slopes=True),
                                  dict(prefix=[0, 3, 40, 700, -2]), dict(window=20, prefix=[5, 16, 33, 400, 0]),
                                  dict(softcap=30.0, slopes=True, window=64, prefix=[1, 200, 1, 1, 1])])
def test_prefill_options(fmt, D, opts):
    opts = dict(opts)
    if "slopes" in opts:
        opts["slopes"] = 2.0 ** -torch.arange(1, 9, device="cuda", dtype=torch.float32)
    if "prefix" in opts:
        opts["prefix"] = ints(opts["prefix"])
    prefill_case(fmt, "bf16" if fmt[0] == "bf16" else "f16", 2, 4, D, 32, [1, 260, 47, 650, 1049], [1, 260, 7, 150, 30], opts)


def test_prefill_long_context_few_rows():
    prefill_case(("bf16", "bf16"), "bf16", 1, 2, 128, 64, [20011, 9000], [3, 1], {})
    prefill_case(("q8_0", "q4_0"), "f16", 1, 5, 128, 64, [20011], [9], {})


def test_prefill_sharp_scores_and_large_queries():
    """One position far above the others, and bf16 queries beyond fp16's range on quantised pages."""
    prefill_case(("f16", "f16"), "f16", 2, 4, 128, 16, [300, 5], [60, 5], {}, q_scale=20.0)
    prefill_case(("q8_0", "q8_0"), "bf16", 2, 4, 64, 16, [300, 5], [60, 5], dict(softcap=1.0), q_scale=1e6)
    prefill_case(("q8_0", "q4_0"), "bf16", 2, 4, 256, 16, [300, 5], [60, 5], {}, q_scale=1e-9)


def test_prefill_rows_before_the_first_position_see_nothing():
    """A chunk longer than the positions held: rows at negative positions give zeros and lse -inf."""
    p = Pages(1, 64, 16, 4, "f16", "f16", Hq=2)
    table, ks, vs = pc.fill(p, 0, [10], 1)
    q = torch.randn((13, 2, 64), device="cuda").half()
    out, lse = torch.full_like(q, 7.0), torch.full((13, 2), 7.0, device="cuda")
    p.cache.prefill_attn(0, q, ints([0, 13]), 13, table, ints([10]), out, lse=lse, prefix=ints([4]))
    want = pc.attention64(q.double(), ks[0], vs[0], torch.arange(-3, 10, device="cuda"), 1 / 8, prefix=4)
    assert not out[:3].any() and (lse[:3] == -math.inf).all()
    pc.check_attention(out, lse, want, "f16", HALF_ULP["f16"], steps_of(10))


def test_prefill_ignores_rows_behind_the_last_position():
    for fmt, dtype in ((("f16", "f16"), "f16"), (("bf16", "bf16"), "bf16"), (("q8_0", "q4_0"), "f16")):
        p = Pages(1, 128, 32, 8, *fmt, Hq=4, max_seqs=2)
        res = []
        for junk in (0x00, 0xff, 0x7c):
            p.pool[256:] = junk
            table, _, _ = pc.fill(p, 0, [70, 33], 5, dtype)
            q = torch.randn((40, 4, 128), generator=torch.Generator().manual_seed(1)).to(DT[dtype]).cuda()
            out = torch.empty_like(q)
            p.cache.prefill_attn(0, q, ints([0, 33, 40]), 33, table, ints([70, 33]), out)
            res.append(out)
        assert torch.isfinite(res[0]).all()
        assert torch.equal(res[0], res[1]) and torch.equal(res[0], res[2])


def test_prefill_later_rows_do_not_reach_earlier_queries():
    """NaN and infinities in the keys and values of later positions: the queries before them stay within the
    bound of the rows as they were (a tile that holds one may weigh its rows unrounded, so not bit for bit)."""
    for fmt, dtype in ((("f16", "f16"), "f16"), (("bf16", "bf16"), "bf16"), (("q8_0", "q8_0"), "f16")):
        p = Pages(1, 128, 32, 8, *fmt, Hq=4, max_seqs=1)
        table, ks, vs = pc.fill(p, 0, [200], 5, dtype)
        q = torch.randn((200, 4, 128), generator=torch.Generator().manual_seed(1)).to(DT[dtype]).cuda()
        want = pc.attention64(q.double(), ks[0], vs[0], torch.arange(200, device="cuda"), 1 / math.sqrt(128))
        bad = torch.full((3, 1, 128), float("nan"), dtype=DT[dtype], device="cuda")
        bad[1] = float("inf")
        slots = [int(table[0, i // 32]) * 32 + i % 32 for i in (151, 160, 199)]
        p.cache.write(0, bad, bad, ints(slots))
        out2 = torch.empty_like(q)
        p.cache.prefill_attn(0, q, ints([0, 200]), 200, table, ints([200]), out2)
        pc.check_attention(out2[:151], None, tuple(x[:151] for x in want), dtype,
                           HALF_ULP["bf16" if fmt[0] == "bf16" else "f16"], steps_of(200))
        assert not torch.isfinite(out2[199]).all()


def test_prefill_reports_bad_lengths():
    p, table, q, out = prefill_case(("f16", "f16"), "f16", 1, 2, 64, 16, [40, 20], [4, 4], {})
    for cu, mq, lens in (([0, 4, 9], 5, [40, 20]), ([0, 4, 8], 3, [40, 20]), ([-1, 4, 8], 5, [40, 20]),
                         ([0, 4, 3], 5, [40, 20]), ([0, 4, 8], 4, [4000, 20]), ([0, 4, 8], 4, [-1, 20])):
        p.cache.prefill_attn(0, q, ints(cu), mq, table, ints(lens), out)
        assert p.cache.status() & _lib.PAGED_BAD_LENGTH
    bad = table.clone()
    bad[1, 0] = -1
    p.cache.prefill_attn(0, q, ints([0, 4, 8]), 4, bad, ints([40, 20]), out)
    assert p.cache.status() == _lib.PAGED_BAD_INDEX


# ------------------------------------------------------------------------------------------------ norm and rotation
def norm64(x, w, cs, pos, inter, eps):
    y = x.double()
    if w is not None:
        y = y / (y.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
    if cs is not None:
        rot = cs.shape[1]
        c, s = cs.double()[pos.long()][:, None].split(rot // 2, -1)
        z = y.clone()
        a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if inter else (y[..., :rot // 2], y[..., rot // 2:rot])
        if inter:
            z[..., 0:rot:2], z[..., 1:rot:2] = a * c - b * s, b * c + a * s
        else:
            z[..., :rot // 2], z[..., rot // 2:rot] = a * c - b * s, b * c + a * s
        return z, y
    return y, y


def check_norm(got, want, dtype, D):
    z, y = want
    # fp32 steps: the sum of D squares in a tree of products (D 2^-24 bounds it), rsqrt, three products, two of
    # the rotation and one sum: of the magnitudes of the pair, which the row's largest value bounds
    step = (D / 2 + 16) * 2.0 ** -24
    tol = HALF_ULP[dtype] * z.abs() + step * 2 * y.abs().amax(-1, keepdim=True) + (2.0 ** -25 if dtype == "f16" else 0.0)
    err = (got.double() - z).abs()
    assert (err <= tol).all(), f"{float((err / tol).max()):.3g} of the tolerance"


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D,rot", [(64, 64), (64, 16), (128, 128), (128, 96), (256, 64), (256, 256), (512, 512), (512, 160), (128, 0)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,Hq,H", [(1, 5, 1), (33, 24, 4), (700, 3, 3)])
def test_norm_rope_matches_64_bits(dtype, D, rot, inter, T, Hq, H):
    g = torch.Generator(device="cuda").manual_seed(D + rot + T)
    x = (3 * torch.randn((T, Hq + 2 * H, D), generator=g, device="cuda")).to(DT[dtype])
    x[0, 0] = 0.0
    q, k = x[:, :Hq], x[:, Hq:Hq + H]
    wq, wk = (1 + 0.2 * torch.randn((2, D), generator=g, device="cuda")).to(DT[dtype])
    ang = torch.rand((900, max(rot // 2, 1)), generator=g, device="cuda") * 7
    cs = torch.cat((ang.cos(), ang.sin()), 1).contiguous() if rot else None
    pos = torch.randint(0, 900, (T,), generator=g, device="cuda", dtype=torch.int32) if rot else None
    qo, ko = torch.empty((T, Hq, D), dtype=DT[dtype], device="cuda"), torch.empty((T, H, D), dtype=DT[dtype], device="cuda")
    qk_norm_rope(q, k, wq, wk, cs, pos, qo, ko, eps=1e-5, interleaved=inter)
    check_norm(qo, norm64(q, wq, cs, pos, inter, 1e-5), dtype, D)
    check_norm(ko, norm64(k, wk, cs, pos, inter, 1e-5), dtype, D)
    # one side without its norm, in place in the fused buffer; the rest of the buffer stays
    keep = x.clone()
    qk_norm_rope(q, k, None, wk, cs, pos, eps=1e-5, interleaved=inter)
    check_norm(q, norm64(keep[:, :Hq], None, cs, pos, inter, 1e-5), dtype, D)
    assert torch.equal(k, ko) and torch.equal(x[:, Hq + H:], keep[:, Hq + H:])


def test_norm_rope_one_side_and_bad_positions():
    x = torch.randn((4, 2, 128), device="cuda").half()
    w = torch.ones(128, device="cuda").half()
    cs = torch.rand((10, 128), device="cuda")
    o = torch.empty_like(x)
    qk_norm_rope(None, x, None, w, cs, ints([0, 10, -1, 9]), None, o)
    assert torch.isnan(o[1]).all() and torch.isnan(o[2]).all() and torch.isfinite(o[0]).all() and torch.isfinite(o[3]).all()
    o2 = torch.empty_like(x)
    qk_norm_rope(x, None, w, None, cs, ints([0, 1, 1, 9]), o2)
    assert torch.equal(o2[0], o[0]) and torch.equal(o2[3], o[3])
    e = torch.empty((0, 2, 128), dtype=torch.float16, device="cuda")
    qk_norm_rope(e, None, w, None, cs, ints([]))


# ------------------------------------------------------------------------------------------------ together
@pytest.mark.parametrize("fmt,dtype", [(("bf16", "bf16"), "bf16"), (("q8_0", "q4_0"), "f16")])
def test_prompt_then_steps(fmt, dtype):
    """A prompt in two chunks and then single tokens, each through the norm and rotation, the write and the
    attention, against 64-bit attention over the rows read back."""
    H, G, D, ps, rot = 2, 3, 128, 16, 64
    Hq = H * G
    p = Pages(H, D, ps, 40, *fmt, Hq=Hq, max_seqs=2, max_tokens=400)
    g = torch.Generator(device="cuda").manual_seed(0)
    table = ints(np.random.default_rng(0).permutation(40)[:34].reshape(2, 17))
    ang = torch.rand((300, rot // 2), generator=g, device="cuda")
    cs = torch.cat((ang.cos(), ang.sin()), 1)
    wq, wk = torch.ones((2, D), device="cuda").to(DT[dtype])
    held = [0, 0]
    for chunk in ([130, 7], [20, 90], [1, 1], [1, 1]):
        T = sum(chunk)
        x = torch.randn((T, Hq + 2 * H, D), generator=g, device="cuda").to(DT[dtype])
        q, k, v = x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:]
        pos = np.concatenate([np.arange(h, h + c) for h, c in zip(held, chunk)])
        seq = np.repeat([0, 1], chunk)
        slots = table.cpu().numpy()[seq, pos // ps] * ps + pos % ps
        qk_norm_rope(q, k, wq, wk, cs, ints(pos), stream=stream())
        p.cache.write(0, k, v, ints(slots), stream=stream())
        held = [h + c for h, c in zip(held, chunk)]
        out, lse = torch.empty((T, Hq, D), dtype=DT[dtype], device="cuda"), torch.empty((T, Hq), device="cuda")
        if T == 2:
            p.cache.decode_attn(0, q, table, ints(held), out, lse=lse, stream=stream())
        else:
            p.cache.prefill_attn(0, q, ints([0, chunk[0], T]), max(chunk), table, ints(held), out, lse=lse, stream=stream())
        rows = [torch.empty((sum(held), H, D), device="cuda") for _ in range(2)]
        p.cache.read(0, table, ints([0, held[0], sum(held)]), *rows, stream=stream())
        kk, vv = (r.half().double() if fmt[0][0] == "q" else r.double() for r in rows)
        for b in range(2):
            r = slice(b * chunk[0], chunk[0] + b * chunk[1])
            c = slice(b * held[0], held[0] + b * held[1])
            want = pc.attention64(q[r].double(), kk[c], vv[c], torch.arange(held[b] - chunk[b], held[b], device="cuda"),
                                  1 / math.sqrt(D))
            pc.check_attention(out[r], lse[r], want, dtype, HALF_ULP["bf16" if dtype == "bf16" else "f16"], steps_of(held[b]))
    assert p.cache.status() == 0


def test_captured_step_follows_lengths_and_slots():
    """A decode step captured once (norm and rotation, write, attention) and replayed with other tokens."""
    H, G, D, ps = 2, 4, 128, 16
    a, b = (Pages(H, D, ps, 60, "f16", "f16", Hq=H * G, max_seqs=3, seed=9) for _ in range(2))
    lens0 = [5, 300, 31]
    for p in (a, b):
        table, _, _ = pc.fill(p, 0, lens0, 4, spare=2)
    spare = [x for x in range(60) if x not in set(table.flatten().tolist())]
    tab = table.cpu().numpy()
    for r in range(3):
        for c in range(tab.shape[1]):
            if tab[r, c] < 0:
                tab[r, c] = spare.pop()
                break
    table = ints(tab)
    lens, slots, pos = ints([0] * 3), ints([0] * 3), ints([0] * 3)
    x = torch.zeros((3, H * G + 2 * H, D), dtype=torch.float16, device="cuda")
    q, k, v = x[:, :H * G], x[:, H * G:H * G + H], x[:, H * G + H:]
    w = torch.ones(D, device="cuda").half()
    cs = torch.rand((400, D), device="cuda")
    out = torch.empty((3, H * G, D), dtype=torch.float16, device="cuda")

    def step(p, o):
        qk_norm_rope(q, k, w, w, cs, pos, stream=stream())
        p.cache.write(0, k, v, slots, stream=stream())
        p.cache.decode_attn(0, q, table, lens, o, stream=stream())

    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        step(a, out)
        side.synchronize()
        with torch.cuda.graph(g, stream=side):
            step(a, out)
    for p in (a, b):
        pc.fill(p, 0, lens0, 4, spare=2)
    for s in range(4):
        n = [l + s + 1 for l in lens0]
        x0 = torch.randn(x.shape, generator=torch.Generator().manual_seed(s)).half().cuda()
        lens.copy_(ints(n))
        pos.copy_(lens - 1)
        slots.copy_(ints([int(tab[i, (n[i] - 1) // ps]) * ps + (n[i] - 1) % ps for i in range(3)]))
        x.copy_(x0)
        g.replay()
        torch.cuda.synchronize()
        x.copy_(x0)
        want = torch.empty_like(out)
        step(b, want)
        assert torch.equal(out, want)


def test_captured_chunk_follows_its_offsets():
    """A chunk's attention captured once and replayed with other chunk bounds, lengths and queries."""
    for fmt, dtype in ((("bf16", "bf16"), "bf16"), (("q8_0", "q8_0"), "f16")):
        p = Pages(2, 128, 32, 40, *fmt, Hq=6, max_seqs=2, max_tokens=300, seed=3)
        table, _, _ = pc.fill(p, 0, [600, 333], 4, dtype)
        cu, lens = ints([0, 100, 300]), ints([600, 333])
        q = torch.randn((300, 6, 128), generator=torch.Generator().manual_seed(0)).to(DT[dtype]).cuda()
        out, lse = torch.empty_like(q), torch.empty((300, 6), device="cuda")
        g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.stream(side):
            p.cache.prefill_attn(0, q, cu, 300, table, lens, out, lse=lse, stream=stream())
            side.synchronize()
            with torch.cuda.graph(g, stream=side):
                p.cache.prefill_attn(0, q, cu, 300, table, lens, out, lse=lse, stream=stream())
        for i, (c, n) in enumerate((([0, 100, 300], [600, 333]), ([0, 299, 300], [299, 20]), ([0, 0, 7], [600, 7]))):
            cu.copy_(ints(c))
            lens.copy_(ints(n))
            q.copy_(torch.randn(q.shape, generator=torch.Generator().manual_seed(i)).to(DT[dtype]).cuda())
            g.replay()
            want, want_lse = torch.empty_like(q), torch.empty_like(lse)
            p.cache.prefill_attn(0, q, cu, 300, table, lens, want, lse=want_lse)
            torch.cuda.synchronize()
            assert torch.equal(out[:c[2]], want[:c[2]]) and torch.equal(lse[:c[2]], want_lse[:c[2]])


def test_two_streams_with_workspaces_of_their_own():
    p, table, q, out, _ = decode_case(("f16", "f16"), "f16", 2, 4, 128, 32, [3000, 20, 700], {})
    lens = ints([3000, 20, 700])
    streams, outs, ws = [torch.cuda.Stream() for _ in range(2)], [torch.empty_like(out) for _ in range(8)], []
    torch.cuda.synchronize()
    for s in streams:
        ws.append(p.cache.new_workspace())
    for i in range(8):
        with torch.cuda.stream(streams[i % 2]):
            p.cache.decode_attn(0, q, table, lens, outs[i], ws=ws[i % 2], stream=stream())
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, out)


def test_layers_share_the_table():
    p = Pages(2, 64, 16, 6, "q8_0", "q8_0", Hq=4, layers=3)
    got = []
    for layer in range(3):
        table, ks, vs = pc.fill(p, layer, [40, 21], 7 + layer // 2)
        q = torch.randn((2, 4, 64), generator=torch.Generator().manual_seed(0)).half().cuda()
        out = torch.empty_like(q)
        p.cache.decode_attn(layer, q, table, ints([40, 21]), out)
        want = pc.attention64(q[:1].double(), ks[0], vs[0], torch.tensor([39], device="cuda"), 1 / 8)
        pc.check_attention(out[:1], None, want, "f16", HALF_ULP["f16"], steps_of(40))
        got.append(out)
    assert torch.equal(got[0], got[1]) and not torch.equal(got[0], got[2])


# ------------------------------------------------------------------------------------------------ refusals
def test_refusals():
    p = Pages(2, 128, 16, 4, "f16", "f16", Hq=8, max_seqs=2, max_tokens=8)
    c, cu = p.cache, "cuda"
    q = torch.zeros((2, 8, 128), dtype=torch.float16, device=cu)
    out, table, lens = torch.empty_like(q), ints([[0, 1], [2, 3]]), ints([5, 6])
    kv = torch.zeros((2, 2, 128), dtype=torch.float16, device=cu)
    bad = [
        lambda: c.write(0, kv, kv[:1], ints([0, 1])),
        lambda: c.write(0, kv, kv.bfloat16(), ints([0, 1])),
        lambda: c.write(0, kv.float(), kv.float(), ints([0, 1])),
        lambda: c.write(0, kv, kv, ints([0, 1]).long()),
        lambda: c.write(0, kv, kv, torch.zeros(2, dtype=torch.int32)),
        lambda: c.write(0, kv.cpu(), kv.cpu(), ints([0, 1])),
        lambda: c.write(0, kv.transpose(1, 2), kv.transpose(1, 2), ints([0, 1])),
        lambda: c.read(0, table, ints([0, 1, 2])),
        lambda: c.read(0, table, ints([0, 1]), kv),
        lambda: c.read(0, table, ints([0, 1, 2]), kv, kv.float()),
        lambda: c.read(0, table.t(), ints([0, 1, 2]), kv),
        lambda: c.decode_attn(0, q[:1], table, lens, out[:1]),
        lambda: c.decode_attn(0, q, table, lens[:1], out),
        lambda: c.decode_attn(0, q, table, lens, out[:1]),
        lambda: c.decode_attn(0, q, table, lens, out.bfloat16()),
        lambda: c.decode_attn(0, q, table, lens, out, slopes=torch.zeros(4, device=cu)),
        lambda: c.decode_attn(0, q, table, lens, out, prefix=ints([1])),
        lambda: c.decode_attn(0, q, table, lens, out, lse=torch.zeros((2, 8), dtype=torch.float16, device=cu)),
        lambda: c.prefill_attn(0, q, ints([0, 2]), 2, table, lens, out),
        lambda: qk_norm_rope(q, kv.bfloat16(), None, None, None, None),
        lambda: qk_norm_rope(q, kv[:1], None, None, None, None),
        lambda: qk_norm_rope(q, kv, torch.ones(64, device=cu).half(), None, None, None),
        lambda: qk_norm_rope(q, kv, None, None, torch.zeros((4, 128), device=cu), None),
        lambda: PagedKVCache(p.cfg, 0, pool=torch.zeros(100, dtype=torch.uint8, device=cu)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was not refused")
    codes = [
        (1, lambda: c.write(1, kv, kv, ints([0, 1]))),
        (1, lambda: c.decode_attn(-1, q, table, lens, out)),
        (1, lambda: c.decode_attn(0, q, table, lens, out, softcap=-1.0)),
        (1, lambda: c.decode_attn(0, q, table, lens, out, softcap=float("inf"))),
        (1, lambda: c.decode_attn(0, q, table, lens, out, softcap=1e-38)),
        (1, lambda: c.decode_attn(0, q, table, lens, out, window=-1)),
        (3, lambda: _lib.kv_paged_prefill_attn(c.h, 0, _lib.F16, 2, 1 << 27, 8, q.data_ptr(), 1024, ints([0, 1, 2]).data_ptr(),
                                               table.data_ptr(), 2, 2, lens.data_ptr(), out.data_ptr(), None, c.ws.data_ptr(),
                                               c.ws_bytes)),
        (3, lambda: _lib.kv_paged_prefill_attn(c.h, 0, _lib.F16, 2, 1 << 26, 1 << 20, q.data_ptr(), 1024,
                                               ints([0, 1, 2]).data_ptr(), table.data_ptr(), 2, 2, lens.data_ptr(), out.data_ptr(),
                                               None, c.ws.data_ptr(), c.ws_bytes)),
        (1, lambda: c.decode_attn(0, q, table, lens, out, ws=torch.empty(16, dtype=torch.uint8, device=cu))),
        (3, lambda: c.decode_attn(0, q.bfloat16(), table, lens, out.bfloat16())),
        (1, lambda: c.prefill_attn(0, q, ints([0, 1, 2]), -1, table, lens, out)),
        (1, lambda: c.write(0, torch.zeros(260 * 2, device=cu).half().as_strided((2, 2, 128), (260, 128, 1)), kv, ints([0, 1]))),
        (1, lambda: c.write(0, torch.zeros(600, device=cu).half()[1:513].view(2, 2, 128), kv, ints([0, 1]))),
        (1, lambda: qk_norm_rope(q, kv, None, None, torch.zeros((4, 24), device=cu), ints([0, 1]))),
    ]
    for code, f in codes:
        with pytest.raises(KVQError) as e:
            f()
        assert e.value.code == code
    assert c.status() == 0
