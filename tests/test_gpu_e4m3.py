"""e4m3 pages on the GPU: what an append leaves byte for byte, rows read back, decode and chunk attention against 64 bits."""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import e4m3_cases as e8                                                                  # noqa: E402
import paged_cases as pc                                                                 # noqa: E402
from e4m3_cases import DT, Pages8                                                        # noqa: E402
from quantized_kv_cache_gb300 import KVQError, PagedKVCache, _lib, paged_config          # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def stream():
    return torch.cuda.current_stream().cuda_stream


def cu_of(n, first=0):
    return ints([first] + [first + int(x) for x in np.cumsum(n)])


def steps_of(n):
    return n / 16 + 64


# ------------------------------------------------------------------------------------------------ append
def append_and_check(p, layer, table, start, n, k, v, first=0):
    """One append, and the pool against the reference byte for byte (the status area apart)."""
    want = p.host()
    p.cache.append(layer, k, v, ints(table), cu_of(n, first), ints(start), stream=stream())
    torch.cuda.synchronize()
    for w, x in enumerate((k, v)):
        x = x.double().cpu().numpy()
        at = first
        for b, c in enumerate(n):
            p.append(want, layer, w, table[b], start[b], x[at:at + c])
            at += c
    got = p.host()
    assert np.array_equal(got[256:], want[256:])


def values(T, H, D, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = scale * torch.randn((T, 2 * H + 1, D), generator=g)
    x[:, :, ::32] *= 6
    if T > 3:
        x[1] = 0.0
        x[2] *= 1e-5
        x[3, :, ::2] = 0.5
    return x.to(DT[dtype]).cuda()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("H,D,ps", [(1, 64, 16), (3, 128, 32), (2, 256, 256), (5, 64, 128), (1, 128, 64)])
def test_append_leaves_the_reference_bytes(dtype, H, D, ps):
    """Ragged sequences grown by ragged pieces: some begin inside a block, one brings nothing, scales grow and stay."""
    lens_at = [[0, 0, 0, 0], [ps + 5, 3, 0, 33], [ps + 6, 3, 40, 34], [2 * ps + 1, 50, 41, 35], [2 * ps + 40, 51, 48, 36]]
    p = Pages8(H, D, ps, 30, layers=2)
    table = e8.table_of(p, [2 * ps + 40, 51, 48, 36], 1)
    for s in range(1, len(lens_at)):
        start, n = lens_at[s - 1], [b - a for a, b in zip(lens_at[s - 1], lens_at[s])]
        T = sum(n) + 5
        x = values(T, H, D, dtype, s, 3.0 ** s if s % 2 else 0.1)
        append_and_check(p, 1, table, start, n, x[:, :H], x[:, H:2 * H], first=2)
    assert p.cache.status() == 0


def test_append_single_tokens_of_many_sequences():
    """Decode steps: 70 and 1,500 sequences of one token each, and one token of a single sequence."""
    for n_seq in (1, 70, 1500):
        p = Pages8(2, 64, 16, 2 * n_seq + 2)
        lens = [1 + (7 * b) % 30 for b in range(n_seq)]
        table = e8.table_of(p, [n + 2 for n in lens], 3)
        kv = values(sum(lens), 2, 64, "f16", 5)
        append_and_check(p, 0, table, [0] * n_seq, lens, kv[:, :2], kv[:, 2:4])
        for s in range(2):
            x = values(n_seq, 2, 64, "f16", 6 + s, 1.0 + 3 * s)
            append_and_check(p, 0, table, [n + s for n in lens], [1] * n_seq, x[:, :2], x[:, 2:4])
        assert p.cache.status() == 0


def test_append_written_again():
    """Positions written a second time: the block's scale does not shrink, the rows before them stay; from a block's first
    position on it begins anew."""
    p = Pages8(2, 128, 32, 4)
    table = e8.table_of(p, [60], 2)
    big, small = values(40, 2, 128, "bf16", 1, 100.0), values(40, 2, 128, "bf16", 2, 0.01)
    append_and_check(p, 0, table, [0], [40], big[:, :2], big[:, 2:4])
    append_and_check(p, 0, table, [35], [9], small[:9, :2], small[:9, 2:4])
    append_and_check(p, 0, table, [32], [3], small[:3, :2], small[:3, 2:4])
    append_and_check(p, 0, table, [16], [16], small[:16, :2], small[:16, 2:4])


def test_append_of_extreme_values():
    p = Pages8(1, 64, 16, 8)
    table = e8.table_of(p, [100], 2)
    x = torch.randn((48, 1, 64), generator=torch.Generator().manual_seed(0)).bfloat16().cuda()
    x[0:8] *= 1e-39                                                # subnormal numbers
    x[16:32] *= 1e-30
    append_and_check(p, 0, table, [0], [48], x, x)
    assert p.cache.status() == 0
    x[5, 0, 3] = 3.3e38                                            # a jump of the scale that leaves nothing of the others
    append_and_check(p, 0, table, [3], [40], x[3:43], x[3:43])
    assert p.cache.status() == _lib.PAGED_RANGE
    x = torch.randn((20, 1, 64), generator=torch.Generator().manual_seed(1)).half().cuda()
    x[2, 0, 5], x[2, 0, 6], x[17, 0, 63] = float("inf"), float("nan"), -float("inf")
    want = p.host()
    p.cache.append(0, x, x, ints(table), ints([0, 20]))
    assert p.cache.status() == _lib.PAGED_NONFINITE
    p.append(want, 0, 0, table[0], 0, x.double().cpu().numpy())
    got, codes = p.host(), p.unit(want, 0, 0, int(table[0, 0]), 0)[0]
    for page in range(2):
        a, b = (p.unit(r, 0, 0, int(table[0, page]), 0) for r in (got, want))
        nan = np.isnan(e8.VALUES[b[0]])
        assert np.array_equal(np.isnan(e8.VALUES[a[0]]), nan) and np.array_equal(a[0][~nan], b[0][~nan]) and np.array_equal(a[1], b[1])
    assert np.isnan(e8.VALUES[codes[2, 5:7]]).all() and np.isfinite(e8.VALUES[codes[2, 7:]]).all()
    x = torch.full((1, 1, 64), float("nan"), dtype=torch.float16, device="cuda")        # a block of nothing else
    p.cache.append(0, x, x, ints(table), ints([0, 1]), ints([64]))
    assert p.cache.status() == _lib.PAGED_NONFINITE
    out = torch.zeros((1, 1, 64), device="cuda")
    p.cache.read(0, ints(table), ints([0, 1]), out, start=ints([64]))
    assert torch.isnan(out).all()


def test_append_reports_bad_pages_and_lengths():
    p = Pages8(2, 64, 16, 6)
    x = values(40, 2, 64, "f16", 1)
    k, v = x[:, :2], x[:, 2:4]
    before = p.host()

    def unchanged(pages=()):
        got = p.host()
        keep = [i for i in range(6) if i not in pages]
        return all(np.array_equal(np.concatenate(list(map(np.ravel, p.unit(got, 0, w, i, h)))),
                                  np.concatenate(list(map(np.ravel, p.unit(before, 0, w, i, h))))) or
                   np.isnan(p.unit(before, 0, w, i, h)[1]).any() for w in range(2) for i in keep for h in range(2))

    p.cache.append(0, k[:16], v[:16], ints([[6, 1]]), ints([0, 16]))
    assert p.cache.status() == _lib.PAGED_BAD_INDEX and unchanged()
    p.cache.append(0, k[:16], v[:16], ints([[-1, 1]]), ints([0, 16]))
    assert p.cache.status() == _lib.PAGED_BAD_INDEX and unchanged()
    p.cache.append(0, k[:16], v[:16], ints([[0, 1]]), ints([0, 16]), ints([32]))         # behind the table's last page
    assert p.cache.status() == _lib.PAGED_BAD_LENGTH and unchanged()
    p.cache.append(0, k[:16], v[:16], ints([[0, 1]]), ints([0, 16]), ints([-16]))
    assert p.cache.status() == _lib.PAGED_BAD_LENGTH and unchanged()
    p.cache.append(0, k[:16], v[:16], ints([[0, 1]]), ints([0, 16]), ints([2147483647]))
    assert p.cache.status() == _lib.PAGED_BAD_LENGTH and unchanged()
    p.cache.append(0, k[:16], v[:16], ints([[2, 3]]), ints([0, 40]))                      # more rows than there are
    assert p.cache.status() == _lib.PAGED_BAD_LENGTH and unchanged((2,))
    p.cache.append(0, k[:16], v[:16], ints([[2, 3]]), ints([-5, 40]))
    assert p.cache.status() == _lib.PAGED_BAD_LENGTH and unchanged((2,))
    p.cache.append(0, k[:0], v[:0], ints([[2, 3]]), ints([0, 0]))
    assert p.cache.status() == 0


@pytest.mark.parametrize("out", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("H,D,ps", [(2, 64, 16), (3, 128, 64), (1, 256, 128)])
def test_read_gives_the_stored_values(out, H, D, ps):
    p = Pages8(H, D, ps, 9)
    lens = [2 * ps + 1, 0, ps, 5]
    table, _, _ = e8.fill(p, 0, lens, 3, scale=0.3)
    raw, tab = p.host(), table.cpu().numpy()
    start, n = [1, 0, ps - 1, 0], [2 * ps, 0, 1, 5]
    cu = cu_of(n, 2)
    rows = 2 + sum(n) + 3
    outs = [torch.full((rows, H, D), 7.0, dtype=DT[out], device="cuda") for _ in range(2)]
    p.cache.read(0, table, cu, outs[0], outs[1], start=ints(start))
    for w in range(2):
        want = torch.full((rows, H, D), 7.0, dtype=torch.float64)
        for b in range(4):
            x = p.rows(raw, 0, w, tab[b], lens[b])[start[b]:start[b] + n[b]]
            want[int(cu[b]):int(cu[b]) + n[b]] = torch.from_numpy(x)
        assert torch.equal(outs[w].cpu(), want.to(DT[out]))
    assert p.cache.status() == 0


# ------------------------------------------------------------------------------------------------ decode
OPTS = [{}, dict(softcap=2.0), dict(window=40), dict(prefix=9, window=21), dict(slopes=True), dict(softcap=30.0, slopes=True, window=100, prefix=3)]


def options(opts, Hq, n_seq):
    o = dict(opts)
    if "prefix" in o:
        o["prefix"] = ints([o["prefix"]] * n_seq)
    if "slopes" in o:
        o["slopes"] = torch.exp2(-torch.arange(1, Hq + 1, device="cuda", dtype=torch.float32) / 2)
    return o


def compare(p, table, ks, vs, lens, qlens, q, out, lse, opts, dtype, first=0):
    at = first
    for b, n in enumerate(lens):
        r = slice(at, at + qlens[b])
        at += qlens[b]
        pre = int(opts["prefix"][b]) if "prefix" in opts else 0
        want = pc.attention64(q[r].double(), ks[b], vs[b], torch.arange(n - qlens[b], n, device="cuda"), 1 / math.sqrt(p.D),
                              opts.get("softcap", 0.0), opts.get("window", 0), opts.get("slopes"), pre)
        pc.check_attention(out[r], lse[r], want, dtype, 2.0 ** -11, steps_of(n))


def decode_case(dtype, H, G, D, ps, lens, opts, seed=0, q_scale=1.0, scale=1.0):
    p = Pages8(H, D, ps, sum(-(-n // ps) for n in lens) + 1, Hq=H * G, max_seqs=len(lens), seed=seed)
    table, ks, vs = e8.fill(p, 0, lens, seed, dtype, scale)
    wide = torch.randn((len(lens), H * G + 2 * H, D), generator=torch.Generator(device="cuda").manual_seed(seed + 1), device="cuda")
    q = (q_scale * wide).to(DT[dtype])[:, :H * G]
    out = torch.full((len(lens), H * G, D), float("nan"), dtype=DT[dtype], device="cuda")
    lse = torch.full((len(lens), H * G), float("nan"), device="cuda")
    opts = options(opts, H * G, len(lens))
    p.cache.decode_attn(0, q, table, ints(lens), out, lse=lse, stream=stream(), **opts)
    torch.cuda.synchronize()
    assert p.cache.status() == 0
    compare(p, table, ks, vs, lens, [1] * len(lens), q, out, lse, opts, dtype)
    return p, table, q, out


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("H,G,D,ps", [(2, 2, 64, 16), (8, 5, 128, 32), (4, 6, 256, 64), (2, 16, 128, 16), (1, 9, 64, 128),
                                      (1, 16, 256, 256), (3, 1, 128, 64), (1, 8, 256, 16)])
def test_decode_matches_64_bits(dtype, H, G, D, ps):
    decode_case(dtype, H, G, D, ps, [1, 16, 17, 300, 15, 2, 1025], {})


@pytest.mark.parametrize("opts", OPTS[1:])
@pytest.mark.parametrize("dtype,D,G", [("f16", 128, 4), ("bf16", 64, 12), ("bf16", 256, 3)])
def test_decode_options(opts, dtype, D, G):
    decode_case(dtype, 2, G, D, 32, [200, 1, 47, 1500], opts)


def test_decode_long_ragged_and_sharp():
    decode_case("f16", 8, 5, 128, 64, [20000, 3, 0, 7777], {})
    decode_case("bf16", 2, 8, 128, 16, [3000, 100], {}, q_scale=20.0)
    decode_case("bf16", 2, 8, 64, 16, [300, 100], {}, q_scale=1e-9)
    decode_case("f16", 1, 2, 256, 16, [70] * 200, {})                     # more heads than CTAs have runs


@pytest.mark.parametrize("scale", [1e-6, 1e-4, 500.0, 2000.0])
def test_scales_far_from_one(scale):
    """Rows down to fp16's subnormal numbers and up to its largest: the values are those that the pages hold."""
    dtype = "bf16" if scale < 1 else "f16"
    decode_case(dtype, 2, 4, 128, 32, [200, 33], {}, scale=scale, q_scale=min(1.0, 1.0 / scale))
    chunk_case(dtype, 2, 4, 128, 32, [200, 33], [50, 33], {}, scale=scale, q_scale=min(1.0, 1.0 / scale))


def test_unused_rows_and_pages_do_not_reach_the_outputs():
    """NaN codes behind the last position, before the window and in other pages: the outputs are those without them."""
    for chunk in (False, True):
        p = Pages8(2, 128, 32, 12, Hq=8, max_seqs=2, max_tokens=64)
        lens = [75, 20]
        table, ks, vs = e8.fill(p, 0, lens, 3)
        raw, tab = p.host(), table.cpu().numpy()
        used = {(int(tab[b, i // 32]), i % 32) for b, n in enumerate(lens) for i in range(n) if i >= n - 30}
        for w in range(2):
            for page in range(12):
                for h in range(2):
                    codes, _ = p.unit(raw, 0, w, page, h)
                    for r in range(32):
                        if (page, r) not in used:
                            codes[r] = 127 + 128 * (r & 1)
        p.pool.copy_(torch.from_numpy(raw))
        n = [9, 5] if chunk else [1, 1]
        q = torch.randn((sum(n), 8, 128), generator=torch.Generator().manual_seed(1)).half().cuda()
        out, lse = torch.empty_like(q), torch.empty((sum(n), 8), device="cuda")
        window = 20
        if chunk:
            p.cache.prefill_attn(0, q, cu_of(n), 9, table, ints(lens), out, lse=lse, window=window)
        else:
            p.cache.decode_attn(0, q, table, ints(lens), out, lse=lse, window=window)
        compare(p, table, ks, vs, lens, n, q, out, lse, dict(window=window), "f16")


def test_blocks_beyond_fp16_are_cut_and_stay_finite():
    p = Pages8(1, 64, 16, 4, Hq=2, max_seqs=1, max_tokens=32)
    x = torch.randn((20, 1, 64), generator=torch.Generator().manual_seed(0)).bfloat16().cuda()
    x[3] *= 1e9
    p.cache.append(0, x, x, ints([[0, 1]]), ints([0, 20]))
    assert p.cache.status() == _lib.PAGED_RANGE
    raw = p.host()
    for w in range(2):
        _, powers = p.unit(raw, 0, w, 0, 0)
        assert powers[0] > 128
        powers[0] = 128                                                # what the attentions take it as
    k, v = (e8.taken(p.rows(raw, 0, w, [0, 1], 20)) for w in range(2))
    q = (1e-6 * torch.randn((20, 2, 64), generator=torch.Generator().manual_seed(1))).bfloat16().cuda()
    out, lse = torch.empty_like(q), torch.empty((20, 2), device="cuda")
    p.cache.prefill_attn(0, q, ints([0, 20]), 20, ints([[0, 1]]), ints([20]), out, lse=lse)
    compare(p, None, [k], [v], [20], [20], q, out, lse, {}, "bf16")
    p.cache.decode_attn(0, q[19:], ints([[0, 1]]), ints([20]), out[19:], lse=lse[19:])
    compare(p, None, [k], [v], [20], [1], q[19:], out[19:], lse[19:], {}, "bf16")


def test_nan_codes_that_a_query_sees_give_nan():
    p = Pages8(1, 64, 16, 4, Hq=2, max_seqs=1, max_tokens=64)
    x = torch.randn((40, 1, 64), generator=torch.Generator().manual_seed(0)).half().cuda()
    x[20, 0, 7] = float("nan")
    p.cache.append(0, x, x, ints([[0, 1, 2]]), ints([0, 40]))
    assert p.cache.status() == _lib.PAGED_NONFINITE
    q = torch.randn((40, 2, 64), generator=torch.Generator().manual_seed(1)).half().cuda()
    out, lse = torch.empty_like(q), torch.empty((40, 2), device="cuda")
    p.cache.prefill_attn(0, q, ints([0, 40]), 40, ints([[0, 1, 2]]), ints([40]), out, lse=lse)
    assert torch.isfinite(out[:20]).all() and torch.isfinite(lse[:20]).all()
    assert torch.isnan(out[20:]).all() and torch.isnan(lse[20:]).all()
    p.cache.decode_attn(0, q[:1], ints([[0, 1, 2]]), ints([40]), out[:1], lse=lse[:1])
    assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all()
    p.cache.decode_attn(0, q[:1], ints([[0, 1, 2]]), ints([20]), out[:1], lse=lse[:1])
    assert torch.isfinite(out[0]).all() and torch.isfinite(lse[0]).all()


# ------------------------------------------------------------------------------------------------ chunk
def wide(H, ps, n_seq):
    """Table entries behind the pages, so that a chunk of few rows goes where few rows go (by what the table could hold)."""
    return 1100000 // (H * ps * n_seq) + 1


def chunk_case(dtype, H, G, D, ps, lens, qlens, opts, seed=0, q_scale=1.0, scale=1.0, gap=3, spare=1):
    T = sum(qlens) + 2 * gap
    p = Pages8(H, D, ps, sum(-(-n // ps) for n in lens) + 1, Hq=H * G, max_seqs=len(lens), max_tokens=T, seed=seed)
    table, ks, vs = e8.fill(p, 0, lens, seed, dtype, scale, spare)
    wide = torch.randn((T, H * G + 2 * H, D), generator=torch.Generator(device="cuda").manual_seed(seed + 1), device="cuda")
    q = (q_scale * wide).to(DT[dtype])[:, :H * G]
    out = torch.full((T, H * G, D), 7.0, dtype=DT[dtype], device="cuda")
    lse = torch.full((T, H * G), 7.0, device="cuda")
    opts = options(opts, H * G, len(lens))
    p.cache.prefill_attn(0, q, cu_of(qlens, gap), max(qlens), table, ints(lens), out, lse=lse, stream=stream(), **opts)
    torch.cuda.synchronize()
    assert p.cache.status() == 0
    for x in (out, lse):
        assert (x[:gap] == 7).all() and (x[T - gap:] == 7).all()
    compare(p, table, ks, vs, lens, qlens, q, out, lse, opts, dtype, gap)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("H,G,D,ps", [(2, 2, 64, 16), (8, 5, 128, 32), (4, 6, 256, 64), (2, 16, 128, 16), (1, 9, 64, 128),
                                      (1, 3, 256, 256)])
def test_chunk_matches_64_bits(dtype, H, G, D, ps):
    chunk_case(dtype, H, G, D, ps, [1, 130, 300, 1025], [1, 130, 0, 77], {})


@pytest.mark.parametrize("opts", OPTS[1:])
@pytest.mark.parametrize("dtype,D,G", [("f16", 128, 4), ("bf16", 64, 12), ("bf16", 256, 3)])
def test_chunk_options(opts, dtype, D, G):
    chunk_case(dtype, 2, G, D, 32, [200, 1, 47, 1500], [150, 1, 47, 9], opts)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("cap,q_scale", [(30.0, 1.0), (50.0, 3.0), (30.0, 20.0), (1.0, 1e-3)])
def test_chunk_caps_near_and_far(D, cap, q_scale):
    chunk_case("bf16", 2, 4, D, 32, [900, 333], [200, 333], dict(softcap=cap), q_scale=q_scale)
    chunk_case("f16", 1, 3, D, 64, [600], [150], dict(softcap=cap), q_scale=q_scale)


def test_more_heads_than_runs():
    """Decode and few rows of 700 sequences: more heads than a launch has CTAs, the joins by runs."""
    lens = [1 + (37 * i) % 90 for i in range(700)]
    decode_case("f16", 2, 4, 128, 16, lens, {})
    chunk_case("bf16", 2, 4, 64, 16, [n + 3 for n in lens], [1 + i % 3 for i in range(700)], {}, spare=wide(2, 16, 700))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_chunk_of_drafted_tokens_and_split_positions(D):
    chunk_case("f16", 8, 5, D, 32, [3000, 700, 3, 5], [5, 5, 3, 1], {})
    chunk_case("bf16", 1, 4, D, 16, [6000], [40], dict(window=3000))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("H,G,D,ps,q", [(2, 2, 64, 16, 7), (8, 5, 128, 32, 5), (4, 6, 256, 64, 5), (2, 16, 128, 16, 4), (1, 9, 64, 128, 7),
                                        (1, 16, 256, 256, 4), (3, 1, 128, 64, 64), (2, 3, 256, 16, 21), (1, 5, 128, 16, 13)])
def test_few_rows_match_64_bits(dtype, H, G, D, ps, q):
    """Up to 64 rows a KV head, and one token more than that, over tables that hold little and much."""
    for spare in (1, wide(H, ps, 6)):
        chunk_case(dtype, H, G, D, ps, [q, 1, 1025, 17, 300, q + 1], [q, 1, q, 0, 2, q], {}, spare=spare)


@pytest.mark.parametrize("opts", OPTS[1:] + [dict(window=1), dict(prefix=60, window=3)])
@pytest.mark.parametrize("dtype,D,G", [("f16", 128, 4), ("bf16", 64, 12), ("bf16", 256, 3)])
def test_few_rows_options(opts, dtype, D, G):
    for spare in (1, wide(2, 32, 4)):
        chunk_case(dtype, 2, G, D, 32, [200, 1, 47, 1500], [5, 1, 4, 3], opts, spare=spare)


@pytest.mark.parametrize("much", [False, True])
def test_few_rows_of_many_sequences(much):
    """More groups than runs, and one sequence that all runs share; odd gaps of a batch padded with empty sequences."""
    many = [i % 4 for i in range(200)]
    chunk_case("f16", 4, 4, 128, 16, [3 + (11 * i) % 60 for i in range(200)], many, {}, gap=5, spare=wide(4, 16, 200) if much else 1)
    chunk_case("bf16", 1, 8, 128, 64, [40000], [8], {}, spare=wide(1, 64, 1) if much else 1)
    chunk_case("f16", 1, 4, 256, 64, [30001], [9], dict(slopes=True), spare=wide(1, 64, 1) if much else 1)


@pytest.mark.parametrize("much", [False, True])
@pytest.mark.parametrize("D,tokens", [(64, 6), (128, 6), (256, 3), (128, 40)])
def test_later_rows_do_not_reach_earlier_queries(D, tokens, much):
    """NaN in the keys and values of some of the chunk's own tokens: the rows before them stay within the bound, those from them on are NaN."""
    for at in ("k", "v"):
        n = 50 + tokens
        p = Pages8(2, D, 32, 8, Hq=8, max_seqs=1, max_tokens=tokens)
        table, ks, vs = e8.fill(p, 0, [n], 5, spare=wide(2, 32, 1) if much else 1)
        raw, j = p.host(), n - 2
        codes, _ = p.unit(raw, 0, 1 if at == "v" else 0, int(table[0, j // 32]), 1)
        codes[j % 32] = 127
        codes[j % 32, ::2] = 255
        p.pool.copy_(torch.from_numpy(raw))
        q = torch.randn((tokens, 8, D), generator=torch.Generator().manual_seed(1)).half().cuda()
        out, lse = torch.empty_like(q), torch.empty((tokens, 8), device="cuda")
        p.cache.prefill_attn(0, q, ints([0, tokens]), tokens, table, ints([n]), out, lse=lse)
        k = tokens - 2
        want = pc.attention64(q.double(), ks[0], vs[0], torch.arange(n - tokens, n, device="cuda"), 1 / math.sqrt(D))
        pc.check_attention(out[:k], lse[:k], tuple(x[:k] for x in want), "f16", 2.0 ** -11, steps_of(n))
        pc.check_attention(out[:, :4].contiguous(), lse[:, :4], tuple(x[:, :4] for x in want), "f16", 2.0 ** -11, steps_of(n))
        assert torch.isnan(out[k:, 4:]).all() and (torch.isnan(lse[k:, 4:]).all() if at == "k" else torch.isfinite(lse).all())


@pytest.mark.parametrize("much", [False, True])
def test_few_rows_at_negative_positions_and_bad_lengths(much):
    p = Pages8(1, 64, 16, 4, Hq=2, max_seqs=2, max_tokens=20)
    table, ks, vs = e8.fill(p, 0, [10, 30], 1, spare=wide(1, 16, 2) if much else 1)
    q = torch.randn((18, 2, 64), device="cuda").half()
    out, lse = torch.full_like(q, 7.0), torch.full((18, 2), 7.0, device="cuda")
    p.cache.prefill_attn(0, q, ints([0, 13, 15]), 13, table, ints([10, 30]), out, lse=lse, prefix=ints([4, 0]))
    assert not out[:3].any() and (lse[:3] == -math.inf).all() and (out[15:] == 7).all()
    want = pc.attention64(q[:13].double(), ks[0], vs[0], torch.arange(-3, 10, device="cuda"), 1 / 8, prefix=4)
    pc.check_attention(out[:13], lse[:13], want, "f16", 2.0 ** -11, steps_of(10))
    p.cache.prefill_attn(0, q, ints([0, 13, 15]), 13, table, ints([0, -1]), out, lse=lse)
    assert not out[:15].any() and (lse[:15] == -math.inf).all() and p.cache.status() == _lib.PAGED_BAD_LENGTH
    out.fill_(7.0)
    p.cache.prefill_attn(0, q, ints([0, 10, 15]), 2, table, ints([10, 30]), out, lse=lse)     # longer than max_q
    assert p.cache.status() == _lib.PAGED_BAD_LENGTH and (out[2:10] == 7).all() and (out[12:] == 7).all()
    want = pc.attention64(q[:2].double(), ks[0], vs[0], torch.arange(2, device="cuda"), 1 / 8)
    pc.check_attention(out[:2], lse[:2], want, "f16", 2.0 ** -11, steps_of(10))
    for cu in ([0, 13, 19], [-1, 3, 5], [0, 5, 3]):
        p.cache.prefill_attn(0, q, ints(cu), 13, table, ints([10, 30]), out, lse=lse)
        assert p.cache.status() == _lib.PAGED_BAD_LENGTH
    bad = table.clone()
    bad[1, 0] = 4
    p.cache.prefill_attn(0, q, ints([0, 5, 10]), 5, bad, ints([10, 30]), out, lse=lse)
    assert p.cache.status() == _lib.PAGED_BAD_INDEX


@pytest.mark.parametrize("much", [False, True])
def test_captured_drafts_follow_their_bounds(much):
    p = Pages8(2, 128, 32, 60, Hq=8, max_seqs=3, max_tokens=24, seed=3)
    table, _, _ = e8.fill(p, 0, [900, 333, 40], 4, spare=wide(2, 32, 3) if much else 1)
    cu, lens = ints([0, 5, 10, 15]), ints([900, 333, 40])
    q = torch.randn((15, 8, 128), generator=torch.Generator().manual_seed(0)).half().cuda()
    out, lse = torch.empty_like(q), torch.empty((15, 8), device="cuda")
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()

    def call(out, lse):
        p.cache.prefill_attn(0, q, cu, 8, table, lens, out, lse=lse, stream=stream())

    with torch.cuda.stream(side):
        call(out, lse)
        side.synchronize()
        with torch.cuda.graph(g, stream=side):
            call(out, lse)
    for i, (c, n) in enumerate((([0, 5, 10, 15], [900, 333, 40]), ([0, 0, 7, 15], [1, 50, 39]), ([0, 1, 2, 2], [800, 333, 40]))):
        cu.copy_(ints(c))
        lens.copy_(ints(n))
        q.copy_(torch.randn(q.shape, generator=torch.Generator().manual_seed(i)))
        g.replay()
        want, want_lse = torch.empty_like(out), torch.empty_like(lse)
        torch.cuda.synchronize()
        call(want, want_lse)
        assert torch.equal(out[:c[3]], want[:c[3]]) and torch.equal(lse[:c[3]], want_lse[:c[3]])


# ------------------------------------------------------------------------------------------------ together
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_prompt_then_steps(dtype):
    """Two pieces of a prompt, then single tokens: append and attention against 64 bits over what the pages then hold."""
    H, G, D, ps = 2, 3, 128, 16
    p = Pages8(H, D, ps, 40, Hq=H * G, max_seqs=2, max_tokens=400)
    table = ints(np.random.default_rng(0).permutation(40)[:34].reshape(2, 17))
    tab, held = table.cpu().numpy(), [0, 0]
    for s, piece in enumerate(([130, 7], [20, 90], [1, 1], [1, 1], [1, 1])):
        T = sum(piece)
        x = ((1.0 + s) * torch.randn((T, (G + 2) * H, D), generator=torch.Generator().manual_seed(s))).to(DT[dtype]).cuda()
        q, k, v = x[:, :H * G], x[:, H * G:H * G + H], x[:, H * G + H:]
        p.cache.append(0, k, v, table, cu_of(piece), ints(held), stream=stream())
        held = [a + b for a, b in zip(held, piece)]
        out, lse = torch.empty((T, H * G, D), dtype=DT[dtype], device="cuda"), torch.empty((T, H * G), device="cuda")
        if T == 2:
            p.cache.decode_attn(0, q, table, ints(held), out, lse=lse, stream=stream())
        else:
            p.cache.prefill_attn(0, q, cu_of(piece), max(piece), table, ints(held), out, lse=lse, stream=stream())
        raw = p.host()
        ks, vs = ([e8.taken(p.rows(raw, 0, w, tab[b], held[b])) for b in range(2)] for w in range(2))
        compare(p, table, ks, vs, held, piece, q, out, lse, {}, dtype)
    assert p.cache.status() == 0


def test_captured_step_follows_lengths():
    """Append and decode attention captured once, replayed with other tokens, starts and a sequence that sits out."""
    H, G, D, ps = 2, 4, 128, 16
    a, b = (Pages8(H, D, ps, 60, Hq=H * G, max_seqs=3, seed=9) for _ in range(2))
    tab = np.arange(60, dtype=np.int32).reshape(3, 20)
    table, cu, start, lens = ints(tab), ints([0, 1, 2, 3]), ints([0] * 3), ints([0] * 3)
    x = torch.zeros((3, (G + 2) * H, D), dtype=torch.float16, device="cuda")
    q, k, v = x[:, :H * G], x[:, H * G:H * G + H], x[:, H * G + H:]
    out = torch.zeros((3, H * G, D), dtype=torch.float16, device="cuda")

    def step(p, o):
        p.cache.append(0, k, v, table, cu, start, stream=stream())
        p.cache.decode_attn(0, q, table, lens, o, stream=stream())

    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        step(a, out)
        side.synchronize()
        with torch.cuda.graph(g, stream=side):
            step(a, out)
    b.pool[256:] = a.pool[256:]
    held = [0, 0, 0]
    for s in range(20):
        on = [1, 1, 0] if s % 3 else [1, 0, 1]
        x.copy_((1.0 + s) * torch.randn(x.shape, generator=torch.Generator().manual_seed(s)))
        cu.copy_(cu_of(on))
        start.copy_(ints(held))
        held = [m + n for m, n in zip(held, on)]
        lens.copy_(ints(held))
        g.replay()
        torch.cuda.synchronize()
        want = torch.zeros_like(out)
        step(b, want)
        assert torch.equal(out, want) and torch.equal(a.pool[256:], b.pool[256:])


def test_large_offsets():
    """Units beyond 2^31 bytes."""
    n_pages, ps, H, D = 6000, 256, 8, 256
    cfg = paged_config(1, H, D, 2 * H, ps, n_pages, "e4m3")
    c = PagedKVCache(cfg, 0, 1, 64)
    assert n_pages * H * ps * D > 1 << 31
    k, v = (torch.randn((300, H, D), generator=torch.Generator().manual_seed(i)).half().cuda() for i in range(2))
    table = ints([[5999, 5998]])
    c.append(0, k, v, table, ints([0, 300]))
    back = [torch.empty((300, H, D), device="cuda") for _ in range(2)]
    c.read(0, table, ints([0, 300]), *back)
    for x, y in zip(back, (k, v)):
        # a code is off by half a step of 2^-3 of its power of two at most, or half of 2^-9 of the block's
        assert ((x.double() - y.double()).abs() <= 2.0 ** -4 * y.double().abs() + 2.0 ** -10 * 2.0 ** -6).all()
    q = torch.randn((1, 2 * H, D), generator=torch.Generator().manual_seed(5)).half().cuda()
    out = torch.empty_like(q)
    want = pc.attention64(q.double(), back[0].double(), back[1].double(), torch.tensor([299], device="cuda"), 1 / 16)
    c.decode_attn(0, q, table, ints([300]), out)
    pc.check_attention(out, None, want, "f16", 2.0 ** -11, steps_of(300))
    out2 = torch.empty_like(q)
    c.prefill_attn(0, q, ints([0, 1]), 1, table, ints([300]), out2)
    pc.check_attention(out2, None, want, "f16", 2.0 ** -11, steps_of(300))
    assert c.status() == 0


# ------------------------------------------------------------------------------------------------ refusals
def test_refusals():
    p = Pages8(2, 128, 16, 4, Hq=8, max_seqs=2, max_tokens=8)
    c = p.cache
    kv, table = torch.zeros((2, 2, 128), dtype=torch.float16, device="cuda"), ints([[0, 1], [2, 3]])
    cu = ints([0, 1, 2])
    for i, f in enumerate([
            lambda: c.append(0, kv, kv[:1], table, cu),
            lambda: c.append(0, kv, kv.bfloat16(), table, cu),
            lambda: c.append(0, kv.float(), kv.float(), table, cu),
            lambda: c.append(0, kv.cpu(), kv.cpu(), table, cu),
            lambda: c.append(0, kv, kv, table, cu[:2]),
            lambda: c.append(0, kv, kv, table, cu.long()),
            lambda: c.append(0, kv, kv, table, cu, ints([0])),
            lambda: c.append(0, kv, kv, table.long(), cu),
            lambda: c.append(0, kv, kv, table.t(), cu),
            lambda: c.append(0, kv.transpose(1, 2), kv, table, cu),
            lambda: c.append(0, kv.clone().requires_grad_(), kv, table, cu)]):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was not refused")
    f16 = PagedKVCache(paged_config(1, 2, 128, 8, 16, 4, "f16"))
    for code, f in [(1, lambda: c.append(1, kv, kv, table, cu)), (3, lambda: c.write(0, kv, kv, ints([0, 1]))),
                    (3, lambda: f16.append(0, kv, kv, table, cu)),
                    (1, lambda: c.append(0, torch.zeros(600, device="cuda").half()[1:513].view(2, 2, 128), kv, table, cu)),
                    (1, lambda: c.append(0, torch.zeros(520, device="cuda").half().as_strided((2, 2, 128), (260, 128, 1)), kv, table, cu))]:
        with pytest.raises(KVQError) as e:
            f()
        assert e.value.code == code
    assert c.status() == 0
