"""Attention of whole packed prompts on the GPU against 64 bits, at the edges of what the call allows."""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import paged_cases as pc                                                                 # noqa: E402
from paged_cases import DT, HALF_ULP                                                     # noqa: E402
from quantized_kv_cache_gb300 import (KVQError, PagedKVCache, _lib, paged_config, prompt_attn, prompt_status,  # noqa: E402
                                      prompt_workspace)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def stream():
    return torch.cuda.current_stream().cuda_stream


def rows_of(T, Hq, H, D, dtype, seed, spare=0):
    """q, k, v as slices of one projection's output."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((T, Hq + 2 * H + spare, D), generator=g, device="cuda").to(DT[dtype])
    return x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:Hq + 2 * H]


def check(q, k, v, cu, lens, out, lse, opts, dtype, scale=None):
    for b, n in enumerate(lens):
        r = slice(cu[b], cu[b] + n)
        pre = int(opts["prefix"][b]) if "prefix" in opts else 0
        want = pc.attention64(q[r].double(), k[r].double(), v[r].double(), torch.arange(n, device="cuda"), scale or 1 / math.sqrt(q.shape[2]),
                              opts.get("softcap", 0.0), opts.get("window", 0), opts.get("slopes"), pre)
        pc.check_attention(out[r], lse[r], want, dtype, HALF_ULP[dtype], n / 16 + 64)


def case(dtype, H, G, D, lens, opts={}, q_scale=1.0, gap=3, seed=0, max_q=None):
    T = sum(lens) + 2 * gap
    q, k, v = rows_of(T, H * G, H, D, dtype, seed, 1)
    q.mul_(q_scale)
    cu = [gap] + [gap + int(x) for x in np.cumsum(lens)]
    out = torch.full((T, H * G, D), 7.0, dtype=DT[dtype], device="cuda")
    lse = torch.full((T, H * G), 7.0, device="cuda")
    opts = dict(opts)
    if "prefix" in opts:
        opts["prefix"] = ints([opts["prefix"]] * len(lens))
    if "slopes" in opts:
        opts["slopes"] = torch.exp2(-torch.arange(1, H * G + 1, device="cuda", dtype=torch.float32) / 2)
    ws = prompt_workspace(T, H * G, D)
    prompt_attn(q, k, v, ints(cu), max_q or max(lens), out, ws, lse=lse, stream=stream(), **opts)
    torch.cuda.synchronize()
    assert prompt_status(ws) == 0
    for x in (out, lse):
        assert (x[:gap] == 7).all() and (x[T - gap:] == 7).all()
    check(q, k, v, cu, lens, out, lse, opts, dtype)
    return q, k, v, cu, out, lse, ws


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("H,G,D", [(2, 2, 64), (8, 5, 128), (4, 6, 256), (2, 16, 128), (1, 9, 64), (1, 3, 256), (3, 1, 128)])
@pytest.mark.parametrize("lens", [[1], [2, 1, 0, 3], [127, 128, 129, 1, 257], [0, 700, 64, 0], [1300]])
def test_matches_64_bits(dtype, H, G, D, lens):
    case(dtype, H, G, D, lens)


@pytest.mark.parametrize("opts", [dict(softcap=2.0), dict(window=40), dict(prefix=9, window=21), dict(slopes=True), dict(window=1),
                                  dict(softcap=30.0, slopes=True, window=200, prefix=300)])
@pytest.mark.parametrize("dtype,D,G", [("f16", 128, 4), ("bf16", 64, 12), ("bf16", 256, 3)])
def test_options(opts, dtype, D, G):
    case(dtype, 2, G, D, [150, 1, 47, 600], opts)


def test_sharp_and_faint_scores():
    case("f16", 2, 4, 128, [300, 5], q_scale=20.0)
    case("bf16", 2, 4, 128, [300, 5], q_scale=1e4)
    case("bf16", 1, 2, 256, [130], q_scale=1e-6)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_positions_split(D):
    """One long prompt of a few rows a head: its positions are split and joined; odd counts of rows and heads."""
    case("bf16", 1, 1, D, [4099])
    case("f16", 1, 3, D, [2500, 7], dict(window=900, prefix=5))


def test_many_short_prompts():
    """More sequences than a warp looks at in one go, some empty."""
    lens = [(7 * i) % 23 for i in range(300)]
    case("f16", 2, 2, 64, lens)
    case("bf16", 1, 4, 128, lens, max_q=1000)


def test_later_rows_and_other_prompts_do_not_reach_earlier_queries():
    """NaN and infinities in later rows, in the next prompt and behind the last: the queries before them stay within the bound."""
    for dtype, D in (("f16", 128), ("bf16", 128), ("bf16", 256), ("f16", 64)):
        q, k, v = rows_of(260, 4, 2, D, dtype, 1)
        k, v = k.clone(), v.clone()
        lens, cu = [100, 90], [0, 100, 190]
        k[60], v[70], k[100:103], v[103:106], k[190:], v[190:] = (float(x) for x in ("nan", "inf", "inf", "nan", "nan", "inf"))
        out, lse, ws = torch.zeros_like(q, memory_format=torch.contiguous_format), torch.zeros((260, 4), device="cuda"), prompt_workspace(260, 4, D)
        prompt_attn(q, k, v, ints(cu), 100, out, ws, lse=lse)
        torch.cuda.synchronize()
        for r in (slice(0, 60),):
            want = pc.attention64(q[r].double(), k[r].double(), v[r].double(), torch.arange(60, device="cuda"), 1 / math.sqrt(D))
            pc.check_attention(out[r], lse[r], want, dtype, HALF_ULP[dtype], 70)
        assert torch.isnan(out[60:100]).all() and torch.isnan(out[100:190]).all()
        assert torch.isnan(lse[60:100]).all() and prompt_status(ws) == 0
        # the second prompt's own rows made good: nothing of the first or of what lies behind reaches it
        k[100:190], v[100:190] = torch.randn((2, 90, 2, D), generator=torch.Generator().manual_seed(0)).to(DT[dtype]).cuda()
        prompt_attn(q, k, v, ints(cu), 100, out, ws, lse=lse)
        r = slice(100, 190)
        want = pc.attention64(q[r].double(), k[r].double(), v[r].double(), torch.arange(90, device="cuda"), 1 / math.sqrt(D))
        pc.check_attention(out[r], lse[r], want, dtype, HALF_ULP[dtype], 70)


def test_prompts_longer_than_max_q_and_bad_bounds():
    q, k, v = rows_of(400, 6, 2, 128, "f16", 2)
    ws = prompt_workspace(400, 6, 128)
    out = torch.full((400, 6, 128), 7.0, dtype=torch.float16, device="cuda")
    lse = torch.full((400, 6), 7.0, device="cuda")
    prompt_attn(q, k, v, ints([0, 300, 400]), 120, out, ws, lse=lse)
    assert prompt_status(ws) == _lib.PAGED_BAD_LENGTH and prompt_status(ws) == 0
    check(q, k, v, [0, 300], [120, 100], out, lse, {}, "f16")
    assert (out[120:300] == 7).all() and (lse[120:300] == 7).all()
    for bad in ([0, 300, 401], [-1, 300, 400], [0, 300, 290]):
        out.fill_(7.0)
        prompt_attn(q, k, v, ints(bad), 400, out, ws, lse=lse)
        assert prompt_status(ws) == _lib.PAGED_BAD_LENGTH
        if bad[0] == 0:
            check(q, k, v, [0], [300], out, lse, {}, "f16")
            assert (out[300:] == 7).all()
        else:
            assert (out[:300] == 7).all()
    empty = q[:0]
    prompt_attn(empty, k[:0], v[:0], ints([0, 0]), 5, out[:0], ws)
    prompt_attn(q, k, v, ints([0]), 5, out, ws)
    assert prompt_status(ws) == 0


def test_softmax_scale_and_single_heads():
    q, k, v = rows_of(77, 1, 1, 64, "bf16", 3)
    q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    out, lse, ws = torch.empty_like(q), torch.empty((77, 1), device="cuda"), prompt_workspace(77, 1, 64)
    prompt_attn(q, k, v, ints([0, 77]), 77, out, ws, lse=lse, softmax_scale=0.3)
    check(q, k, v, [0], [77], out, lse, {}, "bf16", scale=float(np.float32(0.3)))


def test_captured_call_follows_its_bounds():
    q, k, v = (x.contiguous() for x in rows_of(500, 8, 2, 128, "bf16", 4))
    out, lse, cu, ws = torch.empty_like(q), torch.empty((500, 8), device="cuda"), ints([0, 200, 500]), prompt_workspace(500, 8, 128)
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        prompt_attn(q, k, v, cu, 500, out, ws, lse=lse, stream=stream())
        side.synchronize()
        with torch.cuda.graph(g, stream=side):
            prompt_attn(q, k, v, cu, 500, out, ws, lse=lse, stream=stream())
    for i, c in enumerate(([0, 200, 500], [0, 0, 500], [0, 499, 500], [0, 13, 130])):
        cu.copy_(ints(c))
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(i)))
        out.fill_(7.0)
        g.replay()
        want, want_lse = torch.full_like(out, 7.0), torch.empty_like(lse)
        other = prompt_workspace(500, 8, 128)
        prompt_attn(q, k, v, cu, 500, want, other, lse=want_lse)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse[:c[2]], want_lse[:c[2]])


def test_two_streams_with_workspaces_of_their_own():
    """A split call on two streams at once."""
    q, k, v = rows_of(3000, 2, 1, 128, "f16", 5)
    outs = [torch.empty((3000, 2, 128), dtype=torch.float16, device="cuda") for _ in range(6)]
    ws, streams = [prompt_workspace(3000, 2, 128) for _ in range(2)], [torch.cuda.Stream() for _ in range(2)]
    cu = ints([0, 3000])
    torch.cuda.synchronize()
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):
            prompt_attn(q, k, v, cu, 3000, outs[i], ws[i % 2], stream=stream())
    torch.cuda.synchronize()
    for o in outs[1:]:
        assert torch.equal(o, outs[0])
    assert prompt_status(ws[0]) == 0


@pytest.mark.parametrize("fmt,dtype", [("bf16", "bf16"), ("e4m3", "f16")])
def test_prompt_then_step_over_the_pages(fmt, dtype):
    """A prompt's attention from its own rows while they go to the pages, then a step over them."""
    H, G, D, ps, lens = 2, 4, 128, 32, [150, 31]
    c = PagedKVCache(paged_config(1, H, D, H * G, ps, 12, fmt), 0, 2, 256)
    table, cu = ints([[0, 3, 6, 9, 11, 1], [2, 4, 5, 7, 8, 10]]), ints([0, 150, 181])
    q, k, v = rows_of(181, H * G, H, D, dtype, 6)
    out, lse, ws = torch.empty((181, H * G, D), dtype=DT[dtype], device="cuda"), torch.empty((181, H * G), device="cuda"), prompt_workspace(181, H * G, D)
    tab = table.cpu().numpy()
    slots = [int(tab[b, i // ps]) * ps + i % ps for b, n in enumerate(lens) for i in range(n)]

    def store(k, v, bounds, start, slots):
        if fmt == "e4m3":
            c.append(0, k, v, table, ints(bounds), ints(start), stream=stream())
        else:
            c.write(0, k, v, ints(slots), stream=stream())

    prompt_attn(q, k, v, cu, 150, out, ws, lse=lse, stream=stream())
    store(k, v, [0, 150, 181], [0, 0], slots)
    check(q, k, v, [0, 150], lens, out, lse, {}, dtype)
    q1, k1, v1 = rows_of(2, H * G, H, D, dtype, 7)
    store(k1, v1, [0, 1, 2], lens, [int(tab[b, n // ps]) * ps + n % ps for b, n in enumerate(lens)])
    o1 = torch.empty((2, H * G, D), dtype=DT[dtype], device="cuda")
    c.decode_attn(0, q1, table, ints([n + 1 for n in lens]), o1, stream=stream())
    back = [torch.empty((183, H, D), device="cuda") for _ in range(2)]
    c.read(0, table, ints([0, 151, 183]), *back, stream=stream())
    for b, (at, n) in enumerate(((0, 151), (151, 32))):
        kk, vv = (x[at:at + n].double() for x in back)
        want = pc.attention64(q1[b:b + 1].double(), kk, vv, torch.tensor([n - 1], device="cuda"), 1 / math.sqrt(D))
        pc.check_attention(o1[b:b + 1], None, want, dtype, HALF_ULP["f16"] if fmt == "e4m3" else 2.0 ** -16, n / 16 + 64)
    assert c.status() == 0 and prompt_status(ws) == 0


def test_refusals():
    q, k, v = (torch.zeros((4, n, 128), dtype=torch.float16, device="cuda") for n in (8, 2, 2))
    out, ws, cu = torch.empty_like(q), prompt_workspace(4, 8, 128), ints([0, 4])
    for i, f in enumerate([
            lambda: prompt_attn(q, k.bfloat16(), v, cu, 4, out, ws),
            lambda: prompt_attn(q, k[:3], v, cu, 4, out, ws),
            lambda: prompt_attn(q, k, v[:, :1], cu, 4, out, ws),
            lambda: prompt_attn(q, k[..., :64], v, cu, 4, out, ws),
            lambda: prompt_attn(q.float(), k.float(), v.float(), cu, 4, out, ws),
            lambda: prompt_attn(q.cpu(), k.cpu(), v.cpu(), cu, 4, out, ws),
            lambda: prompt_attn(q, k, v, cu.long(), 4, out, ws),
            lambda: prompt_attn(q, k, v, cu.cpu(), 4, out, ws),
            lambda: prompt_attn(q, k, v, ints([[0, 4]]), 4, out, ws),
            lambda: prompt_attn(q, k, v, cu, 4, out[:3], ws),
            lambda: prompt_attn(q, k, v, cu, 4, out.bfloat16(), ws),
            lambda: prompt_attn(q, k, v, cu, 4, out, ws.cpu()),
            lambda: prompt_attn(q, k, v, cu, 4, out, ws, lse=torch.zeros((4, 2), device="cuda")),
            lambda: prompt_attn(q, k, v, cu, 4, out, ws, prefix=ints([1, 2])),
            lambda: prompt_attn(q, k, v, cu, 4, out, ws, slopes=torch.zeros(2, device="cuda")),
            lambda: prompt_attn(q.clone().requires_grad_(), k, v, cu, 4, out, ws)]):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was not refused")
    odd = torch.zeros((4, 3, 128), dtype=torch.float16, device="cuda")
    for code, f in [(1, lambda: prompt_attn(q, odd, odd, cu, 4, out, ws)), (1, lambda: prompt_attn(q, k, v, cu, -1, out, ws)),
                    (1, lambda: prompt_attn(q, k, v, cu, 4, out, ws[:1024])), (1, lambda: prompt_attn(q, k, v, cu, 4, out, ws, softcap=-1.0)),
                    (1, lambda: prompt_attn(q, k, v, cu, 4, out, ws, window=-1)),
                    (1, lambda: prompt_attn(q, k, v, cu, 4, out, ws, softmax_scale=-1.0)),
                    (1, lambda: prompt_attn(q, k, v, cu, 4, out, ws[8:])),
                    (1, lambda: prompt_workspace(4, 8, 96))]:
        with pytest.raises(KVQError) as e:
            f()
        assert e.value.code == code
    assert prompt_status(ws) == 0


@pytest.mark.parametrize("dtype,D,G", [("f16", 128, 4), ("bf16", 64, 3), ("bf16", 256, 2), ("bf16", 128, 5)])
@pytest.mark.parametrize("cap,q_scale", [(30.0, 1.0), (50.0, 3.0), (30.0, 12.0), (1.0, 1.0), (1e6, 1.0), (0.9, 0.5)])
def test_caps_near_and_far(dtype, D, G, cap, q_scale):
    """Scores well inside the cap, beyond it in some tiles, far beyond it in all, and caps at the ends of what the short way takes."""
    case(dtype, 2, G, D, [700, 130], dict(softcap=cap), q_scale=q_scale)


def test_caps_that_some_rows_reach():
    """Every 50th query is long: tiles in which few rows go beyond the polynomial's range, and tiles behind them."""
    q, k, v = rows_of(900, 4, 2, 128, "bf16", 3)
    q[::50] *= 40
    out, lse, ws = torch.empty((900, 4, 128), dtype=torch.bfloat16, device="cuda"), torch.empty((900, 4), device="cuda"), prompt_workspace(900, 4, 128)
    prompt_attn(q, k, v, ints([0, 900]), 900, out, ws, lse=lse, softcap=20.0)
    check(q, k, v, [0], [900], out, lse, dict(softcap=20.0), "bf16")
    assert prompt_status(ws) == 0
