"""Norm and rotation with positions on several axes, on the GPU against 64 bits."""

import pytest

torch = pytest.importorskip("torch")

from paged_cases import DT, HALF_ULP                                                     # noqa: E402
from quantized_kv_cache_gb300 import KVQError, _lib, qk_norm_rope                        # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def axis_of(sections, cyclic):
    if not cyclic:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    taken, out = [0] * len(sections), []
    for r in range(max(sections)):
        for a, n in enumerate(sections):
            if taken[a] < n:
                taken[a] += 1
                out.append(a)
    return out


def want64(x, w, cs, pos, sections, cyclic, inter, eps):
    y = x.double()
    if w is not None:
        y = y / (y.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
    z, n = y.clone(), cs.shape[1] // 2
    for i, a in enumerate(axis_of(sections, cyclic)):
        c, s = (cs[pos[a].long(), k].double()[:, None] for k in (i, n + i))
        p, q = (2 * i, 2 * i + 1) if inter else (i, i + n)
        z[..., p], z[..., q] = y[..., p] * c - y[..., q] * s, y[..., q] * c + y[..., p] * s
    return z, y


def check(got, want, dtype, D):
    z, y = want
    # fp32 steps: the sum of D squares (D 2^-24 bounds it), rsqrt, two products of the weight, two of the rotation and a
    # sum, of the magnitudes of the pair, which the row's largest value bounds; then one rounding
    tol = HALF_ULP[dtype] * z.abs() + (D / 2 + 16) * 2.0 ** -23 * y.abs().amax(-1, keepdim=True) + (2.0 ** -25 if dtype == "f16" else 0.0)
    err = (got.double() - z).abs()
    assert (err <= tol).all(), f"{float((err / tol).max()):.3g} of the tolerance"


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D,rot,sections", [(64, 64, (8, 12, 12)), (64, 16, (5, 3)), (128, 128, (16, 24, 24)), (128, 96, (1, 0, 45, 2)),
                                            (256, 128, (24, 20, 20)), (256, 256, (128,)), (512, 512, (100, 56, 100)), (512, 160, (0, 40, 40)),
                                            (128, 112, (8, 16, 16, 16))])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("cyclic", [False, True])
@pytest.mark.parametrize("T,Hq,H", [(1, 5, 1), (33, 24, 4), (700, 3, 3)])
def test_matches_64_bits(dtype, D, rot, sections, inter, cyclic, T, Hq, H):
    g = torch.Generator(device="cuda").manual_seed(D + rot + T)
    x = (3 * torch.randn((T, Hq + 2 * H, D), generator=g, device="cuda")).to(DT[dtype])
    x[0, 0] = 0.0
    q, k = x[:, :Hq], x[:, Hq:Hq + H]
    wq, wk = (1 + 0.2 * torch.randn((2, D), generator=g, device="cuda")).to(DT[dtype])
    ang = torch.rand((900, rot // 2), generator=g, device="cuda") * 7
    cs = torch.cat((ang.cos(), ang.sin()), 1).contiguous()
    pos = torch.randint(0, 900, (len(sections), T), generator=g, device="cuda", dtype=torch.int32)
    qo, ko = torch.empty((T, Hq, D), dtype=DT[dtype], device="cuda"), torch.empty((T, H, D), dtype=DT[dtype], device="cuda")
    kw = dict(eps=1e-5, interleaved=inter, sections=sections, cyclic=cyclic)
    qk_norm_rope(q, k, wq, wk, cs, pos, qo, ko, **kw)
    args = (cs, pos, sections, cyclic, inter, 1e-5)
    check(qo, want64(q, wq, *args), dtype, D)
    check(ko, want64(k, wk, *args), dtype, D)
    # one side without its norm, in place in the fused buffer; the rest of the buffer stays
    keep = x.clone()
    qk_norm_rope(q, k, None, wk, cs, pos, **kw)
    check(q, want64(keep[:, :Hq], None, *args), dtype, D)
    assert torch.equal(k, ko) and torch.equal(x[:, Hq + H:], keep[:, Hq + H:])


@pytest.mark.parametrize("inter", [False, True])
def test_equal_positions_are_the_rotation_by_one(inter):
    """All axes at one position: what the call with one axis gives, but for the last bits of its fp32 steps."""
    x = torch.randn((50, 6, 128), generator=torch.Generator().manual_seed(0)).cuda().half()
    w, cs = torch.rand(128, device="cuda").half(), torch.rand((60, 128), device="cuda")
    pos = torch.arange(50, device="cuda", dtype=torch.int32)
    a, b = torch.empty_like(x), torch.empty_like(x)
    qk_norm_rope(x, None, w, None, cs, pos, a, interleaved=inter)
    qk_norm_rope(x, None, w, None, cs, pos.repeat(3, 1), b, interleaved=inter, sections=(10, 30, 24), cyclic=True)
    y = want64(x, w, cs, pos.repeat(3, 1), (10, 30, 24), True, inter, 1e-6)
    check(a, y, "f16", 128)
    check(b, y, "f16", 128)


def test_bad_positions_and_axes_without_frequencies():
    x = torch.randn((5, 2, 128), device="cuda").half()
    w, cs = torch.ones(128, device="cuda").half(), torch.rand((10, 128), device="cuda")
    o = torch.empty_like(x)
    pos = torch.tensor([[0, 10, 1, 9, 3], [0, 1, -1, 9, 3], [99, -5, 3, 1 << 30, 3]], dtype=torch.int32, device="cuda")
    qk_norm_rope(None, x, None, w, cs, pos, None, o, sections=(32, 32, 0))
    bad = torch.isnan(o.flatten(1)).all(1)
    assert bad.tolist() == [False, True, True, False, False] and torch.isfinite(o[~bad]).all()
    e = torch.empty((0, 2, 128), dtype=torch.float16, device="cuda")
    qk_norm_rope(e, None, w, None, cs, pos[:2, :0].contiguous(), sections=(60, 4))


def test_captured_call_follows_its_positions():
    x = torch.randn((9, 4, 128), device="cuda").half()
    w, cs, o = torch.ones(128, device="cuda").half(), torch.rand((100, 64), device="cuda"), torch.empty_like(x)
    pos = torch.zeros((2, 9), dtype=torch.int32, device="cuda")
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()

    def call(o, stream=0):
        qk_norm_rope(x, None, w, None, cs, pos, o, sections=(20, 12), stream=stream)

    with torch.cuda.stream(side):
        call(o, side.cuda_stream)
        side.synchronize()
        with torch.cuda.graph(g, stream=side):
            call(o, torch.cuda.current_stream().cuda_stream)
    for i in range(3):
        pos.copy_(torch.randint(0, 100, (2, 9), generator=torch.Generator().manual_seed(i)))
        g.replay()
        want = torch.empty_like(x)
        torch.cuda.synchronize()
        call(want)
        assert torch.equal(o, want)


def test_refusals():
    x = torch.zeros((4, 2, 128), device="cuda").half()
    cs, pos = torch.zeros((4, 128), device="cuda"), torch.zeros((3, 4), dtype=torch.int32, device="cuda")
    for i, f in enumerate([
            lambda: qk_norm_rope(x, None, None, None, cs, pos[:2], sections=(20, 20, 24)),
            lambda: qk_norm_rope(x, None, None, None, cs, pos[0], sections=(20, 20, 24)),
            lambda: qk_norm_rope(x, None, None, None, cs, pos.long(), sections=(20, 20, 24)),
            lambda: qk_norm_rope(x, None, None, None, cs, pos.t().contiguous().t(), sections=(20, 20, 24)),
            lambda: qk_norm_rope(x, None, None, None, cs, None, sections=(20, 20, 24)),
            lambda: qk_norm_rope(x, None, None, None, None, None, sections=(20, 20, 24))]):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was not refused")
    for sections in ((20, 20, 20), (-4, 68), (), (13, 13, 13, 13, 12), (0, 0, 0)):
        with pytest.raises(KVQError) as e:
            qk_norm_rope(x, None, None, None, cs, torch.zeros((len(sections), 4), dtype=torch.int32, device="cuda"), sections=sections)
        assert e.value.code == 1
