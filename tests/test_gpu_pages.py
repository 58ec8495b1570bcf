"""Pages forked, extended, freed, copied and moved on the GPU: tables, counts and bytes against a plain model."""

import random

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import paged_cases as pc                                                                 # noqa: E402
from pages_model import Tables                                                           # noqa: E402
from quantized_kv_cache_gb300 import KVQError, PagedKVCache, _lib, paged_config          # noqa: E402

pytestmark = pytest.mark.gpu
FORMATS = [("f16", "f16"), ("q8_0", "q4_0"), ("q4_0", "q4_0"), ("e4m3", "e4m3")]


@pytest.fixture(autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def stream():
    return torch.cuda.current_stream().cuda_stream


class Pool:
    """A cache over random bytes with its tables on the device, the model beside it, and a host copy of the bytes."""

    def __init__(self, rows, width, n_pages, ps=16, H=2, D=64, fmt=("f16", "f16"), layers=2, stride=None):
        self.cfg = paged_config(layers, H, D, H, ps, n_pages, *fmt)
        n = _lib.kv_paged_required_bytes(self.cfg, 1)[0]
        g = torch.Generator().manual_seed(n_pages)
        self.cache = PagedKVCache(self.cfg, 0, 1, 0, pool=torch.randint(0, 256, (n,), generator=g, dtype=torch.uint8).cuda())
        self.m = Tables(rows, width, n_pages, ps)
        wide = torch.full((rows, stride or width), -1, dtype=torch.int32, device="cuda")
        self.table, self.lens, self.refs = wide[:, :width], ints([0] * rows), ints([0] * n_pages)
        row = {"f16": 2 * D, "q8_0": D + D // 16, "q4_0": D // 2 + D // 16}
        unit = [ps * D + max(32, ps // 4) if f == "e4m3" else ps * row[f] for f in fmt]
        self.page = [H * u for u in unit]                         # bytes of a page in each area
        area = [-(-n_pages * b // 256) * 256 for b in self.page]
        self.areas = [(256 + layer * sum(area) + (area[0] if w else 0), self.page[w]) for layer in range(layers) for w in range(2)]
        self.bytes = self.cache.pool.cpu().numpy().copy()

    def t(self):
        return self.table, self.lens, self.refs

    def moved(self):
        for a, b in self.m.moved:
            for at, n in self.areas:
                self.bytes[at + b * n:at + (b + 1) * n] = self.bytes[at + a * n:at + (a + 1) * n]
        self.m.moved = []

    def check(self, status=0):
        torch.cuda.synchronize()
        assert self.table.tolist() == self.m.table and self.lens.tolist() == self.m.lens and self.refs.tolist() == self.m.refs
        assert self.cache.status() == status
        self.moved()
        assert np.array_equal(self.cache.pool.cpu().numpy()[256:], self.bytes[256:])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("ps,H,D", [(16, 1, 64), (64, 3, 128), (256, 2, 256)])
def test_beams_of_every_format(fmt, ps, H, D):
    """A prompt extended, forked, its beams going on, cut back and freed, the pool compacted."""
    p = Pool(7, 6, 40, ps, H, D, fmt, stride=9)
    p.cache.extend(*p.t(), ints([2 * ps + 5, 0, ps, 0, 0, 0, 1]))
    p.m.extend([2 * ps + 5, 0, ps, 0, 0, 0, 1])
    p.check()
    p.cache.fork(*p.t(), ints([0, 0, 2]), ints([1, 3, 4]))
    p.m.fork([0, 0, 2], [1, 3, 4])
    p.check()
    for add in ([1, 1, 1, 1, 1, 0, 0], [0, ps, 0, 3, 0, 0, 1], [2, 0, 0, 0, 2 * ps, 0, ps - 2]):
        p.cache.extend(*p.t(), ints(add), stream=stream())
        assert p.m.extend(add)
        p.check()
    p.cache.free(*p.t(), ints([3, 0, -1, 5]), ints([ps + 1, 0, 5, 0]))
    p.m.free([3, 0, -1, 5], [ps + 1, 0, 5, 0])
    p.check()
    remap = ints([7] * 40)
    p.cache.compact(*p.t(), remap)
    want = p.m.compact()
    p.check()
    assert remap.tolist() == want
    p.cache.free(*p.t(), ints([0, 1, 2, 3, 4, 5, 6]))
    p.m.free(list(range(7)))
    p.check()
    assert p.refs.sum() == 0


@pytest.mark.parametrize("seed", range(4))
def test_random_calls(seed):
    """Hundreds of calls in random order, among them ones that the pool is too small for."""
    rng = random.Random(seed)
    rows, width, pages = [(12, 9, 60), (3, 40, 50), (70, 3, 100), (1, 5, 4)][seed]
    p = Pool(rows, width, pages, H=1, layers=1)
    for _ in range(120):
        k, status = rng.randrange(4), 0
        if k == 0:
            kids = [rng.randrange(-1, rows + 1) for _ in range(rng.randrange(1, 6))]
            up = [rng.randrange(-1, rows + 1) for _ in kids]
            p.cache.fork(*p.t(), ints(up), ints(kids))
            status = _lib.PAGED_BAD_INDEX * p.m.fork(up, kids)
        elif k == 1:
            add = [rng.choice([0, 0, 1, 5, 20]) for _ in range(rows)]
            over = any(a > width * 16 - n for a, n in zip(add, p.m.lens))
            p.cache.extend(*p.t(), ints(add))
            status = (0 if p.m.extend(add) else _lib.PAGED_NO_PAGES) | _lib.PAGED_BAD_LENGTH * over
        elif k == 2:
            some = [rng.randrange(-1, rows) for _ in range(3)]
            keep = [rng.choice([0, rng.randrange(100)]) for _ in some]
            p.cache.free(*p.t(), ints(some), ints(keep))
            p.m.free(some, keep)
        else:
            remap = ints([0] * pages)
            p.cache.compact(*p.t(), remap)
            assert remap.tolist() == p.m.compact()
        p.check(status)
        p.m.check()


def test_many_rows_and_pages():
    """More rows than the deciding block has threads, more pages than it reads at once, a long sequence and an odd count."""
    rows, pages = 2500, 20011
    p = Pool(rows, 5000, pages, H=1, layers=1)
    add = [(7 * r) % 41 for r in range(rows)]
    add[1700] = 70000
    p.cache.extend(*p.t(), ints(add))
    assert p.m.extend(add)
    p.check()
    gone = [r for r in range(rows) if r % 3 == 1 and r != 1700]
    p.cache.free(*p.t(), ints(gone))
    p.m.free(gone)
    p.check()
    kids = gone[:600]
    up = [(r + 1) % rows for r in kids]
    up[5] = 1700
    p.cache.fork(*p.t(), ints(up), ints(kids))
    assert not p.m.fork(up, kids)
    p.check()
    add = [r % 2 for r in range(rows)]
    p.cache.extend(*p.t(), ints(add))
    assert p.m.extend(add)
    p.check()
    remap = ints([0] * pages)
    p.cache.compact(*p.t(), remap)
    assert remap.tolist() == p.m.compact()
    p.check()


def test_too_few_pages_change_nothing():
    p = Pool(4, 8, 6)
    p.cache.extend(*p.t(), ints([40, 17, 0, 0]))
    assert p.m.extend([40, 17, 0, 0])
    p.check()
    for add in ([9, 0, 1, 1], [0, 0, 0, 100], [0, 100, 0, 0]):
        p.cache.extend(*p.t(), ints(add))
        assert not p.m.extend(add)
        p.check(_lib.PAGED_NO_PAGES)
    p.cache.extend(*p.t(), ints([8, 15, 0, 0]))              # what the pages have room for needs none
    assert p.m.extend([8, 15, 0, 0])
    p.check()


def test_rows_that_do_not_fit_are_left_out():
    """Rows that would outgrow their table, shrink, hold a negative length or go on in no page: the others go on."""
    p = Pool(6, 2, 20)
    p.cache.extend(*p.t(), ints([20, 5, 5, 5, 32, 0]))
    assert p.m.extend([20, 5, 5, 5, 32, 0])
    p.check()
    p.table[2, 0] = 20
    p.m.table[2][0] = 20
    p.cache.extend(*p.t(), ints([12, 1, 1, -1, 1, 2147483647]))
    p.m.extend([12, 1, 0, 0, 0, 0])
    p.check(_lib.PAGED_BAD_LENGTH | _lib.PAGED_BAD_INDEX)
    p.lens[1], p.m.lens[1] = -3, -3
    p.cache.extend(*p.t(), ints([0, 1, 0, 0, 0, 0]))
    p.check(_lib.PAGED_BAD_LENGTH)


def test_a_shared_page_that_some_go_on_in_is_copied_for_them():
    p = Pool(5, 4, 12)
    p.cache.extend(*p.t(), ints([10, 0, 0, 0, 0]))
    p.m.extend([10, 0, 0, 0, 0])
    p.cache.fork(*p.t(), ints([0, 0, 0]), ints([1, 2, 3]))
    p.m.fork([0, 0, 0], [1, 2, 3])
    for add in ([0, 1, 1, 0, 0], [3, 0, 0, 0, 0], [0, 0, 0, 1, 0], [1, 1, 1, 1, 1]):
        p.cache.extend(*p.t(), ints(add))
        assert p.m.extend(add)
        p.check()
    # a page that another owner counts in is copied even for its only row
    p.refs[p.m.table[0][0]] += 1
    p.m.refs[p.m.table[0][0]] += 1
    p.cache.extend(*p.t(), ints([1, 0, 0, 0, 0]))
    p.m.extend([1, 0, 0, 0, 0])
    p.check()


def test_free_twice_and_of_bad_rows():
    p = Pool(4, 4, 12)
    p.cache.extend(*p.t(), ints([60, 20, 5, 0]))
    p.m.extend([60, 20, 5, 0])
    p.cache.free(*p.t(), ints([0, 0, 0, 1, 1]), ints([40, 17, 50, 30, 20]))
    p.m.free([0, 0, 0, 1, 1], [40, 17, 50, 30, 20])
    p.check()
    p.cache.free(*p.t(), ints([4, 1 << 30]))
    p.check(_lib.PAGED_BAD_INDEX)
    p.cache.free(*p.t(), ints([2]), ints([-1]))
    p.check(_lib.PAGED_BAD_LENGTH)
    page = p.m.table[2][0]
    p.refs[page] = 0                                          # a count that was lost: it does not go below zero
    p.cache.free(*p.t(), ints([2]))
    p.m.free([2])
    p.m.refs[page] = 0
    p.check(_lib.PAGED_BAD_INDEX)


@pytest.mark.parametrize("fmt", FORMATS)
def test_copied_pages(fmt):
    p = Pool(1, 1, 30, 32, 3, 128, fmt, layers=3)
    p.cache.copy_pages(ints([3, 29, -1, 5, 7]), ints([4, 0, 6, -2, 8]))
    p.m.moved = [(3, 4), (29, 0), (7, 8)]
    p.check()
    p.cache.copy_pages(ints([3, 30, 2]), ints([10, 11, 1 << 30]))
    p.m.moved = [(3, 10)]
    p.check(_lib.PAGED_BAD_INDEX)
    p.cache.copy_pages(ints([]), ints([]))
    p.check()


def test_compact_of_empty_full_and_compact_pools():
    for pages, used in ((9, []), (9, list(range(9))), (9, [0, 1, 2]), (9, [8]), (1, [0]), (4097, [4096, 4000, 1])):
        p = Pool(2, max(len(used), 1), pages, H=1, layers=1)
        for e, x in enumerate(used):
            p.table[0, e] = x
            p.refs[x] = 1
            p.m.table[0][e], p.m.refs[x] = x, 1
        p.lens[0] = p.m.lens[0] = 16 * len(used)
        remap = ints([5] * pages)
        p.cache.compact(*p.t(), remap)
        assert remap.tolist() == p.m.compact()
        p.check()


def test_calls_captured_and_replayed():
    """Free, fork, extend and compact captured once and replayed on other tables and numbers."""
    p = Pool(6, 6, 50)
    rows, keep, up, kids, add, remap = ints([-1] * 3), ints([0] * 3), ints([-1] * 3), ints([-1] * 3), ints([0] * 6), ints([0] * 50)

    def step():
        p.cache.free(*p.t(), rows, keep, stream=stream())
        p.cache.fork(*p.t(), up, kids, stream=stream())
        p.cache.extend(*p.t(), add, stream=stream())
        p.cache.compact(*p.t(), remap, stream=stream())

    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        step()
        side.synchronize()
        with torch.cuda.graph(g, stream=side):
            step()
    for r, k, u, c, a in (([-1, -1, -1], [0, 0, 0], [-1, -1, -1], [-1, -1, -1], [33, 0, 7, 0, 0, 50]), ([2, -1, -1], [3, 0, 0], [0, 0, 5], [1, 3, 4], [1, 1, 1, 1, 1, 0]),
                         ([5, 0, 1], [0, 20, 0], [0, 2, -1], [5, 1, -1], [1, 0, 30, 2, 1, 16])):
        for x, y in ((rows, r), (keep, k), (up, u), (kids, c), (add, a)):
            x.copy_(ints(y))
        g.replay()
        p.m.free(r, k)
        p.m.fork(u, c)
        assert p.m.extend(a)
        p.moved()
        p.m.compact()
        p.check()


def test_beams_decode_what_they_hold():
    """Beams of one prompt, each going on with tokens of its own: the attention over the shared and copied pages is that over
    each beam's own rows."""
    H, G, D, ps = 2, 2, 64, 16
    for fmt in ("f16", "e4m3"):
        c = PagedKVCache(paged_config(1, H, D, H * G, ps, 30, fmt), 0, 4, 0)
        table, lens, refs = torch.full((4, 5), -1, dtype=torch.int32, device="cuda"), ints([0] * 4), ints([0] * 30)
        held = [[], [], [], []]

        def put(which, seed):
            """One more token of each of the rows `which`."""
            kv = torch.randn((len(which), 2, H, D), generator=torch.Generator().manual_seed(seed)).half().cuda()
            add = [int(r in which) for r in range(4)]
            c.extend(table, lens, refs, ints(add))
            at, tab = lens.tolist(), table.tolist()
            if fmt == "f16":
                c.write(0, kv[:, 0], kv[:, 1], ints([tab[r][(at[r] - 1) // ps] * ps + (at[r] - 1) % ps for r in which]))
            else:
                c.append(0, kv[:, 0], kv[:, 1], table[which].contiguous(), ints(list(range(len(which) + 1))), ints([at[r] - 1 for r in which]))
            for i, r in enumerate(which):
                held[r].append(kv[i])

        for s in range(21):
            put([0], s)
        c.fork(table, lens, refs, ints([0, 0, 0]), ints([1, 2, 3]))
        for r in (1, 2, 3):
            held[r] = list(held[0])
        for s in range(15):
            put([0, 1, 3] if s % 3 else [1, 2], 100 + s)
        c.compact(table, lens, refs, ints([0] * 30))
        q = torch.randn((4, H * G, D), generator=torch.Generator().manual_seed(5)).half().cuda()
        out = torch.empty_like(q)
        c.decode_attn(0, q, table, lens, out)
        assert lens.tolist() == [len(x) for x in held] and c.status() == 0
        if fmt == "e4m3":
            back = [torch.empty((int(lens.sum()), H, D), device="cuda") for _ in range(2)]
            c.read(0, table, ints([0] + list(np.cumsum([len(x) for x in held]))), *back)
        at = 0
        for r in range(4):
            n = len(held[r])
            k, v = (torch.stack([x[i] for x in held[r]]).double() for i in range(2))
            if fmt == "e4m3":
                for mine, pages in ((k, back[0]), (v, back[1])):
                    # half a step of three bits of the value, or of the smallest code (2^-9) under the block's power of two, twice
                    # over where a block's power grew; powers here are 2^-6 at most (values below 7)
                    assert ((pages[at:at + n].double() - mine).abs() <= 2 * (2.0 ** -4 * mine.abs() + 2.0 ** -16)).all()
                k, v = back[0][at:at + n].double(), back[1][at:at + n].double()
            at += n
            want = pc.attention64(q[r:r + 1].double(), k, v, torch.tensor([n - 1], device="cuda"), 1 / 8)
            pc.check_attention(out[r:r + 1], None, want, "f16", 2.0 ** -11, 70)


def test_refusals():
    p = Pool(4, 4, 12)
    c, (table, lens, refs) = p.cache, p.t()
    x = ints([0, 1])
    for i, f in enumerate([
            lambda: c.fork(table.long(), lens, refs, x, x), lambda: c.fork(table, lens[:3], refs, x, x), lambda: c.fork(table, lens, refs[:5], x, x),
            lambda: c.fork(table, lens, refs, x, x[:1]), lambda: c.fork(table, lens, refs, x.long(), x), lambda: c.fork(table.cpu(), lens, refs, x, x),
            lambda: c.extend(table, lens, refs, x), lambda: c.extend(table, lens, refs.cpu(), lens), lambda: c.extend(table, lens, refs, lens, ws=torch.zeros(9)),
            lambda: c.free(table, lens, refs, x, x[:1]), lambda: c.free(table, lens, refs, x.cpu()), lambda: c.free(table[0], lens, refs, x),
            lambda: c.compact(table, lens, refs, lens), lambda: c.copy_pages(x, x[:1]), lambda: c.copy_pages(x.float(), x), lambda: c.copy_pages(x[None], x[None]),
            lambda: c.compact(table, lens, refs, torch.zeros(24, dtype=torch.int32, device="cuda")[::2])]):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was not refused")
    small, long = torch.empty(64, dtype=torch.uint8, device="cuda"), torch.zeros(65536, dtype=torch.int32, device="cuda")
    for code, f in [(1, lambda: c.extend(table, lens, refs, lens, ws=small)), (1, lambda: c.compact(table, lens, refs, refs.clone(), ws=small)),
                    (3, lambda: c.fork(table, lens, refs, long, long))]:
        with pytest.raises(KVQError) as e:
            f()
        assert e.value.code == code
    p.check()
    c.extend(table, lens, refs, ints([20, 0, 0, 1]), ws=c.new_pages_workspace())
    p.m.extend([20, 0, 0, 1])
    p.check()
