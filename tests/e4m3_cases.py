"""Pages of e4m3 codes for the tests: their layout, the codec in 64 bits and what an append leaves, written out on their own.

256 bytes of status, then per layer the K area and the V area (each padded to 256 bytes), a unit per (page, head), page-major:
[page_size] rows of D codes, then a power of two in fp32 for each 16 rows, padded to 32 bytes.
"""

import numpy as np
import torch

from quantized_kv_cache_gb300 import PagedKVCache, paged_config

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = 16

# the value of each code (0x7f and 0xff: NaN)
_c = np.arange(256)
VALUES = np.where(_c // 8 % 16 == 0, (_c % 8) * 2.0 ** -9, (1 + _c % 8 / 8) * 2.0 ** (_c // 8 % 16 - 7.0)) * np.where(_c < 128, 1.0, -1.0)
VALUES[[127, 255]] = np.nan


def encode(x):
    """fp64 values (448 at most; NaN and infinities give NaN) to codes, nearest, ties to the even code."""
    x = np.asarray(x, np.float64)
    ok = np.isfinite(x)
    a = np.where(ok, np.abs(x), 0.0)
    hi = np.searchsorted(VALUES[:127], a, side="left").clip(max=126)
    lo = np.maximum(hi - 1, 0)
    up, down = VALUES[hi] - a, a - VALUES[lo]
    c = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return np.where(ok, c + 128 * np.signbit(x), np.where(np.signbit(x) & ~np.isnan(x), 255, 127)).astype(np.uint8)


def power(amax):
    """Exponent of the smallest power of two p >= 2^-126 with amax <= 448 p."""
    e = -126
    if amax > 0:
        m, x = np.frexp(np.float64(amax) / 448)
        e = max(-126, int(x) - (1 if m == 0.5 else 0))
    return e


class Pages8:
    """A PagedKVCache of e4m3 pages over a pool of random bytes, and units as numpy views of a host copy."""

    def __init__(self, H, D, ps, n_pages, Hq=None, layers=1, max_seqs=8, max_tokens=4096, seed=0):
        self.H, self.D, self.ps, self.n_pages, self.layers = H, D, ps, n_pages, layers
        self.cfg = paged_config(layers, H, D, Hq or H, ps, n_pages, "e4m3")
        self.dev = torch.device("cuda", 0)
        self.ub = ps * D + max(32, ps // 4)
        self.area = -(-n_pages * H * self.ub // 256) * 256
        g = torch.Generator().manual_seed(seed)
        n = 256 + 2 * layers * self.area
        self.pool = torch.randint(0, 256, (n,), generator=g, dtype=torch.uint8).to(self.dev)
        self.cache = PagedKVCache(self.cfg, 0, max_seqs, max_tokens, pool=self.pool)
        assert self.cache.pool_bytes == n

    def host(self):
        return self.pool.cpu().numpy().copy()

    def unit(self, raw, layer, w, page, head):
        """(codes [ps, D], powers [ps / 16] fp32) of a unit: views of the host copy."""
        at = 256 + (2 * layer + w) * self.area + (page * self.H + head) * self.ub
        u = raw[at:at + self.ub]
        return u[:self.ps * self.D].reshape(self.ps, self.D), u[self.ps * self.D:self.ps * self.D + self.ps // 4].view(np.float32)

    def append(self, raw, layer, w, table, start, x):
        """What an append of rows x [n, H, D] (fp64 numpy) at `start` of the sequence with the given page row leaves."""
        n, ps = len(x), self.ps
        for at in range(start // BLOCK * BLOCK, start + n, BLOCK):
            lo, hi = max(at, start), min(at + BLOCK, start + n)
            for h in range(self.H):
                codes, powers = self.unit(raw, layer, w, int(table[at // ps]), h)
                r, y = at % ps, x[lo - start:hi - start, h]
                e = power(np.abs(y[np.isfinite(y)]).max(initial=0.0))
                if lo > at:
                    held = int(np.frexp(powers[r // BLOCK])[1]) - 1
                    e = max(e, held)
                    if e > held:
                        codes[r:r + lo - at] = encode(VALUES[codes[r:r + lo - at]] * 2.0 ** (held - e))
                codes[r + lo - at:r + hi - at] = encode(y * 2.0 ** -e)
                powers[r // BLOCK] = np.float32(2.0 ** e)

    def rows(self, raw, layer, w, table, n):
        """Values [n, H, D] (fp64) of positions 0 .. n - 1."""
        out = np.zeros((n, self.H, self.D))
        for at in range(0, n, BLOCK):
            for h in range(self.H):
                codes, powers = self.unit(raw, layer, w, int(table[at // self.ps]), h)
                r, k = at % self.ps, min(BLOCK, n - at)
                out[at:at + k, h] = VALUES[codes[r:r + k]] * np.float64(powers[r // BLOCK])
        return out


def taken(x):
    """Row values as the attentions take them: fp16 numbers (fp64 tensors)."""
    return torch.from_numpy(x.astype(np.float16).astype(np.float64)).cuda()


def table_of(p, lens, seed, spare=1):
    """A table over shuffled pages, -7 behind each sequence's pages."""
    need = [-(-n // p.ps) for n in lens]
    assert sum(need) <= p.n_pages
    order, at = np.random.default_rng(seed).permutation(p.n_pages), 0
    table = np.full((len(lens), max(need + [1]) + spare), -7, np.int32)
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        at += k
    return table


def fill(p, layer, lens, seed, dtype="f16", scale=1.0, spare=1):
    """Appends random rows of sequences of the given lengths (through the cache's own call); returns (table CUDA, K rows, V
    rows as the attentions take them: lists of fp64 CUDA)."""
    table = table_of(p, lens, seed, spare)
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = [(scale * torch.randn((sum(lens), p.H, p.D), generator=g, device="cuda")).to(DT[dtype]) for _ in range(2)]
    x[0][:, :, ::32] *= 4
    tt = torch.from_numpy(table).cuda()
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda")
    p.cache.append(layer, x[0], x[1], tt, cu)
    torch.cuda.synchronize()
    raw = p.host()
    k, v = ([taken(p.rows(raw, layer, w, table[b], n)) for b, n in enumerate(lens)] for w in range(2))
    return tt, k, v
