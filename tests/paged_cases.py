"""Paged-cache test helpers: a pool with known contents, and attention over it in 64 bits.

The layout is written out here on its own: 256 bytes of status, then per layer the K area and the V
area (each padded to 256 bytes), a unit per (page, head), page-major; a unit is page_size code rows,
then for q8_0 / q4_0 the scales [page_size][D / 32] fp16.
"""

import math

import numpy as np
import torch

from oracle import codecs, fp
from quantized_kv_cache_gb300 import PagedKVCache, paged_config

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
HALF_ULP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def row_bytes(fmt, D):
    return {"f16": 2 * D, "bf16": 2 * D, "q8_0": D, "q4_0": D // 2}[fmt]


def unit_bytes(fmt, D, ps):
    return ps * (row_bytes(fmt, D) + (D // 16 if fmt[0] == "q" else 0))


class Pages:
    """A PagedKVCache over a pool of random bytes, and its areas as numpy views of a host copy."""

    def __init__(self, H, D, ps, n_pages, k_fmt, v_fmt, Hq=None, layers=1, max_seqs=8, max_tokens=4096, seed=0, dev=0):
        self.H, self.D, self.ps, self.n_pages, self.fmt, self.layers = H, D, ps, n_pages, (k_fmt, v_fmt), layers
        self.cfg = paged_config(layers, H, D, Hq or H, ps, n_pages, k_fmt, v_fmt)
        self.dev = torch.device("cuda", dev)
        self.area = [-(-n_pages * H * unit_bytes(f, D, ps) // 256) * 256 for f in self.fmt]
        g = torch.Generator().manual_seed(seed)
        n = 256 + layers * sum(self.area)
        self.pool = torch.randint(0, 256, (n,), generator=g, dtype=torch.uint8).to(self.dev)
        self.cache = PagedKVCache(self.cfg, dev, max_seqs, max_tokens, pool=self.pool)
        assert self.cache.pool_bytes == n

    def host(self):
        return self.pool.cpu().numpy().copy()

    def unit(self, raw, layer, w, page, head):
        ub = unit_bytes(self.fmt[w], self.D, self.ps)
        at = 256 + layer * sum(self.area) + (self.area[0] if w else 0) + (page * self.H + head) * ub
        return raw[at:at + ub]

    def put(self, raw, layer, w, page, row, x):
        """Stores x [H, D] (fp32 numpy) in a host copy, by the oracle's codecs."""
        fmt, D = self.fmt[w], self.D
        for h in range(self.H):
            u, rb = self.unit(raw, layer, w, page, h), row_bytes(fmt, D)
            if fmt == "f16":
                b = x[h].astype(np.float16).view(np.uint8)
            elif fmt == "bf16":
                b = fp.bf16_bits_from_f32(x[h].astype(np.float32)).view(np.uint8)
            else:
                d, q = (codecs.q8_encode if fmt == "q8_0" else codecs.q4_encode)(x[h][None].astype(np.float32))
                b = q.reshape(-1).view(np.uint8) if fmt == "q8_0" else codecs.pack_nibbles(q.reshape(1, -1)).reshape(-1)
                at = self.ps * rb + row * (D // 16)
                u[at:at + D // 16] = d.reshape(-1).view(np.uint8)
            u[row * rb:(row + 1) * rb] = b

    def get(self, raw, layer, w, page, row):
        """The values [H, D] (fp32, exact) of a row of a host copy."""
        fmt, D, out = self.fmt[w], self.D, []
        for h in range(self.H):
            u, rb = self.unit(raw, layer, w, page, h), row_bytes(fmt, D)
            b = np.ascontiguousarray(u[row * rb:(row + 1) * rb])
            if fmt == "f16":
                out.append(b.view(np.float16).astype(np.float32))
            elif fmt == "bf16":
                out.append(fp.bf16_bits_to_f32(b.view(np.uint16)))
            else:
                at = self.ps * rb + row * (D // 16)
                d = np.ascontiguousarray(u[at:at + D // 16]).view(np.float16)[None]
                q = b.view(np.int8) if fmt == "q8_0" else codecs.unpack_nibbles(b[None]).reshape(-1)
                out.append((codecs.q8_decode if fmt == "q8_0" else codecs.q4_decode)(d, q.reshape(1, -1, 32))[0])
        return np.stack(out)


def fill(p, layer, lens, seed, dtype="f16", spare=1, scale=1.0):
    """Writes random rows of sequences of the given lengths (through the cache's own write) over shuffled
    pages; returns (table int32 CUDA, K rows, V rows as the attention takes them: lists of fp64 CUDA)."""
    rng = np.random.default_rng(seed)
    need = [-(-n // p.ps) for n in lens]
    assert sum(need) <= p.n_pages
    order = rng.permutation(p.n_pages)
    width = max(need + [1]) + spare
    table = np.full((len(lens), width), -7, np.int32)
    slots, at = [], 0
    for b, n in enumerate(lens):
        pages = order[at:at + need[b]]
        at += need[b]
        table[b, :need[b]] = pages
        i = np.arange(n)
        slots.append(pages[i // p.ps] * p.ps + i % p.ps if n else np.zeros(0, np.int64))
    slots = np.concatenate(slots).astype(np.int32)
    g = torch.Generator(device=p.dev).manual_seed(seed)
    x = [(scale * torch.randn((len(slots), p.H, p.D), generator=g, device=p.dev)).to(DT[dtype]) for _ in range(2)]
    st = torch.from_numpy(slots).to(p.dev)
    p.cache.write(layer, x[0], x[1], st)
    n, dev = len(slots), p.dev
    back = [torch.zeros((n, p.H, p.D), device=dev) for _ in range(2)]
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device=dev)
    tt = torch.from_numpy(table).to(dev)
    if n:
        p.cache.read(layer, tt, cu, back[0], back[1])
    torch.cuda.synchronize()
    rows = []
    for w in range(2):
        y = back[w] if p.fmt[w][0] != "q" else back[w].half().float()
        rows.append([y[sum(lens[:b]):sum(lens[:b + 1])].double() for b in range(len(lens))])
    return tt, rows[0], rows[1]


def attention64(q, k, v, pos, scale, softcap=0.0, window=0, slopes=None, prefix=0):
    """q [n, Hq, D], k, v [L, H, D], pos [n], all fp64: (out, lse, mean |v| by the same weights, bound on the
    error of a score in fp32 steps)."""
    n, Hq, D = q.shape
    L, H = k.shape[:2]
    G = Hq // H
    out = torch.zeros_like(q)
    lse = torch.full((n, Hq), -math.inf, dtype=torch.float64, device=q.device)
    wabs = torch.zeros_like(q)
    ds = torch.zeros((n, Hq), dtype=torch.float64, device=q.device)
    if L == 0 or n == 0:
        return out, lse, wabs, ds
    j = torch.arange(L, device=q.device)
    see = j <= pos[:, None]
    if window:
        see = see & (j > pos[:, None] - window)
    see = (see | (j < prefix)) & (pos[:, None] >= 0)
    some = see.any(1)
    for h in range(Hq):
        s = scale * (q[:, h] @ k[:, h // G].T)
        mag = scale * (q[:, h].abs() @ k[:, h // G].abs().T)
        if softcap:
            s = softcap * torch.tanh(s / softcap)
        if slopes is not None:
            s = s - slopes[h].double() * (pos[:, None] - j).abs()
        s = torch.where(see, s, -math.inf)
        z = torch.logsumexp(s, 1)
        w = torch.where(some[:, None], torch.exp(s - torch.where(some, z, 0.0)[:, None]), 0.0)
        out[:, h], wabs[:, h], lse[:, h] = w @ v[:, h // G], w @ v[:, h // G].abs(), z
        # fp32 sums of the products (D / 16 accumulations of 16 terms, each step off by at most 2^-22 of the
        # magnitudes), the scale, cap and bias in fp32, and the base-2 exponent of |s| up to 2^-22 |s|
        big = torch.where(see, s.abs(), 0.0).amax(1)
        ds[:, h] = 2.0 ** -22 * ((D / 16 + 4) * torch.where(see, mag, 0.0).amax(1) + 4 * big + 4 * softcap + 4)
    return out, lse, wabs, ds


def check_attention(got, lse_got, want, dtype, p_half_ulp, steps):
    """|got - want| against: the output's rounding, the weights' rounding (p_half_ulp relative, and half of the
    smallest fp16 step), the scores' error, and `steps` fp32 accumulations of the outputs."""
    out, lse, wabs, ds = want
    assert torch.isfinite(got).all()
    rel = p_half_ulp + 4 * ds[..., None] + steps * 2.0 ** -23
    tol = HALF_ULP[dtype] * out.abs() + (1 + HALF_ULP[dtype]) * rel * wabs + 2.0 ** -24
    tol = tol + 2.0 ** -25 * wabs.amax(-1, keepdim=True) * 64
    err = (got.double() - out).abs()
    bad = err > tol
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off: {float((err / tol).max()):.3g} of the tolerance"
    if lse_got is not None:
        empty = torch.isinf(lse)
        assert torch.equal(torch.isinf(lse_got) & (lse_got < 0), empty)
        d = (lse_got.double() - lse)[~empty].abs()
        lim = (2 * ds + 2.0 ** -21 * (lse.abs() + 1) + steps * 2.0 ** -24)[~empty]
        assert (d <= lim).all(), f"lse off by {float((d / lim).max()):.3g} of the tolerance"
