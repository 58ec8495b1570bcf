"""The paged-cache operators: what is measured, their plain forms and their definition in 64 bits.

Operators (case["op"]):
- "norm_rope": RMS norm of every query and key head and the rotation by position, one pass over a projection's output.
- "write":     key and value rows to pages at given slots; 16-bit pages come back whole, 8- and 4-bit pages as the
               values they stand for, read back from the pages the call has written.
- "read":      positions of ragged sequences gathered from the pages into contiguous rows.
- "decode":    attention of one new token per sequence over its pages.
- "prefill":   attention of a chunk of new tokens per sequence over its pages (their own rows are in the pages).

Pages: a pool of bytes, [256 B status | K units | V units], a unit per (page, KV head): [page_size] rows of D codes, then
for q8_0 / q4_0 [page_size][D / 32] fp16 scales; each of the two areas is padded to 256 bytes.
"""

import math

import numpy as np
import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
LEVELS = {"q8_0": 127, "q4_0": 7}


# ------------------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # a decode step's projections: 8 sequences, the hybrid shape (24 query and 4 KV heads of 256)
        dict(name="norm_rope_step", op="norm_rope", tokens=8, Hq=24, H=4, D=256, rot=256, interleaved=False,
             dtype="bf16", max_pos=262144),
        # a prompt chunk of an odd length, the 14B shape (40 query and 8 KV heads of 128), half of the channels rotated
        dict(name="norm_rope_chunk", op="norm_rope", tokens=8191, Hq=40, H=8, D=128, rot=64, interleaved=True,
             dtype="f16", max_pos=131072),
        # a decode step's new rows: 32 sequences, 16-bit pages
        dict(name="write_step", op="write", tokens=32, H=8, D=128, page_size=16, pages=1024, k_fmt="bf16", v_fmt="bf16",
             dtype="bf16", pad=0.0),
        # a prompt chunk quantised into pages, with padded rows (slot -1) among its tokens
        dict(name="write_chunk_q8q4", op="write", tokens=16383, H=8, D=128, page_size=64, pages=1024, k_fmt="q8_0",
             v_fmt="q4_0", dtype="f16", pad=0.02),
        # a long cache read back for a second pass over it
        dict(name="read_q8", op="read", seqs=3, longest=65536, H=4, D=256, page_size=64, k_fmt="q8_0", v_fmt="q8_0",
             dtype="bf16", ragged=0.7),
        # a few short prefixes read back from 16-bit pages
        dict(name="read_short", op="read", seqs=5, longest=300, H=8, D=128, page_size=16, k_fmt="f16", v_fmt="f16",
             dtype="f16", ragged=0.9),
        # one short sequence: the latency of a decode call
        dict(name="decode_tiny", op="decode", seqs=1, longest=1024, Hq=4, H=2, D=128, page_size=16, k_fmt="f16",
             v_fmt="f16", dtype="f16", ragged=0.0, softcap=0.0, window=0, prefix=0, slopes=False),
        # a batch of ragged sequences, capped scores
        dict(name="decode_batch", op="decode", seqs=48, longest=24001, Hq=40, H=8, D=128, page_size=32, k_fmt="bf16",
             v_fmt="bf16", dtype="bf16", ragged=0.9, softcap=30.0, window=0, prefix=0, slopes=False),
        # one long sequence over a quantised cache (the 14B shape at its full context)
        dict(name="decode_long_q8q4", op="decode", seqs=1, longest=131072, Hq=40, H=8, D=128, page_size=64,
             k_fmt="q8_0", v_fmt="q4_0", dtype="f16", ragged=0.0, softcap=0.0, window=0, prefix=0, slopes=False),
        # the long-context batch of the hybrid shape, distance biases
        dict(name="decode_longctx", op="decode", seqs=4, longest=262144, Hq=24, H=4, D=256, page_size=64, k_fmt="f16",
             v_fmt="f16", dtype="f16", ragged=0.75, softcap=0.0, window=0, prefix=0, slopes=True),
        # the second half of a prompt over the pages of both halves
        dict(name="prefill_chunk", op="prefill", seqs=1, longest=8192, q_longest=4096, Hq=40, H=8, D=128, page_size=64,
             k_fmt="bf16", v_fmt="bf16", dtype="bf16", ragged=0.0, softcap=0.0, window=0, prefix=0, slopes=False),
        # packed prompts of odd lengths: capped scores, a sliding window and a prefix all tokens see, quantised pages
        dict(name="prefill_docs", op="prefill", seqs=6, longest=2500, q_longest=1201, Hq=24, H=4, D=256, page_size=16,
             k_fmt="q8_0", v_fmt="q8_0", dtype="f16", ragged=0.8, softcap=50.0, window=1024, prefix=100, slopes=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "write", "read", "decode", "decode", "prefill"])
    D = rng.choice([64, 128, 128, 256])
    H, G = rng.choice([(2, 2), (4, 6), (8, 5), (2, 16), (8, 1), (1, 8), (3, 3)])
    dtype = rng.choice(["f16", "bf16"])
    c = dict(op=op, H=H, D=D, dtype=dtype)
    if op == "norm_rope":
        c.update(tokens=_log(rng, 1, 8191), Hq=H * G, rot=rng.choice([D, D // 2]), interleaved=rng.random() < 0.5,
                 max_pos=rng.choice([32768, 262144]))
        return c
    c["page_size"] = rng.choice([16, 32, 64, 128])
    k, v = rng.choice([(dtype, dtype), ("q8_0", "q8_0"), ("q8_0", "q4_0"), ("q4_0", "q4_0")])
    c.update(k_fmt=k, v_fmt=v)
    if op == "write":
        T = _log(rng, 1, 16384)
        c.update(tokens=T, pages=2 * (T // c["page_size"] + 1), pad=rng.choice([0.0, 0.05]))
        return c
    c.update(seqs=_log(rng, 1, 24), ragged=rng.choice([0.0, 0.5, 0.95]))
    if op == "read":
        c.update(longest=max(1, _log(rng, 1, 65536) // c["seqs"]))
        return c
    c.update(Hq=H * G, softcap=rng.choice([0.0, 0.0, 30.0]), window=rng.choice([0, 0, 500]),
             prefix=rng.choice([0, 0, 37]), slopes=rng.random() < 0.3)
    if op == "decode":
        c.update(longest=max(1, _log(rng, 8, 262144) // c["seqs"]))
    else:
        c["q_longest"] = max(1, _log(rng, 1, 4096) // c["seqs"])
        c["longest"] = c["q_longest"] + _log(rng, 1, 4096) // c["seqs"]
    return c


# ------------------------------------------------------------------------------------------------ inputs
def _lens(case):
    """Lengths from the case alone: the longest first, the others between (1 - ragged) of it and it."""
    n, m, r = case["seqs"], case["longest"], case["ragged"]
    rng = np.random.default_rng(n * 1000003 + m)
    u = rng.random(n)
    u[0] = 0.0
    lens = [max(1, int(m * (1 - r * x))) for x in u]
    return lens


def _qlens(case):
    lens = _lens(case)
    q = case["q_longest"]
    return [max(1, min(n, int(round(q * n / lens[0])))) for n in lens]


def _unit_bytes(fmt, ps, D):
    return ps * {"f16": 2 * D, "bf16": 2 * D, "q8_0": D + D // 16, "q4_0": D // 2 + D // 16}[fmt]


def _areas(case, n_pages):
    """Byte offsets of the K and V areas, and the pool's size."""
    off, at = [], 256
    for w in ("k_fmt", "v_fmt"):
        off.append(at)
        at += -(-n_pages * case["H"] * _unit_bytes(case[w], case["page_size"], case["D"]) // 256) * 256
    return off, at


def _views(case, pool, n_pages, w):
    """(codes or values, scales) of the K (w = 0) or V (w = 1) area, as views of the pool."""
    H, D, ps = case["H"], case["D"], case["page_size"]
    fmt = case["v_fmt" if w else "k_fmt"]
    ub = _unit_bytes(fmt, ps, D)
    at = _areas(case, n_pages)[0][w]
    u = pool[at:at + n_pages * H * ub].view(n_pages, H, ub)
    if fmt in DT:
        return u.view(DT[fmt]).view(n_pages, H, ps, D), None
    rows = D if fmt == "q8_0" else D // 2
    codes = u[:, :, :ps * rows].unflatten(2, (ps, rows))
    return codes, u[:, :, ps * rows:].view(torch.float16).unflatten(2, (ps, D // 32))


def _codes(x, fmt):
    """Integer codes and fp16 scales of rows x [..., D], the block formats' definition in fp32 steps."""
    b = x.float().unflatten(-1, (-1, 32))
    top = torch.tensor(float(LEVELS[fmt]), device=x.device)
    d = (b.abs().amax(-1) / top).half()
    inv = torch.where(d == 0, torch.zeros_like(d, dtype=torch.float32), 1.0 / d.float())
    return (b * inv[..., None]).round().clamp(-top, top).flatten(-2).to(torch.int32), d


def _store(case, pool, n_pages, w, slots, x):
    """Rows x [n, H, D] to the slots [n] of an area (indexing, no loop)."""
    ps = case["page_size"]
    fmt = case["v_fmt" if w else "k_fmt"]
    page, at = slots // ps, slots % ps
    codes, scales = _views(case, pool, n_pages, w)
    if fmt in DT:
        codes[page, :, at] = x.to(DT[fmt])
        return
    q, d = _codes(x, fmt)
    if fmt == "q8_0":
        codes[page, :, at] = q.to(torch.int8).view(torch.uint8)
    else:
        n = (q + 8).to(torch.uint8)
        codes[page, :, at] = n[..., 0::2] | (n[..., 1::2] << 4)
    scales[page, :, at] = d


def _load(case, pool, n_pages, w, page, at):
    """Values [..., H, D] in fp32 of the rows at (page, at), two index tensors of one shape."""
    fmt = case["v_fmt" if w else "k_fmt"]
    codes, scales = _views(case, pool, n_pages, w)
    c = codes.movedim(2, 1)[page, at]
    if fmt in DT:
        return c.float()
    if fmt == "q8_0":
        q = c.view(torch.int8).float()
    else:
        q = torch.stack((c & 15, c >> 4), -1).flatten(-2).float() - 8.0
    return (q.unflatten(-1, (-1, 32)) * scales.movedim(2, 1)[page, at].float()[..., None]).flatten(-2)


def _table(case, lens, rng, dev):
    """A page table over shuffled pages, -1 behind each sequence's last page, and the number of pages."""
    ps = case["page_size"]
    need = [-(-n // ps) for n in lens]
    n_pages = sum(need) + 3
    order = rng.permutation(n_pages)
    table = np.full((len(lens), max(need) + 1), -1, np.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        at += k
    return torch.from_numpy(table).to(dev), n_pages


def _handle(case, pool, n_pages, Hq):
    from quantized_kv_cache_gb300 import PagedKVCache, paged_config
    cfg = paged_config(n_layers=1, n_kv_heads=case["H"], head_dim=case["D"], n_q_heads=Hq, page_size=case["page_size"],
                       n_pages=n_pages, k_fmt=case["k_fmt"], v_fmt=case["v_fmt"])
    return PagedKVCache(cfg, pool.device.index, max_seqs=case.get("seqs", 1),
                        max_tokens=case.get("seqs", 1) * case.get("q_longest", 1), pool=pool)


def _normal(g, shape, dtype, dev):
    return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(DT[dtype])


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev).manual_seed(seed)
    rng = np.random.default_rng(seed)
    H, D, op = case["H"], case["D"], case["op"]
    s = {"case": case}
    if op == "norm_rope":
        T, Hq, rot = case["tokens"], case["Hq"], case["rot"]
        qkv = _normal(g, (T, Hq + 2 * H, D), case["dtype"], dev)     # one projection's output, V beside Q and K
        s["q"], s["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + H]
        s["wq"], s["wk"] = (1 + 0.1 * _normal(g, (2, D), "f32", dev)).to(DT[case["dtype"]]).unbind(0)
        i = torch.arange(rot // 2, device=dev, dtype=torch.float64)
        ang = torch.arange(case["max_pos"], device=dev, dtype=torch.float64)[:, None] * 1e6 ** (-2 * i / rot)
        s["cos_sin"] = torch.cat((ang.cos(), ang.sin()), 1).float()
        p0 = int(rng.integers(0, case["max_pos"] - T))
        s["pos"] = torch.arange(p0, p0 + T, device=dev, dtype=torch.int32)
        s["q_out"], s["k_out"] = (torch.empty((T, n, D), dtype=DT[case["dtype"]], device=dev) for n in (Hq, H))
        return s
    if op == "write":
        T, ps, n_pages = case["tokens"], case["page_size"], case["pages"]
        slots = rng.permutation(n_pages)[:T // ps + 1, None] * ps + np.arange(ps)
        slots = slots.reshape(-1)[:T].astype(np.int32)
        slots[rng.random(T) < case["pad"]] = -1
        s["slots"], s["n_pages"] = torch.from_numpy(slots).to(dev), n_pages
        kv = _normal(g, (T, 2 * H, D), case["dtype"], dev)
        kv[:, :H, ::32] *= 12                                          # outlier channels of keys
        s["k"], s["v"] = kv[:, :H], kv[:, H:]
        s["pool"] = torch.zeros(_areas(case, n_pages)[1], dtype=torch.uint8, device=dev)
        if case["k_fmt"] not in DT:                                    # quantised rows are read back
            s["table"] = torch.arange(n_pages, device=dev, dtype=torch.int32)[None]
            s["cu"] = torch.tensor([0, n_pages * ps], device=dev, dtype=torch.int32)
            s["k_out"], s["v_out"] = (torch.empty((n_pages * ps, H, D), dtype=torch.float32, device=dev) for _ in range(2))
        if own:
            s["cache"] = _handle(case, s["pool"], n_pages, H)
        return s
    lens = _lens(case)
    s["table"], n_pages = _table(case, lens, rng, dev)
    s["n_pages"], s["lens_host"] = n_pages, lens
    s["lens"] = torch.tensor(lens, device=dev, dtype=torch.int32)
    s["pool"] = torch.zeros(_areas(case, n_pages)[1], dtype=torch.uint8, device=dev)
    ps = case["page_size"]
    step = max(1, (1 << 26) // (H * D))
    for w in range(2):
        for at in range(0, n_pages * ps, step):                        # every page of the pool holds rows
            slots = torch.arange(at, min(at + step, n_pages * ps), device=dev)
            x = _normal(g, (slots.numel(), H, D), case["dtype"], dev)
            if w == 0:
                x[:, :, ::32] *= 4                                     # outlier channels of keys
            _store(case, s["pool"], n_pages, w, slots, x)
    if op == "read":
        s["cu"] = torch.tensor([0] + list(np.cumsum(lens)), device=dev, dtype=torch.int32)
        s["k_out"], s["v_out"] = (torch.empty((sum(lens), H, D), dtype=DT[case["dtype"]], device=dev) for _ in range(2))
        if own:
            s["cache"] = _handle(case, s["pool"], n_pages, H)
        return s
    Hq = case["Hq"]
    ql = _qlens(case) if op == "prefill" else [1] * len(lens)
    s["q"] = _normal(g, (sum(ql), Hq, D), case["dtype"], dev)
    s["cu"], s["max_q"] = torch.tensor([0] + list(np.cumsum(ql)), device=dev, dtype=torch.int32), max(ql)
    head = torch.arange(1, Hq + 1, device=dev, dtype=torch.float32)
    s["slopes"] = torch.exp2(-8.0 * head / Hq) if case["slopes"] else None
    s["prefix"] = torch.full((len(lens),), case["prefix"], device=dev, dtype=torch.int32) if case["prefix"] else None
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((sum(ql), Hq), dtype=torch.float32, device=dev)
    if own:
        s["cache"] = _handle(case, s["pool"], n_pages, Hq)
    return s


# ------------------------------------------------------------------------------------------------ plain forms
def _norm_rope(x, w, cos_sin, pos, interleaved, eps=1e-6):
    y = x.float()
    y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + eps) * w.float()
    rot = cos_sin.shape[1]
    cs = cos_sin[pos.long()][:, None]
    cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]
    if interleaved:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, y[..., rot:]), -1).to(x.dtype)


def _plain_rows(s, w, page, at):
    """Page values in fp32 as the attention takes them: 16-bit rows as they are, the others rounded to fp16."""
    c = s["case"]
    x = _load(c, s["pool"], s["n_pages"], w, page, at)
    return x if c["v_fmt" if w else "k_fmt"] in DT else x.half().float()


def _attention(s):
    """Attention of padded queries over padded rows, whole scores at once."""
    c, lens, cu = s["case"], s["lens"].long(), s["cu"].long()
    dev, ps, D, H = lens.device, c["page_size"], c["D"], c["H"]
    G, B = c["Hq"] // H, lens.numel()
    L, Q = c["longest"], s["max_q"]
    j = torch.arange(L, device=dev)
    page = s["table"].long()[:, j // ps].clamp(min=0)
    at = (j % ps).expand(B, L)
    ql = cu[1:] - cu[:-1]
    i = torch.arange(Q, device=dev)
    row = (cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][row].float().unflatten(2, (H, G))                       # [B, Q, H, G, D]
    pos = (lens - ql)[:, None] + i
    sc = torch.einsum("bihgd,bjhd->bhgij", q, _plain_rows(s, 0, page, at)) * (1.0 / math.sqrt(D))
    if c["softcap"]:
        sc = c["softcap"] * torch.tanh(sc / c["softcap"])
    dist = pos[:, :, None] - j
    if s["slopes"] is not None:
        sc = sc - s["slopes"].view(1, H, G, 1, 1) * dist.abs()[:, None, None]
    see = dist >= 0
    if c["window"]:
        see = see & (dist < c["window"])
    if c["prefix"]:
        see = see | (j < s["prefix"][:, None, None])
    see = see & (j < lens[:, None, None]) & (pos[:, :, None] >= 0)
    sc = sc.masked_fill(~see[:, None, None], -math.inf)
    top = sc.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(sc - top)
    tot = p.sum(-1, keepdim=True)
    v = _plain_rows(s, 1, page, at)
    o = torch.einsum("bhgij,bjhd->bihgd", p / torch.where(tot == 0, torch.ones_like(tot), tot), v)
    lse = (top + torch.log(tot))[..., 0].permute(0, 3, 1, 2)
    keep = i < ql[:, None]
    return o.flatten(2, 3)[keep].to(s["q"].dtype), lse.flatten(2, 3)[keep]


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        st = torch.cuda.current_stream().cuda_stream
        if op == "norm_rope":
            from quantized_kv_cache_gb300 import qk_norm_rope
            qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["cos_sin"], s["pos"], s["q_out"], s["k_out"], eps=1e-6,
                         interleaved=c["interleaved"], stream=st)
            return s["q_out"], s["k_out"]
        cache = s["cache"]
        if op == "write":
            cache.write(0, s["k"], s["v"], s["slots"], stream=st)
            if c["k_fmt"] in DT:
                return _views(c, s["pool"], s["n_pages"], 0)[0], _views(c, s["pool"], s["n_pages"], 1)[0]
            cache.read(0, s["table"], s["cu"], s["k_out"], s["v_out"], stream=st)
            return s["k_out"], s["v_out"]
        if op == "read":
            cache.read(0, s["table"], s["cu"], s["k_out"], s["v_out"], stream=st)
            return s["k_out"], s["v_out"]
        if op == "decode":
            cache.decode_attn(0, s["q"], s["table"], s["lens"], s["out"], lse=s["lse"], softcap=c["softcap"],
                              window=c["window"], slopes=s["slopes"], prefix=s["prefix"], stream=st)
        else:
            cache.prefill_attn(0, s["q"], s["cu"], s["max_q"], s["table"], s["lens"], s["out"], lse=s["lse"],
                               softcap=c["softcap"], window=c["window"], slopes=s["slopes"], prefix=s["prefix"], stream=st)
        return s["out"], s["lse"]
    if op == "norm_rope":
        return (_norm_rope(s["q"], s["wq"], s["cos_sin"], s["pos"], c["interleaved"]),
                _norm_rope(s["k"], s["wk"], s["cos_sin"], s["pos"], c["interleaved"]))
    if op == "write":
        keep = s["slots"] >= 0
        slots = s["slots"][keep].long()
        _store(c, s["pool"], s["n_pages"], 0, slots, s["k"][keep])
        _store(c, s["pool"], s["n_pages"], 1, slots, s["v"][keep])
        if c["k_fmt"] in DT:
            return _views(c, s["pool"], s["n_pages"], 0)[0], _views(c, s["pool"], s["n_pages"], 1)[0]
        every = torch.arange(s["n_pages"] * c["page_size"], device=slots.device)
        page, at = every // c["page_size"], every % c["page_size"]
        return _load(c, s["pool"], s["n_pages"], 0, page, at), _load(c, s["pool"], s["n_pages"], 1, page, at)
    if op == "read":
        cu = s["cu"].long()
        row = torch.arange(s["k_out"].shape[0], device=cu.device)
        b = torch.searchsorted(cu, row, right=True) - 1
        p = row - cu[b]
        page, at = s["table"].long()[b, p // c["page_size"]], p % c["page_size"]
        return tuple(_load(c, s["pool"], s["n_pages"], w, page, at).to(DT[c["dtype"]]) for w in range(2))
    return _attention(s)


# ------------------------------------------------------------------------------------------------ the work
def _row_bytes(case, w):
    fmt = case["v_fmt" if w else "k_fmt"]
    return case["H"] * _unit_bytes(fmt, 1, 32) * case["D"] // 32


def _visible(case):
    """(query, position) pairs that take part, over the sequences; and rows that any query sees."""
    lens = _lens(case)
    ql = _qlens(case) if case["op"] == "prefill" else [1] * len(lens)
    pairs = rows = 0
    for n, q in zip(lens, ql):
        pos = np.arange(n - q, n)
        w, x = case["window"], min(case["prefix"], n)
        lo = np.maximum(0, pos - w + 1) if w else np.zeros_like(pos)
        pairs += int((pos + 1 - lo + np.minimum(lo, x) + np.maximum(0, x - pos - 1)).sum())
        rows += min(n, n - int(lo[0]) + min(x, int(lo[0])))
    return pairs, rows


def work(case):
    op, H, D = case["op"], case["H"], case["D"]
    if op == "norm_rope":
        T, heads = case["tokens"], case["Hq"] + H
        return {"bytes": 2 * T * heads * D * 2 + T * case["rot"] * 4 + 4 * T + 4 * D,
                "flops": T * heads * (4 * D + 3 * case["rot"])}
    rb = _row_bytes(case, 0) + _row_bytes(case, 1)
    if op == "write":
        T = case["tokens"]
        n = 2 * T * H * D * 2 + 4 * T + T * rb
        if case["k_fmt"] not in DT:                       # read back: every page, as fp32
            rows = case["pages"] * case["page_size"]
            n += rows * (rb + 2 * H * D * 4)
        return {"bytes": n, "flops": 4 * T * H * D}
    if op == "read":
        rows = sum(_lens(case))
        return {"bytes": rows * (rb + 2 * H * D * 2) + 4 * (rows // case["page_size"] + 1), "flops": 2 * rows * H * D}
    T = sum(_qlens(case)) if op == "prefill" else case["seqs"]
    pairs, rows = _visible(case)
    return {"bytes": rows * rb + 4 * (rows // case["page_size"] + 1) + T * case["Hq"] * (4 * D + 4),
            "flops": 4 * pairs * case["Hq"] * D}


# ------------------------------------------------------------------------------------------------ 64 bits
def _exact_rows(s, w, pages, ps, n):
    """Page values in fp64 of positions [0, n) of a sequence with the given pages."""
    c = s["case"]
    fmt = c["v_fmt" if w else "k_fmt"]
    H, D = c["H"], c["D"]
    ub = _unit_bytes(fmt, ps, D)
    at = _areas(c, s["n_pages"])[0][w]
    raw = s["pool"][at:at + s["n_pages"] * H * ub].view(s["n_pages"], H, ub)[pages.long()]
    if fmt in DT:
        x = raw.view(DT[fmt]).reshape(len(pages), H, ps, D).double()
    else:
        nb = D if fmt == "q8_0" else D // 2
        code = raw[..., :ps * nb].reshape(len(pages), H, ps, nb)
        scale = raw[..., ps * nb:].contiguous().view(torch.float16).double()
        if fmt == "q8_0":
            q = code.contiguous().view(torch.int8).double()
        else:
            q = torch.empty((len(pages), H, ps, D), dtype=torch.float64, device=code.device)
            q[..., 0::2], q[..., 1::2] = (code % 16).double() - 8, (code // 16).double() - 8
        x = q * scale.reshape(len(pages), H, ps, D // 32).repeat_interleave(32, -1)
    return x.transpose(1, 2).reshape(len(pages) * ps, H, D)[:n]


def exact(case, seed):
    op, D, H = case["op"], case["D"], case["H"]
    s = prepare(case, seed)
    if op == "norm_rope":
        rot, cs = case["rot"], s["cos_sin"].double()[s["pos"].long()]
        outs = []
        for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
            y = x.double()
            y = y / ((y * y).sum(-1, keepdim=True) / D + 1e-6).sqrt() * w.double()
            z = y.clone()
            i = torch.arange(rot // 2, device=y.device)
            ia, ib = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + rot // 2)
            cos, sin = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
            z[..., ia] = y[..., ia] * cos - y[..., ib] * sin
            z[..., ib] = y[..., ib] * cos + y[..., ia] * sin
            outs.append(z)
        return tuple(outs)
    ps = case["page_size"]
    if op == "write":
        outs = []
        slots = s["slots"].long()
        for x, fmt in ((s["k"], case["k_fmt"]), (s["v"], case["v_fmt"])):
            x = x[slots >= 0].double()
            if fmt not in DT:                              # the definition's steps, each rounded where it says so
                b = x.reshape(x.shape[0], H, D // 32, 32)
                d = (b.abs().max(-1).values / LEVELS[fmt]).to(torch.float16).double()
                inv = torch.where(d > 0, 1 / d, torch.zeros_like(d)).float().double()
                t = (b * inv[..., None]).float().double()
                x = (t.round().clamp(-LEVELS[fmt], LEVELS[fmt]) * d[..., None]).reshape(x.shape)
            rows = torch.zeros((s["n_pages"] * ps, H, D), dtype=torch.float64, device=x.device)
            rows[slots[slots >= 0]] = x
            outs.append(rows if fmt not in DT else rows.view(s["n_pages"], ps, H, D).transpose(1, 2))
        return tuple(outs)
    if op == "read":
        return tuple(torch.cat([_exact_rows(s, w, s["table"][b, :-(-n // ps)], ps, n) for b, n in enumerate(s["lens_host"])])
                     for w in range(2))
    G, cu = case["Hq"] // H, s["cu"].tolist()
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=o.device)
    for b, n in enumerate(s["lens_host"]):
        pages = s["table"][b, :-(-n // ps)]
        k, v = (_exact_rows(s, w, pages, ps, n) for w in range(2))
        if case["k_fmt"] not in DT:                        # quantised rows enter the attention as fp16 values
            k, v = k.half().double(), v.half().double()
        pos = torch.arange(n - (cu[b + 1] - cu[b]), n, device=o.device)
        gap = pos[:, None] - torch.arange(n, device=o.device)
        hide = gap < 0
        if case["window"]:
            hide = hide | (gap >= case["window"])
        hide[:, :case["prefix"]] = False
        for h in range(case["Hq"]):
            t = s["q"][cu[b]:cu[b + 1], h].double() @ k[:, h // G].T / math.sqrt(D)
            if case["softcap"]:
                t = torch.tanh(t / case["softcap"]) * case["softcap"]
            if case["slopes"]:
                t = t - s["slopes"][h].double() * gap.abs()
            t[hide] = -math.inf
            z = torch.logsumexp(t, 1)
            lse[cu[b]:cu[b + 1], h] = z
            o[cu[b]:cu[b + 1], h] = torch.exp(t - z[:, None]) @ v[:, h // G]
    return o, lse
