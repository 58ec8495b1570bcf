"""More operators of the paged cache and what stands around it: what is measured, their plain forms and their definition in
64 bits.

Operators (case["op"]):
- "append":  key and value rows to the positions start[b].. of each sequence, in 8-bit pages with one scale for each block of 16
             positions and head; the rows of the blocks touched come back as the values that the pages hold.
- "decode":  attention of one new token per sequence over such pages.
- "chunk":   attention of a chunk of new tokens per sequence over such pages (their own rows are in the pages).
- "prompt":  causal attention over whole prompts, packed, from the projections' own rows: no cache is read.
- "rope":    RMS norm of every query and key head and a rotation whose frequencies go by the positions of several axes.
- "beams":   sequences freed and cut back, forked and made longer: pages shared, counted, copied where a shared one is written.
- "compact": the pages in use moved to the front of the pool.

8-bit pages: a pool of bytes, [256 B status | K units | V units], a unit per (page, KV head): [page_size] rows of D e4m3 codes, then
a power of two in fp32 for each 16 rows, padded to 32 bytes; each of the two areas is padded to 256 bytes. A block's power is the
smallest with the block's largest magnitude within 448 times it (2^-126 at least); it grows as rows are added, and the rows
that are there are rounded to the new one. The attentions take code x power as fp16 numbers.
"""

import math

import numpy as np
import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = 16


# ------------------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # a decode step's new rows: 32 sequences, each somewhere in a block
        dict(name="append_step", op="append", seqs=32, longest=700, new=1, H=8, D=128, page_size=16, dtype="bf16", ragged=0.9),
        # three prompts' rows stored whole
        dict(name="append_prompts", op="append", seqs=3, longest=16383, new=16383, H=4, D=256, page_size=64, dtype="f16", ragged=0.6),
        # one short sequence: the latency of a decode call
        dict(name="decode8_tiny", op="decode", seqs=1, longest=1000, Hq=4, H=2, D=128, page_size=16, dtype="f16", ragged=0.0,
             softcap=0.0, window=0, prefix=0, slopes=False),
        # a ragged batch at long contexts, the 14B shape
        dict(name="decode8_batch", op="decode", seqs=24, longest=50001, Hq=40, H=8, D=128, page_size=64, dtype="bf16",
             ragged=0.9, softcap=0.0, window=0, prefix=0, slopes=False),
        # drafted tokens of 20 sequences, looked at together by the target
        dict(name="chunk8_drafts", op="chunk", seqs=20, longest=16001, q_longest=5, Hq=40, H=8, D=128, page_size=32, dtype="f16",
             ragged=0.8, softcap=0.0, window=0, prefix=0, slopes=False),
        # the next piece of five prompts, the hybrid shape
        dict(name="chunk8_docs", op="chunk", seqs=5, longest=6000, q_longest=1501, Hq=24, H=4, D=256, page_size=64, dtype="bf16",
             ragged=0.7, softcap=30.0, window=0, prefix=0, slopes=False),
        # one short prompt: the latency of the call
        dict(name="prompt_short", op="prompt", seqs=1, longest=333, Hq=4, H=2, D=128, dtype="f16", ragged=0.0, softcap=0.0,
             window=0, prefix=0, slopes=False),
        # packed prompts of odd lengths, the 14B shape
        dict(name="prompt_packed", op="prompt", seqs=9, longest=8191, Hq=40, H=8, D=128, dtype="bf16", ragged=0.95, softcap=0.0,
             window=0, prefix=0, slopes=False),
        # a step's tokens with three axes of positions
        dict(name="rope_step", op="rope", tokens=8, Hq=40, H=8, D=128, rot=128, sections="16,24,24", cyclic=False,
             dtype="bf16", max_pos=32768),
        # the patches of some images between text: three axes, frequencies dealt out in turn
        dict(name="rope_images", op="rope", tokens=12001, Hq=24, H=4, D=256, rot=128, sections="24,20,20", cyclic=True,
             dtype="bf16", max_pos=131072),
        # 16 requests of eight beams: the beams are cut back to one each, forked anew and made longer by a token
        dict(name="beams_step", op="beams", parents=16, children=7, longest=4001, layers=8, H=8, D=128, page_size=64, spare=300,
             dtype="bf16", add=1),
        # a pool that requests have come and gone in, a third of it free
        dict(name="compact_pool", op="compact", rows=60, pages=3000, used=0.66, layers=8, H=8, D=128, page_size=16, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "chunk", "chunk", "prompt", "prompt", "rope", "beams", "compact"])
    dtype = rng.choice(["f16", "bf16"])
    D = rng.choice([64, 128, 128, 256])
    H, G = rng.choice([(2, 2), (4, 6), (8, 5), (2, 16), (8, 1), (1, 8), (3, 3)])
    c = dict(op=op, H=H, D=D, dtype=dtype)
    if op == "rope":
        rot = rng.choice([D, D // 2])
        axes = rng.choice([2, 3, 3, 4])
        cut = sorted(rng.sample(range(1, rot // 2), axes - 1))
        sections = [b - a for a, b in zip([0] + cut, cut + [rot // 2])]
        c.update(tokens=_log(rng, 1, 8191), Hq=H * G, rot=rot, sections=",".join(map(str, sections)), cyclic=rng.random() < 0.5,
                 max_pos=rng.choice([32768, 131072]))
        return c
    if op == "beams":
        c.update(parents=_log(rng, 1, 20), children=_log(rng, 1, 7), longest=_log(rng, 1, 3000), layers=rng.choice([1, 4]), H=rng.choice([2, 4, 8]),
                 page_size=rng.choice([16, 32, 64, 128]), add=_log(rng, 1, 70))
        c["spare"] = c["parents"] * (c["children"] + 1) * (2 + c["add"] // c["page_size"])
        return c
    if op == "compact":
        c.update(rows=_log(rng, 1, 100), pages=_log(rng, 4, 2500), used=rng.choice([0.1, 0.5, 0.8, 0.97]), layers=rng.choice([1, 3, 6]),
                 page_size=rng.choice([16, 32]), H=rng.choice([1, 2, 4]))
        return c
    c.update(seqs=_log(rng, 1, 24), ragged=rng.choice([0.0, 0.5, 0.95]), page_size=rng.choice([16, 32, 64, 128]))
    if op == "append":
        c["longest"] = max(2, _log(rng, 2, 30000) // c["seqs"])
        c["new"] = min(c["longest"], _log(rng, 1, c["longest"]))
        return c
    c.update(Hq=H * G, softcap=rng.choice([0.0, 0.0, 30.0]), window=rng.choice([0, 0, 500]), prefix=rng.choice([0, 0, 37]),
             slopes=rng.random() < 0.3)
    if op == "decode":
        c["longest"] = max(1, _log(rng, 8, 262144) // c["seqs"])
    elif op == "chunk":
        c["q_longest"] = max(1, _log(rng, 1, 4096) // c["seqs"])
        c["longest"] = c["q_longest"] + _log(rng, 1, 16384) // c["seqs"]
    else:
        del c["page_size"]
        c["longest"] = max(1, _log(rng, 1, 8191) // min(c["seqs"], 4))
    return c


# ------------------------------------------------------------------------------------------------ inputs
def _lens(case):
    """Lengths from the case alone: the longest first, the others between (1 - ragged) of it and it."""
    n, m, r = case["seqs"], case["longest"], case["ragged"]
    rng = np.random.default_rng(n * 1000003 + m)
    u = rng.random(n)
    u[0] = 0.0
    return [max(1, int(m * (1 - r * x))) for x in u]


def _qlens(case):
    lens = _lens(case)
    if case["op"] == "prompt":
        return lens
    if case["op"] == "decode":
        return [1] * len(lens)
    q = case["new" if case["op"] == "append" else "q_longest"]
    return [max(1, min(n, int(round(q * n / lens[0])))) for n in lens]


def _unit_bytes(ps, D):
    return ps * D + max(32, ps // BLOCK * 4)


def _areas(case, n_pages):
    """Byte offsets of the K and V areas, and the pool's size."""
    n = -(-n_pages * case["H"] * _unit_bytes(case["page_size"], case["D"]) // 256) * 256
    return [256, 256 + n], 256 + 2 * n


def _views(case, pool, n_pages, w):
    """Codes [pages, H, page_size, D] and scales [pages, H, page_size / 16] of the K (w = 0) or V (w = 1) area."""
    H, D, ps = case["H"], case["D"], case["page_size"]
    ub = _unit_bytes(ps, D)
    at = _areas(case, n_pages)[0][w]
    u = pool[at:at + n_pages * H * ub].view(n_pages, H, ub)
    scales = u[:, :, ps * D:ps * D + ps // BLOCK * 4].view(torch.float32)
    return u[:, :, :ps * D].unflatten(2, (ps, D)), scales


def _power(amax):
    """Exponent of the smallest power of two that amax / 448 does not exceed, -126 at least."""
    m, x = torch.frexp(amax)
    e = x - 9 + (m > 0.875)
    return torch.where(amax > 0, e, torch.full_like(e, -126)).clamp(min=-126)


def _two(e):
    """2^e in fp32, e from -126 to 127."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _code(x):
    return x.to(torch.float8_e4m3fn).view(torch.uint8)


def _value(c):
    return c.view(torch.float8_e4m3fn).float()


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


def _normal(g, shape, dtype, dev):
    return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(DT[dtype])


def _ints(x, dev):
    return torch.tensor(x, device=dev, dtype=torch.int32)


def _cache(case, pool, n_pages, fmt="e4m3", layers=1):
    from quantized_kv_cache_gb300 import PagedKVCache, paged_config
    cfg = paged_config(n_layers=layers, n_kv_heads=case["H"], head_dim=case["D"], n_q_heads=case.get("Hq", case["H"]),
                       page_size=case["page_size"], n_pages=n_pages, k_fmt=fmt)
    return PagedKVCache(cfg, pool.device.index, max_seqs=case.get("seqs", 1),
                        max_tokens=case.get("seqs", 1) * case.get("q_longest", 1), pool=pool)


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev).manual_seed(seed)
    rng = np.random.default_rng(seed)
    op, H, D = case["op"], case["H"], case["D"]
    s = {"case": case}
    if op in ("beams", "compact"):
        return _prepare_pages(case, s, g, rng, dev)
    if op == "rope":
        T, Hq, rot = case["tokens"], case["Hq"], case["rot"]
        qkv = _normal(g, (T, Hq + 2 * H, D), case["dtype"], dev)     # one projection's output, V beside Q and K
        s["q"], s["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + H]
        s["wq"], s["wk"] = (1 + 0.1 * _normal(g, (2, D), "f32", dev)).to(DT[case["dtype"]]).unbind(0)
        i = torch.arange(rot // 2, device=dev, dtype=torch.float64)
        ang = torch.arange(case["max_pos"], device=dev, dtype=torch.float64)[:, None] * 1e6 ** (-2 * i / rot)
        s["cos_sin"] = torch.cat((ang.cos(), ang.sin()), 1).float()
        s["sections"] = tuple(map(int, case["sections"].split(",")))
        # a frame's number, and a patch's row and column
        t = torch.arange(T, device=dev)
        p0 = int(rng.integers(0, case["max_pos"] - T))
        axes = [p0 + t // 97] + [p0 + t // (7 * a + 1) % 61 for a in range(len(s["sections"]) - 1)]
        s["pos"] = torch.stack(axes).to(torch.int32)
        s["q_out"], s["k_out"] = (torch.empty((T, n, D), dtype=DT[case["dtype"]], device=dev) for n in (Hq, H))
        return s
    lens, ql = _lens(case), _qlens(case)
    s["lens_host"], s["q_host"] = lens, ql
    s["lens"] = _ints(lens, dev)
    s["cu"], s["max_q"] = _ints([0] + list(np.cumsum(ql)), dev), max(ql)
    if op != "append":
        Hq = case["Hq"]
        head = torch.arange(1, Hq + 1, device=dev, dtype=torch.float32)
        s["slopes"] = torch.exp2(-8.0 * head / Hq) if case["slopes"] else None
        s["prefix"] = torch.full((len(lens),), case["prefix"], device=dev, dtype=torch.int32) if case["prefix"] else None
        s["out"] = torch.empty((sum(ql), Hq, D), dtype=DT[case["dtype"]], device=dev)
        s["lse"] = torch.empty((sum(ql), Hq), dtype=torch.float32, device=dev)
    if op == "prompt":
        qkv = _normal(g, (sum(ql), Hq + 2 * H, D), case["dtype"], dev)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
        if own:
            from quantized_kv_cache_gb300 import prompt_workspace
            s["ws"] = prompt_workspace(sum(ql), Hq, D, dev)
        return s
    s["table"], n_pages = _table(case, lens, rng, dev)
    s["n_pages"] = n_pages
    s["pool"] = torch.zeros(_areas(case, n_pages)[1], dtype=torch.uint8, device=dev)
    ps = case["page_size"]
    step = max(1, (1 << 25) // (H * ps * D))
    for w in range(2):
        codes, scales = _views(case, s["pool"], n_pages, w)
        for at in range(0, n_pages, step):                             # every page of the pool holds rows
            x = torch.randn((min(step, n_pages - at), H, ps // BLOCK, BLOCK, D), generator=g, device=dev)
            if w == 0:
                x[..., ::32] *= 4                                      # outlier channels of keys
            e = _power(x.abs().amax((3, 4)))
            codes[at:at + step] = _code(x * _two(-e)[..., None, None]).flatten(2, 3)
            scales[at:at + step] = _two(e)
    if op == "append":
        kv = 1.5 * torch.randn((sum(ql), 2 * H, D), generator=g, device=dev)
        kv[:, :H, ::32] *= 4
        kv = kv.to(DT[case["dtype"]])
        s["k"], s["v"] = kv[:, :H], kv[:, H:]
        start = [n - q for n, q in zip(lens, ql)]
        s["start_host"], s["start"] = start, _ints(start, dev)
        first = [x // BLOCK * BLOCK for x in start]
        back = [n - f for n, f in zip(lens, first)]
        s["first_host"], s["first"], s["back"] = first, _ints(first, dev), _ints([0] + list(np.cumsum(back)), dev)
        s["k_out"], s["v_out"] = (torch.empty((sum(back), H, D), dtype=torch.float32, device=dev) for _ in range(2))
    else:
        s["q"] = _normal(g, (sum(ql), Hq, D), case["dtype"], dev)
    if own:
        s["cache"] = _cache(case, s["pool"], n_pages)
    return s


def _prepare_pages(case, s, g, rng, dev):
    H, D, ps, layers = case["H"], case["D"], case["page_size"], case["layers"]
    if case["op"] == "beams":
        P, C = case["parents"], case["children"]
        R = P * (C + 1)
        lens = np.zeros(R, np.int32)
        lens[:P] = np.maximum(1, (case["longest"] * (1 - 0.9 * np.random.default_rng(P * 1009 + C).random(P))).astype(np.int32))
        lens[0] = case["longest"]
        need = -(-lens // ps)
        n_pages = int(need.sum()) + case["spare"]
        width = int(need.max()) + 2 + case["add"] // ps
    else:
        R, n_pages = case["rows"], case["pages"]
        used = max(1, int(n_pages * case["used"]))
        R = min(R, used)
        need = np.full(R, used // R)
        need[:used % R] += 1
        lens = (need * ps - np.random.default_rng(n_pages).integers(0, ps, R)).astype(np.int32)
        width = int(need.max()) + 1
    table = np.full((R, width), -1, np.int32)
    refs = np.zeros(n_pages, np.int32)
    order, at = rng.permutation(n_pages), 0
    for b in range(R):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    refs[order[:at]] = 1
    page = H * ps * D
    half = -(-n_pages * page * 2 // 256) * 256
    s["pool"] = torch.zeros(256 + 2 * layers * half, dtype=torch.uint8, device=dev)
    s["areas"] = []                                                    # K and V of each layer: [pages, values of a page]
    for i in range(2 * layers):
        v = s["pool"][256 + i * half:256 + i * half + n_pages * page * 2].view(DT[case["dtype"]]).view(n_pages, page)
        v.copy_(torch.randn((n_pages, page), generator=g, device=dev))
        s["areas"].append(v)
    s["table"], s["lens"], s["refs"] = (torch.from_numpy(x).to(dev) for x in (table, lens, refs))
    s["host"] = (table.copy(), lens.copy(), refs.copy())
    if case["op"] == "beams":
        rows = np.arange(R)
        s["rows"], s["keep"] = _ints(rows.tolist(), dev), _ints(lens.tolist(), dev)
        s["parents"], s["children"] = _ints((rows[P:] - P) // C, dev), _ints(rows[P:].tolist(), dev)
        s["add"] = torch.full((R,), case["add"], dtype=torch.int32, device=dev)
    else:
        s["table0"], s["refs0"] = s["table"].clone(), s["refs"].clone()
        s["remap"] = torch.empty(n_pages, dtype=torch.int32, device=dev)
    if own:
        s["cache"] = _cache(case, s["pool"], n_pages, case["dtype"], layers)
    return s


# ------------------------------------------------------------------------------------------------ plain forms
def _axis_of(sections, cyclic):
    """The axis of each frequency: in runs, or dealt out in turn until an axis has its number."""
    if not cyclic:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    left, out = list(sections), []
    while any(left):
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                out.append(a)
    return out


def _norm_rope(x, w, cos, sin, eps=1e-6):
    y = x.float()
    y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + eps) * w.float()
    n = cos.shape[-1]
    a, b = y[..., :n], y[..., n:2 * n]
    return torch.cat((a * cos - b * sin, b * cos + a * sin, y[..., 2 * n:]), -1).to(x.dtype)


def _plain_rope(s):
    n = s["cos_sin"].shape[1] // 2
    axis = torch.tensor(_axis_of(s["sections"], s["case"]["cyclic"]), device=s["q"].device)
    at = s["pos"].long()[axis].T                                       # [tokens, frequencies]
    i = torch.arange(n, device=at.device)
    cos, sin = s["cos_sin"][at, i][:, None], s["cos_sin"][at, n + i][:, None]
    return _norm_rope(s["q"], s["wq"], cos, sin), _norm_rope(s["k"], s["wk"], cos, sin)


def _plain_append(s):
    c, ps = s["case"], s["case"]["page_size"]
    per = ps // BLOCK
    cu, start, table = s["cu"].long(), s["start"].long(), s["table"].long()
    dev = cu.device
    row = torch.arange(s["k"].shape[0], device=dev)
    b = torch.searchsorted(cu, row, right=True) - 1
    pos = start[b] + row - cu[b]
    page, at = table[b, pos // ps], pos % ps
    block = page * per + at // BLOCK
    # the rows that are there in the block of each sequence's first new one
    first = start // BLOCK * BLOCK
    j = torch.arange(BLOCK, device=dev)
    old = first[:, None] + j < start[:, None]
    page0 = table.gather(1, (first // ps)[:, None])[:, 0]
    block0 = page0 * per + first % ps // BLOCK
    at0 = (first % ps)[:, None] + j
    for w, x in enumerate((s["k"], s["v"])):
        codes, scales = _views(c, s["pool"], s["n_pages"], w)
        x = x.float()
        H = x.shape[1]
        e = _power(x.abs().amax(2))
        top = torch.full((s["n_pages"] * per, H), -126, dtype=e.dtype, device=dev)
        held = torch.frexp(scales[page0, :, first % ps // BLOCK])[1] - 1
        top[block0] = torch.where((start > first)[:, None], held, top[block0])
        top.scatter_reduce_(0, block[:, None].expand(-1, H), e, "amax")
        new = top[block0]
        was = _value(codes[page0].gather(2, at0[:, None, :, None].expand(-1, H, -1, c["D"])))
        now = _code(was * _two((held - new).clamp(min=-126))[:, :, None, None])
        keep = codes[page0[:, None], :, at0]                           # [sequences, 16, H, D]
        codes[page0[:, None], :, at0] = torch.where(old[:, :, None, None], now.transpose(1, 2), keep)
        codes[page, :, at] = _code(x * _two(-top[block])[..., None])
        scales[page, :, at // BLOCK] = _two(top[block])
    cu, row = s["back"].long(), torch.arange(s["k_out"].shape[0], device=dev)
    b = torch.searchsorted(cu, row, right=True) - 1
    pos = first[b] + row - cu[b]
    return tuple(_plain_rows(s, w, table[b, pos // ps], pos % ps) for w in range(2))


def _plain_rows(s, w, page, at):
    codes, scales = _views(s["case"], s["pool"], s["n_pages"], w)
    return _value(codes.movedim(2, 1)[page, at]) * scales.movedim(2, 1)[page, at // BLOCK][..., None]


def _softmax(s, sc, dist, hide):
    """Weights and log-sum-exp over the last axis of scores [.., H, G, queries, positions]."""
    c = s["case"]
    if c["softcap"]:
        sc = c["softcap"] * torch.tanh(sc / c["softcap"])
    if s["slopes"] is not None:
        sc = sc - s["slopes"].view(c["H"], -1, 1, 1) * dist.abs()
    sc = sc.masked_fill_(hide, -math.inf)
    top = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - top)
    tot = p.sum(-1, keepdim=True)
    return p.div_(tot), (top + torch.log(tot))[..., 0]


def _hidden(s, pos, n, prefix):
    """What the query at each position does not see of n positions."""
    j = torch.arange(n, device=pos.device)
    dist = pos[..., None] - j
    hide = dist < 0
    if s["case"]["window"]:
        hide = hide | (dist >= s["case"]["window"])
    if prefix is not None:
        hide = hide & (j >= prefix)
    return dist, hide


def _plain_pages(s):
    """Attention of padded queries over padded page rows, whole scores at once."""
    c, lens, cu = s["case"], s["lens"].long(), s["cu"].long()
    dev, ps, D, H = lens.device, c["page_size"], c["D"], c["H"]
    G, B, L, Q = c["Hq"] // H, lens.numel(), c["longest"], s["max_q"]
    j = torch.arange(L, device=dev)
    page = s["table"].long()[:, j // ps].clamp(min=0)
    at = (j % ps).expand(B, L)
    ql = cu[1:] - cu[:-1]
    i = torch.arange(Q, device=dev)
    row = (cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][row].float().unflatten(2, (H, G))                       # [B, Q, H, G, D]
    pos = (lens - ql)[:, None] + i
    sc = torch.einsum("bihgd,bjhd->bhgij", q, _plain_rows(s, 0, page, at).half().float()) * (1.0 / math.sqrt(D))
    dist, hide = _hidden(s, pos, L, None if s["prefix"] is None else s["prefix"][:, None, None])
    hide = hide | (j >= lens[:, None, None])
    p, lse = _softmax(s, sc, dist[:, None, None], hide[:, None, None])
    o = torch.einsum("bhgij,bjhd->bihgd", p, _plain_rows(s, 1, page, at).half().float())
    keep = i < ql[:, None]
    return o.flatten(2, 3)[keep].to(s["q"].dtype), lse.permute(0, 3, 1, 2).flatten(2, 3)[keep]


def _plain_prompt(s):
    """Attention prompt by prompt, whole scores of some heads at once."""
    c, out, lse = s["case"], s["out"], s["lse"]
    H, D = c["H"], c["D"]
    G, at = c["Hq"] // H, 0
    for b, n in enumerate(s["q_host"]):
        q, k, v = (x[at:at + n].float() for x in (s["q"], s["k"], s["v"]))
        pos = torch.arange(n, device=q.device)
        dist, hide = _hidden(s, pos, n, None if s["prefix"] is None else s["prefix"][b])
        q = q.unflatten(1, (H, G))
        sc = torch.einsum("ihgd,jhd->hgij", q, k) * (1.0 / math.sqrt(D))
        p, z = _softmax(s, sc, dist, hide)
        out[at:at + n] = torch.einsum("hgij,jhd->ihgd", p, v).flatten(1, 2).to(out.dtype)
        lse[at:at + n] = z.permute(2, 0, 1).flatten(1, 2)
        at += n
    return out, lse


def _counted(s, page, on, by):
    """refs[page] += by where `on` (several entries may name a page)."""
    n = s["refs"].numel()
    at = torch.where(on, page, torch.full_like(page, n)).flatten()     # the others go behind the end
    s["refs"] += _times(at, n)[:n] * by


def _times(at, n):
    """How often each number up to n comes."""
    return torch.zeros(n + 1, dtype=torch.int32, device=at.device).scatter_add_(0, at, torch.ones_like(at, dtype=torch.int32))


def _free_pages(refs):
    """Pages in the order: free ones by number, then the others."""
    return torch.argsort((refs > 0).to(torch.int32), stable=True)


def _plain_beams(s):
    ps = s["case"]["page_size"]
    table, lens, refs = s["table"], s["lens"], s["refs"]
    R, W = table.shape
    n = refs.numel()
    e = torch.arange(W, device=table.device)
    # freed and cut back
    keep = torch.minimum(lens, s["keep"])
    gone = (e >= ((keep + ps - 1) // ps)[:, None]) & (table >= 0)
    _counted(s, table.long().clamp(min=0), gone, -1)
    table.copy_(torch.where(gone, torch.full_like(table, -1), table))
    lens.copy_(keep)
    # forked: pages shared
    pa, ch = s["parents"].long(), s["children"].long()
    _counted(s, table[pa].long().clamp(min=0), table[pa] >= 0, 1)
    table[ch] = table[pa]
    lens[ch] = lens[pa]
    # longer: a part-filled page that others hold too is copied, except by the lowest of its rows if all of them go on
    have = (lens + ps - 1) // ps
    want = (lens + s["add"] + ps - 1) // ps
    part = (lens % ps > 0) & (s["add"] > 0)
    last = table.gather(1, (have - 1).clamp(min=0)[:, None].long())[:, 0].long()
    key = torch.where(part, last, torch.full_like(last, n))
    going = _times(key, n)[key]
    row = torch.arange(R, device=table.device)
    lowest = torch.full((n + 1,), R, device=table.device).scatter_reduce_(0, key, row, "amin")[key]
    copied = part & ((going < refs[last.clamp(max=n - 1)]) | (row != lowest))
    need = (want - have) + copied
    first = torch.cumsum(need, 0) - need
    free = _free_pages(refs)
    dst = torch.where(copied, free[first.clamp(max=n - 1).long()], last)
    for v in s["areas"]:
        v[dst] = v[last]                                               # without a copy: the page onto itself
    new = (e >= have[:, None]) & (e < want[:, None])
    k = (first + copied)[:, None] + e - have[:, None]
    table.copy_(torch.where(new, free[k.clamp(0, n - 1).long()].to(torch.int32), table))
    at = (have - 1).clamp(min=0)[:, None].long()
    table.scatter_(1, at, torch.where(copied, dst.to(torch.int32), table.gather(1, at)[:, 0])[:, None])
    _counted(s, last.clamp(max=n - 1), copied, -1)
    _counted(s, torch.where(copied, dst, 0), copied, 1)
    _counted(s, table.long().clamp(min=0), new, 1)
    lens += s["add"]
    return [table, lens, refs] + s["areas"]


def _plain_compact(s):
    ps = s["case"]["page_size"]
    table, refs, remap = s["table"], s["refs"], s["remap"]
    table.copy_(s["table0"])
    refs.copy_(s["refs0"])
    used = refs > 0
    live = used.sum()
    p = torch.arange(refs.numel(), device=refs.device)
    mover, hole = used & (p >= live), ~used & (p < live)
    movers, holes = (torch.argsort((~x).to(torch.int32), stable=True) for x in (mover, hole))
    to = torch.where(mover, holes[(torch.cumsum(mover, 0) - 1).clamp(min=0)], p)
    come = torch.where(hole, movers[(torch.cumsum(hole, 0) - 1).clamp(min=0)], p)
    for v in s["areas"]:
        v.copy_(v[come])
    remap.copy_(torch.where(used, to, torch.full_like(p, -1)))
    refs.copy_(torch.where(p < live, refs[come], 0))
    e = torch.arange(table.shape[1], device=table.device)
    held = e < ((s["lens"] + ps - 1) // ps)[:, None]
    table.copy_(torch.where(held, remap[table.long().clamp(min=0)], table))
    return [table, refs, remap] + s["areas"]


def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        if op == "rope":
            return _plain_rope(s)
        if op == "append":
            return _plain_append(s)
        if op == "prompt":
            return _plain_prompt(s)
        if op == "beams":
            return _plain_beams(s)
        if op == "compact":
            return _plain_compact(s)
        return _plain_pages(s)
    st = torch.cuda.current_stream().cuda_stream
    if op == "rope":
        from quantized_kv_cache_gb300 import qk_norm_rope
        qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["cos_sin"], s["pos"], s["q_out"], s["k_out"], eps=1e-6,
                     sections=s["sections"], cyclic=c["cyclic"], stream=st)
        return s["q_out"], s["k_out"]
    if op == "prompt":
        from quantized_kv_cache_gb300 import prompt_attn
        prompt_attn(s["q"], s["k"], s["v"], s["cu"], s["max_q"], s["out"], s["ws"], lse=s["lse"], softcap=c["softcap"],
                    window=c["window"], slopes=s["slopes"], prefix=s["prefix"], stream=st)
        return s["out"], s["lse"]
    cache = s["cache"]
    if op == "append":
        cache.append(0, s["k"], s["v"], s["table"], s["cu"], s["start"], stream=st)
        cache.read(0, s["table"], s["back"], s["k_out"], s["v_out"], start=s["first"], stream=st)
        return s["k_out"], s["v_out"]
    if op == "beams":
        cache.free(s["table"], s["lens"], s["refs"], s["rows"], s["keep"], stream=st)
        cache.fork(s["table"], s["lens"], s["refs"], s["parents"], s["children"], stream=st)
        cache.extend(s["table"], s["lens"], s["refs"], s["add"], stream=st)
        return [s["table"], s["lens"], s["refs"]] + s["areas"]
    if op == "compact":
        s["table"].copy_(s["table0"])
        s["refs"].copy_(s["refs0"])
        cache.compact(s["table"], s["lens"], s["refs"], s["remap"], stream=st)
        return [s["table"], s["refs"], s["remap"]] + s["areas"]
    if op == "decode":
        cache.decode_attn(0, s["q"], s["table"], s["lens"], s["out"], lse=s["lse"], softcap=c["softcap"], window=c["window"],
                          slopes=s["slopes"], prefix=s["prefix"], stream=st)
    else:
        cache.prefill_attn(0, s["q"], s["cu"], s["max_q"], s["table"], s["lens"], s["out"], lse=s["lse"],
                           softcap=c["softcap"], window=c["window"], slopes=s["slopes"], prefix=s["prefix"], stream=st)
    return s["out"], s["lse"]


# ------------------------------------------------------------------------------------------------ the work
def _visible(case):
    """(query, position) pairs that take part, over the sequences; and rows that any query sees."""
    pairs = rows = 0
    for n, q in zip(_lens(case), _qlens(case)):
        pos = np.arange(n - q, n)
        w, x = case["window"], min(case["prefix"], n)
        lo = np.maximum(0, pos - w + 1) if w else np.zeros_like(pos)
        pairs += int((pos + 1 - lo + np.minimum(lo, x) + np.maximum(0, x - pos - 1)).sum())
        rows += min(n, n - int(lo[0]) + min(x, int(lo[0])))
    return pairs, rows


def _page_counts(case):
    """Pages copied by "beams" and by "compact", from the lengths and the counts that a case has."""
    ps = case["page_size"]
    if case["op"] == "beams":
        P, C = case["parents"], case["children"]
        lens = np.maximum(1, (case["longest"] * (1 - 0.9 * np.random.default_rng(P * 1009 + C).random(P))).astype(np.int32))
        lens[0] = case["longest"]
        return int((lens % ps > 0).sum()) * C
    used = max(1, int(case["pages"] * case["used"]))
    return int(used * (case["pages"] - used) / case["pages"])          # movers, on the mean


def work(case):
    op, H, D = case["op"], case["H"], case["D"]
    if op == "rope":
        T, heads = case["tokens"], case["Hq"] + H
        axes = case["sections"].count(",") + 1
        return {"bytes": 2 * T * heads * D * 2 + T * case["rot"] * 4 + 4 * T * axes + 4 * D, "flops": T * heads * (4 * D + 3 * case["rot"])}
    if op in ("beams", "compact"):
        page = 2 * case["layers"] * H * case["page_size"] * D * 2
        n = 2 * page * _page_counts(case) + 4 * (case["pages"] if op == "compact" else case["spare"])
        return {"bytes": n, "flops": n // 16}
    row = 2 * H * (D + 4 / BLOCK)                                      # K and V of a position in the pages
    if op == "append":
        T = sum(_qlens(case))
        back = sum(n - (n - q) // BLOCK * BLOCK for n, q in zip(_lens(case), _qlens(case)))
        return {"bytes": int(2 * T * H * D * 2 + T * row + back * (row + 2 * H * D * 4)), "flops": 6 * T * H * D}
    T = sum(_qlens(case))
    pairs, rows = _visible(case)
    kv = T * 4 * H * D if op == "prompt" else int(rows * row) + 4 * (rows // case["page_size"] + 1)
    return {"bytes": kv + T * case["Hq"] * (4 * D + 4), "flops": 4 * pairs * case["Hq"] * D}


# ------------------------------------------------------------------------------------------------ 64 bits
def _exact_code(v):
    """fp64 values (448 at most) to the nearest e4m3 numbers, ties to even."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -30))).clamp(min=-6.0)
    e = torch.where(v.abs() >= torch.exp2(e + 1), e + 1, e)
    step = torch.exp2(e - 3)
    return torch.round(v / step) * step


def _exact_values(raw, ps, D):
    """Units as bytes [n, H, unit] to codes' values [n, H, ps, D] and powers [n, H, ps / 16], fp64."""
    b = raw[..., :ps * D].reshape(*raw.shape[:2], ps, D).to(torch.int32)
    x, m = b // 8 % 16, (b % 8).double()
    v = torch.where(x == 0, m * 2.0 ** -9, (1 + m / 8) * torch.exp2((x - 7).double()))
    v = torch.where(b >= 128, -v, v)
    s = raw[..., ps * D:ps * D + ps // BLOCK * 4].contiguous().view(torch.float32).double()
    return v, s


def _exact_unit(s, w, pages):
    c = s["case"]
    H, D, ps = c["H"], c["D"], c["page_size"]
    ub, at = _unit_bytes(ps, D), _areas(c, s["n_pages"])[0][w]
    return _exact_values(s["pool"][at:at + s["n_pages"] * H * ub].view(s["n_pages"], H, ub)[pages.long()], ps, D)


def _exact_append(case, s):
    ps, cu, outs = case["page_size"], s["cu"].tolist(), []
    for w, x in enumerate((s["k"], s["v"])):
        rows = []
        for b, n in enumerate(s["lens_host"]):
            start, first = s["start_host"][b], s["first_host"][b]
            v, power = _exact_unit(s, w, s["table"][b, first // ps:-(-n // ps)])
            v = v.transpose(1, 2).reshape(-1, v.shape[1], v.shape[3])                  # [rows, H, D] from a page's start
            power = power.transpose(1, 2).reshape(-1, power.shape[1])                  # [blocks, H]
            skip = first % ps
            held = power[skip // BLOCK]
            v = torch.cat((v[skip:skip + start - first] * held[:, None], x[cu[b]:cu[b + 1]].double()))
            for at in range(0, n - first, BLOCK * 4096):                               # by blocks from the first one on
                y = v[at:at + BLOCK * 4096]
                pad = -len(y) % BLOCK
                z = torch.cat((y, y.new_zeros(pad, *y.shape[1:]))).unflatten(0, (-1, BLOCK))
                z0 = z.clone()
                if at == 0:
                    z0[0, :start - first] = 0                                          # rows that are there: their power holds them
                top = z0.abs().amax((1, 3)) / 448
                p = torch.exp2(torch.ceil(torch.log2(top.clamp(min=2.0 ** -126))))
                p = torch.where(p / 2 >= top, p / 2, p)
                p = torch.where(p < top, p * 2, p).clamp(min=2.0 ** -126)
                if at == 0 and start > first:
                    p[0] = torch.maximum(p[0], held)
                z = _exact_code(z / p[:, None, :, None]) * p[:, None, :, None]
                rows.append(z.flatten(0, 1)[:len(y)])
        outs.append(torch.cat(rows))
    return tuple(outs)


def _exact_attention(case, s):
    H, D, G, cu = case["H"], case["D"], case["Hq"] // case["H"], s["cu"].tolist()
    ps = case.get("page_size")
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=o.device)
    for b, n in enumerate(s["lens_host"]):
        if ps:
            kv = []
            for w in range(2):
                v, power = _exact_unit(s, w, s["table"][b, :-(-n // ps)])
                v = (v * power.repeat_interleave(BLOCK, 2)[..., None]).half().double()     # they enter as fp16 numbers
                kv.append(v.transpose(1, 2).reshape(-1, H, D)[:n])
        else:
            kv = [s[x][cu[b]:cu[b + 1]].double() for x in "kv"]
        pos = torch.arange(n - (cu[b + 1] - cu[b]), n, device=o.device)
        gap = pos[:, None] - torch.arange(n, device=o.device)
        hide = gap < 0
        if case["window"]:
            hide = hide | (gap >= case["window"])
        hide[:, :case["prefix"]] = False
        for h in range(case["Hq"]):
            t = s["q"][cu[b]:cu[b + 1], h].double() @ kv[0][:, h // G].T / math.sqrt(D)
            if case["softcap"]:
                t = torch.tanh(t / case["softcap"]) * case["softcap"]
            if case["slopes"]:
                t = t - s["slopes"][h].double() * gap.abs()
            t[hide] = -math.inf
            z = torch.logsumexp(t, 1)
            lse[cu[b]:cu[b + 1], h] = z
            o[cu[b]:cu[b + 1], h] = torch.exp(t - z[:, None]) @ kv[1][:, h // G]
    return o, lse


def _exact_rope(case, s):
    rot, outs, axis, taken = case["rot"], [], [], [0] * len(s["sections"])
    if case["cyclic"]:
        a = 0
        while len(axis) < rot // 2:
            if taken[a] < s["sections"][a]:
                taken[a] += 1
                axis.append(a)
            a = (a + 1) % len(taken)
    else:
        ends = np.cumsum(s["sections"])
        axis = [int((i >= ends).sum()) for i in range(rot // 2)]
    cs, pos = s["cos_sin"].double(), s["pos"].long()
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        y = x.double()
        y = y / ((y * y).sum(-1, keepdim=True) / case["D"] + 1e-6).sqrt() * w.double()
        z = y.clone()
        for i, a in enumerate(axis):
            cos, sin = cs[pos[a], i][:, None], cs[pos[a], rot // 2 + i][:, None]
            z[..., i] = y[..., i] * cos - y[..., i + rot // 2] * sin
            z[..., i + rot // 2] = y[..., i + rot // 2] * cos + y[..., i] * sin
        outs.append(z)
    return tuple(outs)


def _exact_pages(case, s):
    """The counts and tables worked out row by row on the host, the pages by the list of copies."""
    table, lens, refs = (x.tolist() for x in s["host"])
    ps, moves = case["page_size"], []
    if case["op"] == "beams":
        P, C, add = case["parents"], case["children"], case["add"]
        for i in range(P * C):                                         # forked (nothing is there to be freed at first)
            p, c = i // C, P + i
            table[c], lens[c] = list(table[p]), lens[p]
            for x in table[p]:
                if x >= 0:
                    refs[x] += 1
        before = list(refs)
        going = {}
        for r, n in enumerate(lens):
            if n % ps:
                going.setdefault(table[r][n // ps], []).append(r)
        free = iter([x for x, k in enumerate(before) if k == 0])
        for r, n in enumerate(lens):
            if n % ps:
                x = table[r][n // ps]
                if not (len(going[x]) == before[x] and going[x][0] == r):
                    y = next(free)
                    moves.append((x, y))
                    refs[x] -= 1
                    refs[y] += 1
                    table[r][n // ps] = y
            for e in range(-(-n // ps), -(-(n + add) // ps)):
                table[r][e] = next(free)
                refs[table[r][e]] += 1
            lens[r] = n + add
        ints = [table, lens, refs]
    else:
        live = sum(k > 0 for k in refs)
        holes = [x for x in range(live) if refs[x] == 0]
        remap = [x if k > 0 else -1 for x, k in enumerate(refs)]
        for x in range(live, len(refs)):
            if refs[x] > 0:
                y = holes.pop(0)
                moves.append((x, y))
                remap[x], refs[y], refs[x] = y, refs[x], 0
        for r, n in enumerate(lens):
            for e in range(-(-n // ps)):
                table[r][e] = remap[table[r][e]]
        ints = [table, refs, remap]
    out = [torch.tensor(x, dtype=torch.int32, device=s["refs"].device) for x in ints]
    for v in s["areas"]:
        y = v.double()
        if moves:
            y[[d for _, d in moves]] = v[[x for x, _ in moves]].double()
        out.append(y)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(case, s)
    if case["op"] in ("beams", "compact"):
        return _exact_pages(case, s)
    return _exact_append(case, s) if case["op"] == "append" else _exact_attention(case, s)
