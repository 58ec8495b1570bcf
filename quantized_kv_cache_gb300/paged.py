"""The paged KV cache on PyTorch CUDA tensors: rows to pages, back from them, and attention over them.

``PagedKVCache`` owns (or takes) a pool of pages and a workspace and forwards to the C ABI of
``include/kvq_paged.h``; ``qk_norm_rope`` needs no cache. The tensors are checked here (device, type,
shape, strides) and an argument that does not fit raises ``ValueError`` before anything is enqueued;
what the C side refuses raises ``KVQError``. Nothing here has a gradient: where autograd records, a tensor that
requires one raises ``ValueError`` too (``torch.no_grad()`` or ``detach()`` says that none is wanted), and tensors that a
call writes count as changed in place. As in ``KVCache``, ``stream`` is a raw CUDA stream handle
and 0 the legacy default stream; a caller on another stream passes its handle
(``torch.cuda.current_stream().cuda_stream``) and keeps the tensors alive until the work is done.
Page tables, lengths, slots, offsets and positions are int32 CUDA tensors, read when the call runs on the
GPU, so a captured call follows their later contents.
"""

import ctypes

import torch

from . import _lib

_DT = {torch.float16: _lib.F16, torch.bfloat16: _lib.BF16}
_DT_READ = dict(_DT)
_DT_READ[torch.float32] = _lib.PAGED_F32


def paged_config(n_layers, n_kv_heads, head_dim, n_q_heads, page_size, n_pages, k_fmt="f16", v_fmt=None, softmax_scale=0.0):
    """A kvq_paged_config; formats by name ("f16", "bf16", "q8_0", "q4_0"), v_fmt None meaning k_fmt."""
    c = _lib.kvq_paged_config()
    c.n_layers, c.n_kv_heads, c.head_dim, c.n_q_heads = n_layers, n_kv_heads, head_dim, n_q_heads
    c.page_size, c.n_pages = page_size, n_pages
    c.k_fmt = _lib.FMT_NAMES[k_fmt]
    c.v_fmt = _lib.FMT_NAMES[k_fmt if v_fmt is None else v_fmt]
    c.softmax_scale = softmax_scale
    return c


# The checks run on every call of a decode step, so they build no message unless they fail.
def _bad(what):
    raise ValueError(what)


def _ints(x, name, n, dev):
    """Address of a contiguous int32 vector of n elements on device `dev`."""
    if x.dtype is not torch.int32 or x.get_device() != dev or x.shape != (n,) or not x.is_contiguous():
        _bad(f"{name}: a contiguous int32 tensor of shape ({n},) on cuda:{dev} is wanted")
    return x.data_ptr()


def _rows(x, name, heads, D, dev, dtype):
    """(tokens, token stride) of [tokens, heads, D] rows whose heads lie behind one another."""
    shape = x.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != D or x.get_device() != dev or x.dtype is not dtype:
        _bad(f"{name}: {dtype} [tokens, {heads}, {D}] on cuda:{dev} is wanted, not {x.dtype} {tuple(shape)} on {x.device}")
    n, (st, sh, sd) = shape[0], x.stride()
    if n and (sd != 1 or (sh != D and heads != 1)):
        _bad(f"{name}: a token's heads must be contiguous")
    return n, (st if n > 1 else heads * D)


def _out_rows(x, name, n, heads, D, dev, dtype):
    if x.shape != (n, heads, D) or x.get_device() != dev or x.dtype is not dtype or not x.is_contiguous():
        _bad(f"{name}: contiguous {dtype} of shape ({n}, {heads}, {D}) on cuda:{dev} is wanted")
    return x.data_ptr()


def _type_of(x, name, types):
    t = types.get(x.dtype)
    if t is None:
        _bad(f"{name}: one of {', '.join(map(str, types))} is wanted, not {x.dtype}")
    return t


def _no_grad(*tensors):
    """Refuses tensors whose gradient would be lost, or wrong after a write in place."""
    if torch.is_grad_enabled():
        for x in tensors:
            if x is not None and x.requires_grad:
                _bad("a tensor requires a gradient, which this call does not have: call it under torch.no_grad() or detach")


# Written tensors: autograd finds out if it had saved one of them.
_changed = torch.autograd.graph.increment_version

_one_device = None


def _guarded(dev, call, *args):
    """call(*args) with device `dev` current."""
    global _one_device
    if _one_device is None:
        _one_device = torch.cuda.device_count() == 1
    if _one_device or torch.cuda.current_device() == dev:
        return call(*args)
    with torch.cuda.device(dev):
        return call(*args)


class PagedKVCache:
    """Pages of one or more layers on one device. ``pool`` (uint8, as large as ``pool_bytes``) is taken
    as it is; without it a zeroed one is made. The workspace serves calls of up to ``max_seqs`` sequences and
    ``max_tokens`` query rows of a prefill; calls that may overlap on the GPU (two streams, two captured
    graphs replayed side by side) each pass a workspace of their own (``new_workspace``)."""

    def __init__(self, cfg, device=0, max_seqs=1, max_tokens=0, pool=None):
        self.h = None
        self.cfg = cfg
        self.device = torch.device("cuda", device)
        self.max_seqs, self.max_tokens = max_seqs, max_tokens
        self.pool_bytes, self.ws_bytes = _lib.kv_paged_required_bytes(cfg, max_seqs, max_tokens)
        if pool is None:
            pool = torch.zeros(self.pool_bytes, dtype=torch.uint8, device=self.device)
        if (pool.device != self.device or pool.dtype is not torch.uint8 or not pool.is_contiguous() or
                pool.numel() < self.pool_bytes):
            _bad(f"pool: {self.pool_bytes} contiguous bytes on {self.device} are wanted")
        self.pool = pool
        self.ws = self.new_workspace()
        self._dev, self._H, self._Hq, self._D = device, cfg.n_kv_heads, cfg.n_q_heads, cfg.head_dim
        torch.cuda.current_stream(self.device).synchronize()      # the pool's contents, before the status word is set
        self.h = _guarded(device, _lib.kv_paged_create, cfg, pool.data_ptr(), pool.numel(), device)

    def new_workspace(self):
        return torch.empty(self.ws_bytes, dtype=torch.uint8, device=self.device)

    def close(self):
        if self.h is not None:
            _lib.kv_paged_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def status(self):
        """The device status word (bits PAGED_* of ``_lib``), read when the device has finished all work, and cleared."""
        return _guarded(self._dev, _lib.kv_paged_get_status, self.h)

    def write(self, layer, k, v, slots, stream=0):
        """k, v: [tokens, H, D] fp16 or bf16, token stride free; slots: int32 [tokens], page * page_size + row,
        negative to skip. Slots of one call must differ from one another."""
        dt = _type_of(k, "k", _DT)
        n, ks = _rows(k, "k", self._H, self._D, self._dev, k.dtype)
        nv, vs = _rows(v, "v", self._H, self._D, self._dev, k.dtype)
        if nv != n:
            _bad("k and v: the same number of tokens is wanted")
        sp = _ints(slots, "slots", n, self._dev)
        _no_grad(k, v)
        _guarded(self._dev, _lib.kv_paged_write, self.h, layer, dt, n, k.data_ptr(), ks, v.data_ptr(), vs, sp, stream)

    def _table(self, table):
        """(address, sequences, entries of a row, row stride) of a page table."""
        if table.dtype is not torch.int32 or table.get_device() != self._dev or table.dim() != 2:
            _bad(f"page_table: int32 [sequences, pages] on {self.device} is wanted")
        (n, w), (st, se) = table.shape, table.stride()
        if se != 1 and w > 1:
            _bad("page_table: a sequence's entries must be contiguous")
        return table.data_ptr(), n, w, st if n > 1 else w

    def read(self, layer, page_table, cu_rows, k_out=None, v_out=None, start=None, stream=0):
        """Rows cu_rows[b].. of k_out / v_out ([rows, H, D] contiguous fp16, bf16 or fp32; either may be
        None) receive positions start[b].. of sequence b. cu_rows: int32 [sequences + 1]."""
        tp, n, w, ts = self._table(page_table)
        x = k_out if k_out is not None else v_out
        if x is None:
            _bad("read: k_out or v_out is wanted")
        dt, rows = _type_of(x, "k_out, v_out", _DT_READ), x.shape[0]
        kp = None if k_out is None else _out_rows(k_out, "k_out", rows, self._H, self._D, self._dev, x.dtype)
        vp = None if v_out is None else _out_rows(v_out, "v_out", rows, self._H, self._D, self._dev, x.dtype)
        cp = _ints(cu_rows, "cu_rows", n + 1, self._dev)
        sp = None if start is None else _ints(start, "start", n, self._dev)
        _no_grad(k_out, v_out)
        _guarded(self._dev, _lib.kv_paged_read, self.h, layer, dt, n, tp, w, ts, cp, sp, rows, kp, vp, stream)
        _changed([x for x in (k_out, v_out) if x is not None])

    def _opts(self, n, rows, lse, softcap, window, slopes, prefix):
        sp = pp = lp = None
        if slopes is not None:
            if (slopes.dtype is not torch.float32 or slopes.get_device() != self._dev or slopes.shape != (self._Hq,) or
                    not slopes.is_contiguous()):
                _bad(f"slopes: contiguous fp32 of shape ({self._Hq},) on {self.device} is wanted")
            sp = slopes.data_ptr()
        if prefix is not None:
            pp = _ints(prefix, "prefix", n, self._dev)
        if lse is not None:
            if (lse.dtype is not torch.float32 or lse.get_device() != self._dev or lse.shape != (rows, self._Hq) or
                    not lse.is_contiguous()):
                _bad(f"lse: contiguous fp32 of shape ({rows}, {self._Hq}) on {self.device} is wanted")
            lp = lse.data_ptr()
        return ctypes.byref(_lib.kvq_attn_opts(softcap, window, sp, pp, lp))

    def _space(self, ws):
        if ws is None:
            return self.ws.data_ptr(), self.ws_bytes
        if ws.get_device() != self._dev or not ws.is_contiguous():
            _bad(f"ws: contiguous, on {self.device}")
        return ws.data_ptr(), ws.numel() * ws.element_size()

    def decode_attn(self, layer, q, page_table, lens, out, lse=None, softcap=0.0, window=0, slopes=None, prefix=None,
                    ws=None, stream=0):
        """Attention of one query per sequence. q: [sequences, Hq, D] fp16 or bf16 (token stride free), out alike
        and contiguous; lens: int32 [sequences], the new position included; lse: fp32 [sequences, Hq]."""
        dt, dev = _type_of(q, "q", _DT), self._dev
        tp, n, w, ts = self._table(page_table)
        rows, qs = _rows(q, "q", self._Hq, self._D, dev, q.dtype)
        if rows != n:
            _bad(f"q: one row per row of page_table ({n}) is wanted, not {rows}")
        lp = _ints(lens, "lens", n, dev)
        op = _out_rows(out, "out", n, self._Hq, self._D, dev, q.dtype)
        o = self._opts(n, n, lse, softcap, window, slopes, prefix)
        wp, wb = self._space(ws)
        _no_grad(q, out, slopes)
        _guarded(dev, _lib.kv_paged_decode_attn, self.h, layer, dt, n, q.data_ptr(), qs, tp, w, ts, lp, op, o, wp, wb, stream)
        _changed(out if lse is None else (out, lse))

    def prefill_attn(self, layer, q, cu_q, max_q, page_table, lens, out, lse=None, softcap=0.0, window=0, slopes=None,
                     prefix=None, ws=None, stream=0):
        """Attention of a chunk of new tokens per sequence, whose rows are in the pages already: rows
        cu_q[b] .. cu_q[b+1]-1 of q ([rows, Hq, D]) are the last positions of the lens[b] that sequence b holds.
        max_q: at least the longest chunk (of a longer one only the first max_q rows are computed)."""
        dt, dev = _type_of(q, "q", _DT), self._dev
        tp, n, w, ts = self._table(page_table)
        rows, qs = _rows(q, "q", self._Hq, self._D, dev, q.dtype)
        lp, cp = _ints(lens, "lens", n, dev), _ints(cu_q, "cu_q", n + 1, dev)
        op = _out_rows(out, "out", rows, self._Hq, self._D, dev, q.dtype)
        o = self._opts(n, rows, lse, softcap, window, slopes, prefix)
        wp, wb = self._space(ws)
        _no_grad(q, out, slopes)
        _guarded(dev, _lib.kv_paged_prefill_attn, self.h, layer, dt, n, rows, max_q, q.data_ptr(), qs, cp, tp, w, ts, lp, op,
                 o, wp, wb, stream)
        _changed(out if lse is None else (out, lse))


def qk_norm_rope(q, k, q_weight, k_weight, cos_sin, positions, q_out=None, k_out=None, eps=1e-6, interleaved=False,
                 stream=0):
    """RMS norm of every head of q [tokens, Hq, D] and k [tokens, H, D] and their rotation by position, in one
    pass; q or k may be None, a weight None leaves its side without the norm. cos_sin: fp32 [positions, rot],
    cosines then sines (None: no rotation); positions: int32 [tokens]. Outputs default to the inputs (in place)."""
    x = q if q is not None else k
    if x is None or x.dim() != 3 or not x.is_cuda:
        _bad("q, k: [tokens, heads, D] CUDA tensors are wanted")
    dt, dev, dtype, n, D = _type_of(x, "q, k", _DT), x.get_device(), x.dtype, x.shape[0], x.shape[2]
    sides = []
    for name, t, w, o in (("q", q, q_weight, q_out), ("k", k, k_weight, k_out)):
        if t is None:
            if o is not None:
                _bad(f"{name}_out without {name}")
            sides.append((0, None, None, None, 0, 0))
            continue
        heads = t.shape[1] if t.dim() == 3 else -1
        rows, st = _rows(t, name, heads, D, dev, dtype)
        if rows != n:
            _bad("q and k: the same number of tokens is wanted")
        op, ost = t.data_ptr(), st
        if o is not None:
            op = o.data_ptr()
            rows, ost = _rows(o, name + "_out", heads, D, dev, dtype)
            if rows != n:
                _bad(f"{name}_out: as many tokens as {name} is wanted")
        wp = None
        if w is not None:
            if w.dtype is not dtype or w.get_device() != dev or w.shape != (D,) or not w.is_contiguous():
                _bad(f"{name}_weight: contiguous {dtype} of shape ({D},) on cuda:{dev} is wanted")
            wp = w.data_ptr()
        sides.append((heads, t.data_ptr(), wp, op, st, ost))
    max_pos = rot = 0
    cp = pp = None
    if cos_sin is not None:
        if (cos_sin.dtype is not torch.float32 or cos_sin.get_device() != dev or cos_sin.dim() != 2 or
                not cos_sin.is_contiguous()):
            _bad(f"cos_sin: contiguous fp32 [positions, rot] on cuda:{dev} is wanted")
        if positions is None:
            _bad("positions are wanted with cos_sin")
        max_pos, rot = cos_sin.shape
        cp, pp = cos_sin.data_ptr(), _ints(positions, "positions", n, dev)
    (hq, qp, qw, qo, qs, qos), (hk, kp, kw, ko, ks, kos) = sides
    a = _lib.kvq_norm_rope_args(dt, n, hq, hk, D, rot, 1 if interleaved else 0, max_pos, eps, 0, qp, kp, qw, kw, cp, pp, qo, ko,
                                qs, ks, qos, kos)
    _no_grad(q, k, q_weight, k_weight, q_out, k_out, cos_sin)
    _guarded(dev, _lib.kv_qk_norm_rope, ctypes.byref(a), stream)
    _changed([t if o is None else o for t, o in ((q, q_out), (k, k_out)) if t is not None])
