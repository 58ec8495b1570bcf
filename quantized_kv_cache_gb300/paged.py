"""The paged KV cache on PyTorch CUDA tensors: rows to pages, back from them, and attention over them.

``PagedKVCache`` owns (or takes) a pool of pages and a workspace and forwards to the C ABI of
``include/kvq_paged.h``; ``qk_norm_rope`` needs no cache. The tensors are checked here (device, type,
shape, strides) and an argument that does not fit raises ``ValueError`` before anything is enqueued;
what the C side refuses raises ``KVQError``. As in ``KVCache``, ``stream`` is a raw CUDA stream handle
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


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _ints(x, name, shape, dev):
    _need(x.dtype is torch.int32 and x.device == dev, f"{name}: an int32 tensor on {dev} is wanted")
    _need(tuple(x.shape) == shape and x.is_contiguous(), f"{name}: contiguous, of shape {shape}")
    return x.data_ptr()


def _rows(x, name, heads, D, dev, dtype=None):
    """Token stride of [tokens, heads, D] rows whose heads lie behind one another."""
    _need(x.device == dev and x.dim() == 3 and x.shape[1] == heads and x.shape[2] == D,
          f"{name}: [tokens, {heads}, {D}] on {dev} is wanted, not {tuple(x.shape)} on {x.device}")
    _need(dtype is None or x.dtype is dtype, f"{name}: {dtype} is wanted, not {x.dtype}")
    st = x.stride()
    _need(x.numel() == 0 or (st[2] == 1 and (heads == 1 or st[1] == D)), f"{name}: a token's heads must be contiguous")
    if x.shape[0] <= 1:
        return max(st[0], heads * D) // 8 * 8
    return st[0]


def _on(dev):
    """Makes `dev` current for a call where it is not."""
    return torch.cuda.device(dev) if torch.cuda.current_device() != dev.index else _Here


class _HereType:
    def __enter__(self):
        return self

    def __exit__(self, *a):
        return False


_Here = _HereType()


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
        _need(pool.device == self.device and pool.dtype is torch.uint8 and pool.is_contiguous() and
              pool.numel() >= self.pool_bytes, f"pool: {self.pool_bytes} contiguous bytes on {self.device} are wanted")
        self.pool = pool
        self.ws = self.new_workspace()
        with _on(self.device):
            torch.cuda.current_stream().synchronize()      # the pool's contents, before the status word is set
            self.h = _lib.kv_paged_create(cfg, pool.data_ptr(), pool.numel(), device)

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
        """The device status word (bits PAGED_* of ``_lib``), read synchronously and cleared."""
        with _on(self.device):
            return _lib.kv_paged_get_status(self.h)

    def write(self, layer, k, v, slots, stream=0):
        """k, v: [tokens, H, D] fp16 or bf16, token stride free; slots: int32 [tokens], page * page_size + row,
        negative to skip. Slots of one call must differ from one another."""
        c = self.cfg
        _need(k.dtype in _DT, f"k: fp16 or bf16 is wanted, not {k.dtype}")
        ks = _rows(k, "k", c.n_kv_heads, c.head_dim, self.device)
        vs = _rows(v, "v", c.n_kv_heads, c.head_dim, self.device, k.dtype)
        n = k.shape[0]
        _need(v.shape[0] == n, "k and v: the same number of tokens")
        sp = _ints(slots, "slots", (n,), self.device)
        with _on(self.device):
            _lib.kv_paged_write(self.h, layer, _DT[k.dtype], n, k.data_ptr(), ks, v.data_ptr(), vs, sp, stream)

    def _table(self, table):
        _need(table.dtype is torch.int32 and table.device == self.device and table.dim() == 2 and
              (table.stride(1) == 1 or table.shape[1] == 1),
              f"page_table: int32 [sequences, pages] on {self.device}, rows contiguous")
        n, w = table.shape
        return table.data_ptr(), n, w, max(table.stride(0), w) if n <= 1 else table.stride(0)

    def read(self, layer, page_table, cu_rows, k_out=None, v_out=None, start=None, stream=0):
        """Rows cu_rows[b].. of k_out / v_out ([rows, H, D] contiguous fp16, bf16 or fp32; either may be
        None) receive positions start[b].. of sequence b. cu_rows: int32 [sequences + 1]."""
        c = self.cfg
        tp, n, w, ts = self._table(page_table)
        outs = [x for x in (k_out, v_out) if x is not None]
        _need(outs, "read: k_out or v_out is wanted")
        _need(outs[0].dtype in _DT_READ, f"read: fp16, bf16 or fp32 rows are wanted, not {outs[0].dtype}")
        for x in outs:
            _rows(x, "out", c.n_kv_heads, c.head_dim, self.device, outs[0].dtype)
            _need(x.is_contiguous() and x.shape == outs[0].shape, "k_out, v_out: contiguous, of one shape")
        cp = _ints(cu_rows, "cu_rows", (n + 1,), self.device)
        sp = None if start is None else _ints(start, "start", (n,), self.device)
        with _on(self.device):
            _lib.kv_paged_read(self.h, layer, _DT_READ[outs[0].dtype], n, tp, w, ts, cp, sp, outs[0].shape[0],
                               None if k_out is None else k_out.data_ptr(), None if v_out is None else v_out.data_ptr(),
                               stream)

    def _attn(self, q, page_table, lens, out, lse, softcap, window, slopes, prefix, ws):
        c = self.cfg
        _need(q.dtype in _DT, f"q: fp16 or bf16 is wanted, not {q.dtype}")
        qs = _rows(q, "q", c.n_q_heads, c.head_dim, self.device)
        tp, n, w, ts = self._table(page_table)
        lp = _ints(lens, "lens", (n,), self.device)
        _rows(out, "out", c.n_q_heads, c.head_dim, self.device, q.dtype)
        _need(out.is_contiguous() and out.shape[0] == q.shape[0], "out: contiguous, of q's shape")
        o = _lib.kvq_attn_opts()
        o.softcap, o.window = softcap, window
        for name, x, shape, dt in (("slopes", slopes, (c.n_q_heads,), torch.float32), ("prefix", prefix, (n,), torch.int32),
                                   ("lse", lse, (q.shape[0], c.n_q_heads), torch.float32)):
            if x is not None:
                _need(x.dtype is dt and x.device == self.device and tuple(x.shape) == shape and x.is_contiguous(),
                      f"{name}: contiguous {dt} of shape {shape} on {self.device}")
                setattr(o, name, x.data_ptr())
        ws = self.ws if ws is None else ws
        _need(ws.device == self.device and ws.is_contiguous(), f"ws: contiguous, on {self.device}")
        return qs, tp, n, w, ts, lp, ctypes.byref(o), ws.data_ptr(), ws.numel() * ws.element_size()

    def decode_attn(self, layer, q, page_table, lens, out, lse=None, softcap=0.0, window=0, slopes=None, prefix=None,
                    ws=None, stream=0):
        """Attention of one query per sequence. q: [sequences, Hq, D] fp16 or bf16 (token stride free), out alike
        and contiguous; lens: int32 [sequences], the new position included; lse: fp32 [sequences, Hq]."""
        qs, tp, n, w, ts, lp, o, wp, wb = self._attn(q, page_table, lens, out, lse, softcap, window, slopes, prefix, ws)
        _need(q.shape[0] == n, "q: one row per row of page_table")
        with _on(self.device):
            _lib.kv_paged_decode_attn(self.h, layer, _DT[q.dtype], n, q.data_ptr(), qs, tp, w, ts, lp, out.data_ptr(), o, wp,
                                      wb, stream)

    def prefill_attn(self, layer, q, cu_q, max_q, page_table, lens, out, lse=None, softcap=0.0, window=0, slopes=None,
                     prefix=None, ws=None, stream=0):
        """Attention of a chunk of new tokens per sequence, whose rows are in the pages already: rows
        cu_q[b] .. cu_q[b+1]-1 of q ([rows, Hq, D]) are the last positions of the lens[b] that sequence b holds.
        max_q: at least the longest chunk."""
        qs, tp, n, w, ts, lp, o, wp, wb = self._attn(q, page_table, lens, out, lse, softcap, window, slopes, prefix, ws)
        cp = _ints(cu_q, "cu_q", (n + 1,), self.device)
        with _on(self.device):
            _lib.kv_paged_prefill_attn(self.h, layer, _DT[q.dtype], n, q.shape[0], max_q, q.data_ptr(), qs, cp, tp, w, ts, lp,
                                       out.data_ptr(), o, wp, wb, stream)


def qk_norm_rope(q, k, q_weight, k_weight, cos_sin, positions, q_out=None, k_out=None, eps=1e-6, interleaved=False,
                 stream=0):
    """RMS norm of every head of q [tokens, Hq, D] and k [tokens, H, D] and their rotation by position, in one
    pass; q or k may be None, a weight None leaves its side without the norm. cos_sin: fp32 [positions, rot],
    cosines then sines (None: no rotation); positions: int32 [tokens]. Outputs default to the inputs (in place)."""
    a = _lib.kvq_norm_rope_args()
    x = q if q is not None else k
    _need(x is not None and x.dim() == 3 and x.dtype in _DT and x.is_cuda, "q, k: [tokens, heads, D] fp16 or bf16 CUDA tensors")
    dev, dt, n, D = x.device, x.dtype, x.shape[0], x.shape[2]
    a.dtype, a.n_tok, a.head_dim, a.eps, a.interleaved = _DT[dt], n, D, eps, 1 if interleaved else 0
    for name, t, wt, o in (("q", q, q_weight, q_out), ("k", k, k_weight, k_out)):
        if t is None:
            _need(o is None, f"{name}_out without {name}")
            continue
        o = t if o is None else o
        heads = t.shape[1] if t.dim() == 3 else -1
        setattr(a, f"n_{name}_heads", heads)
        setattr(a, f"{name}_stride", _rows(t, name, heads, D, dev, dt))
        setattr(a, f"{name}_out_stride", _rows(o, name + "_out", heads, D, dev, dt))
        _need(t.shape[0] == n and o.shape[0] == n, "q, k and outputs: the same number of tokens")
        setattr(a, name, t.data_ptr())
        setattr(a, name + "_out", o.data_ptr())
        if wt is not None:
            _need(wt.dtype is dt and wt.device == dev and tuple(wt.shape) == (D,) and wt.is_contiguous(),
                  f"{name}_weight: contiguous {dt} of shape ({D},) on {dev}")
            setattr(a, name + "_weight", wt.data_ptr())
    if cos_sin is not None:
        _need(cos_sin.dtype is torch.float32 and cos_sin.device == dev and cos_sin.dim() == 2 and cos_sin.is_contiguous(),
              f"cos_sin: contiguous fp32 [positions, rot] on {dev}")
        a.max_pos, a.rot_dim = cos_sin.shape
        a.cos_sin = cos_sin.data_ptr()
        _need(positions is not None, "positions are wanted with cos_sin")
        a.positions = _ints(positions, "positions", (n,), dev)
    with _on(dev):
        _lib.kv_qk_norm_rope(ctypes.byref(a), stream)
