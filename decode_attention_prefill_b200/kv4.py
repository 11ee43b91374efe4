"""The 4-bit paged cache and the norm with rotation: binding of the pnmix_kv4_* calls and
pnmix_norm_rope (include/pnmix.h).

    rope  = Rope.make(128)                                   what a model's heads are rotated by
    cache = KV4Cache(KV4Config.make(32, 8), n_pages)         pages of one layer
    batch = KV4Batch(kv_len, page_table, q_start, ...)       the sequences of one step
    q = cache.append_qkv(batch, rope, q, k, v, positions)    norm, rotate, quantise, write
    out = cache.attend(batch, q)                             causal attention over the pages

Token tensors are packed bf16 [n_tokens][heads][head_dim]; any strides that are multiples
of 8 elements do as long as the channels of a head lie together (views of one projection).
Every call runs on the device of its tensors and, unless `stream` names another, on that
device's current stream.
"""
from __future__ import annotations

import ctypes

import torch

from . import OK, ERR_DEVICE, PNMixError, _check, _lib

_vp, _i, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t


class KV4Config(ctypes.Structure):
    """pnmix_kv4_config: heads and pages of a 4-bit cache."""
    _fields_ = [("head_dim", ctypes.c_int32), ("n_q_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("page_tokens", ctypes.c_int32), ("softmax_scale", ctypes.c_float)]

    @classmethod
    def make(cls, n_q_heads: int, n_kv_heads: int, head_dim: int = 128, page_tokens: int = 64,
             softmax_scale: float = 0.0) -> "KV4Config":
        return cls(head_dim, n_q_heads, n_kv_heads, page_tokens, softmax_scale)


class Rope(ctypes.Structure):
    """pnmix_rope: norm epsilon and rotation of query and key heads."""
    _fields_ = [("head_dim", ctypes.c_int32), ("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("n_axes", ctypes.c_int32), ("eps", ctypes.c_float), ("inv_freq", ctypes.c_float * 128),
                ("axis", ctypes.c_uint8 * 128)]

    @classmethod
    def make(cls, head_dim: int, rot_dim: int | None = None, theta: float = 500000.0, inv_freq=None, axes=None,
             interleaved: bool = False, eps: float = 1e-6) -> "Rope":
        """inv_freq: one per pair (default theta^(-2i / rot_dim)); axes: the position axis of
        each pair (default: all 0).  rot_dim defaults to 2 * len(inv_freq), else head_dim."""
        if inv_freq is None:
            rot_dim = head_dim if rot_dim is None else rot_dim
            inv_freq = [theta ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)]
        inv_freq = [float(f) for f in inv_freq]
        if rot_dim is None:
            rot_dim = 2 * len(inv_freq)
        axes = [0] * len(inv_freq) if axes is None else [int(x) for x in axes]
        if len(inv_freq) > 128 or 2 * len(inv_freq) != rot_dim or len(axes) != len(inv_freq):
            raise ValueError("inv_freq and axes hold rot_dim / 2 entries, at most 128")
        if any(not 0 <= x <= 3 for x in axes):
            raise ValueError("axes are 0 .. 3")
        r = cls(head_dim, rot_dim, int(interleaved), max(axes, default=0) + 1, eps)
        r.inv_freq[:len(inv_freq)] = inv_freq
        r.axis[:len(axes)] = axes
        return r


class _Rows(ctypes.Structure):
    _fields_ = [("data", _vp), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class _Batch(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("n_tokens", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("max_q", ctypes.c_int32), ("q_start", _vp), ("kv_len", _vp), ("page_table", _vp)]


class _Cache(ctypes.Structure):
    _fields_ = [("n_pages", ctypes.c_int32), ("page_tokens", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("pages", _vp), ("error", _vp), ("base", _vp),
                ("total_bytes", _sz)]


_P = ctypes.POINTER
_RP, _BP, _KP, _CP, _OP = _P(_Rows), _P(_Batch), _P(_Cache), _P(KV4Config), _P(Rope)
SIGNATURES = {
    "pnmix_norm_rope": (_i, [_OP, _i, _i, _i, _RP, _RP, _vp, _vp, _vp, _RP, _RP, _vp]),
    "pnmix_kv4_cache_bytes": (_i, [_CP, _i, _P(_sz)]),
    "pnmix_kv4_cache_init": (_i, [_CP, _i, _vp, _sz, _KP]),
    "pnmix_kv4_cache_reset": (_i, [_KP, _vp]),
    "pnmix_kv4_append": (_i, [_CP, _BP, _RP, _RP, _KP, _vp]),
    "pnmix_kv4_append_qkv": (_i, [_CP, _OP, _BP, _RP, _RP, _RP, _vp, _vp, _vp, _RP, _KP, _vp]),
    "pnmix_kv4_read": (_i, [_CP, _BP, _KP, _RP, _RP, _vp]),
    "pnmix_kv4_workspace_bytes": (_sz, [_CP, _BP]),
    "pnmix_kv4_attention": (_i, [_CP, _BP, _RP, _KP, _RP, _vp, _sz, _vp]),
    "pnmix_kv4_read_error": (_i, [_KP, _i, _P(ctypes.c_uint32)]),
}
for _name, (_res, _args) in SIGNATURES.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


def _rows(t: torch.Tensor, heads: int, dim: int, device, name: str, tokens: int | None = None) -> _Rows:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != dim or (tokens is not None and t.shape[0] != tokens):
        raise ValueError(f"{name} must be [{'tokens' if tokens is None else tokens}][{heads}][{dim}], "
                         f"got {list(t.shape)}")
    s0, s1, s2 = t.stride()
    if s2 != 1:
        raise ValueError(f"{name}: the channels of a head must be contiguous")
    return _Rows(t.data_ptr(), 0 if t.shape[0] == 1 else s0, 0 if heads == 1 else s1)


def _ints(t: torch.Tensor, shape: tuple, device, name: str) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.int32:
        raise TypeError(f"{name} must be an int32 CUDA tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {list(shape)}, got {list(t.shape)}")
    return t.data_ptr()


def _weight(t, dim: int, device, name: str):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be a bfloat16 CUDA tensor")
    if t.device != device or tuple(t.shape) != (dim,) or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous [{dim}] on {device}")
    return t.data_ptr()


class _On:
    """The device a call runs on and the stream it goes to; outputs made inside belong to
    that stream."""

    def __init__(self, device, stream):
        self.device, self.stream = device, stream

    def __enter__(self):
        self._prev = None
        if self.device.index != torch.cuda.current_device():
            self._prev = torch.cuda.device(self.device)
            self._prev.__enter__()
        self._ctx = None
        if self.stream is None:
            return torch.cuda.current_stream().cuda_stream
        s = self.stream
        if not hasattr(s, "cuda_stream"):
            s = torch.cuda.ExternalStream(int(s), device=self.device)
        if s.device != self.device:
            self.__exit__()
            raise ValueError(f"stream is on {s.device}, the tensors on {self.device}")
        self._ctx = torch.cuda.stream(s)
        self._ctx.__enter__()
        return s.cuda_stream

    def __exit__(self, *exc):
        if self._ctx is not None:
            self._ctx.__exit__(None, None, None)
        if self._prev is not None:
            self._prev.__exit__(None, None, None)


def norm_rope(rope: Rope, q: torch.Tensor, k: torch.Tensor, positions: torch.Tensor, q_weight=None, k_weight=None,
              q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None, stream=None):
    """Norm of every head of q and k (where a weight is given) and rotation by position.
    q, k bf16 [n][heads][head_dim]; positions int32 [n_axes][n] ([n] with one axis).  Returns
    (q_out, k_out), which may be the inputs themselves."""
    dev, D = q.device, rope.head_dim
    n, hq, hk = q.shape[0], q.shape[1], k.shape[1]
    if rope.n_axes == 1 and positions.dim() == 1:
        positions = positions[None]
    rq, rk = _rows(q, hq, D, dev, "q"), _rows(k, hk, D, dev, "k", n)
    pos = _ints(positions, (rope.n_axes, n), dev, "positions")
    wq, wk = _weight(q_weight, D, dev, "q_weight"), _weight(k_weight, D, dev, "k_weight")
    with _On(dev, stream) as s:
        q_out = torch.empty((n, hq, D), dtype=q.dtype, device=dev) if q_out is None else q_out
        k_out = torch.empty((n, hk, D), dtype=q.dtype, device=dev) if k_out is None else k_out
        oq, ok = _rows(q_out, hq, D, dev, "q_out", n), _rows(k_out, hk, D, dev, "k_out", n)
        _check(_lib.pnmix_norm_rope(ctypes.byref(rope), n, hq, hk, ctypes.byref(rq), ctypes.byref(rk), wq, wk, pos,
                                    ctypes.byref(oq), ctypes.byref(ok), s), "pnmix_norm_rope")
    return q_out, k_out


class KV4Batch:
    """The sequences of one call (pnmix_kv4_batch).  The tensors are kept, not copied: their
    contents may change between calls (and between replays of a graph).

    kv_len int32 [B], the calls' rows included; page_table int32 [B][max_pages]; q_start
    int32 [B + 1], or None for n_tokens / B rows of every sequence.  n_tokens: rows of the
    token tensors (padding behind q_start[B] included).  max_q: no sequence has more rows
    (default: n_tokens / B without q_start, else n_tokens)."""

    def __init__(self, kv_len: torch.Tensor, page_table: torch.Tensor, q_start: torch.Tensor | None = None, *,
                 n_tokens: int, max_q: int | None = None):
        if not isinstance(kv_len, torch.Tensor) or kv_len.dim() != 1 or kv_len.numel() < 1:
            raise ValueError("kv_len must be [batch]")
        if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
            raise ValueError("page_table must be [batch][max_pages]")
        B, dev = kv_len.numel(), kv_len.device
        if max_q is None:
            max_q = n_tokens if q_start is not None else n_tokens // B
        self.device, self.n_tokens = dev, n_tokens
        self.kv_len, self.page_table, self.q_start = kv_len, page_table, q_start
        self.c = _Batch(B, n_tokens, page_table.shape[1], max_q,
                        None if q_start is None else _ints(q_start, (B + 1,), dev, "q_start"),
                        _ints(kv_len, (B,), dev, "kv_len"),
                        _ints(page_table, (B, page_table.shape[1]), dev, "page_table"))


class KV4Cache:
    """The pages of one layer.  `buffer`: uint8 memory to use, 256-byte aligned and at least
    kv4_cache_bytes long (its contents stay); without it zeroed memory is taken."""

    def __init__(self, cfg: KV4Config, n_pages: int, device="cuda", buffer: torch.Tensor | None = None):
        self.cfg, self.n_pages = cfg, n_pages
        nbytes = kv4_cache_bytes(cfg, n_pages)
        if buffer is None:
            buffer = torch.zeros(nbytes, dtype=torch.uint8, device=device)
        if not buffer.is_cuda or buffer.dtype != torch.uint8 or not buffer.is_contiguous():
            raise TypeError("buffer must be contiguous uint8 CUDA memory")
        self.buffer, self.device = buffer, buffer.device
        self.c = _Cache()
        _check(_lib.pnmix_kv4_cache_init(ctypes.byref(cfg), n_pages, buffer.data_ptr(), buffer.numel(),
                                         ctypes.byref(self.c)), "pnmix_kv4_cache_init")
        self._refs = (ctypes.byref(cfg), ctypes.byref(self.c))

    def reset(self, stream=None):
        """Zero the pages and the error word."""
        with _On(self.device, stream) as s:
            _check(_lib.pnmix_kv4_cache_reset(self._refs[1], s), "pnmix_kv4_cache_reset")

    def _on(self, batch: KV4Batch, stream):
        if batch.device != self.device:
            raise ValueError(f"the batch is on {batch.device}, the cache on {self.device}")
        return _On(self.device, stream)

    def append(self, batch: KV4Batch, k: torch.Tensor, v: torch.Tensor, stream=None):
        """Quantise rows k, v bf16 [n][Hkv][head_dim] (after RoPE) into the batch's places."""
        H, D, n = self.cfg.n_kv_heads, self.cfg.head_dim, batch.n_tokens
        rk, rv = _rows(k, H, D, self.device, "k", n), _rows(v, H, D, self.device, "v", n)
        with self._on(batch, stream) as s:
            _check(_lib.pnmix_kv4_append(self._refs[0], ctypes.byref(batch.c), ctypes.byref(rk), ctypes.byref(rv),
                                         self._refs[1], s), "pnmix_kv4_append")

    def append_qkv(self, batch: KV4Batch, rope: Rope, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                   positions: torch.Tensor, q_weight=None, k_weight=None, q_out: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
        """norm_rope of q and k and append of the rotated k and v in one pass; returns q_out."""
        c, n, dev = self.cfg, batch.n_tokens, self.device
        D = c.head_dim
        if rope.n_axes == 1 and positions.dim() == 1:
            positions = positions[None]
        rq, rk = _rows(q, c.n_q_heads, D, dev, "q", n), _rows(k, c.n_kv_heads, D, dev, "k", n)
        rv = _rows(v, c.n_kv_heads, D, dev, "v", n)
        pos = _ints(positions, (rope.n_axes, n), dev, "positions")
        wq, wk = _weight(q_weight, D, dev, "q_weight"), _weight(k_weight, D, dev, "k_weight")
        with self._on(batch, stream) as s:
            if q_out is None:
                q_out = torch.empty((n, c.n_q_heads, D), dtype=q.dtype, device=dev)
            ro = _rows(q_out, c.n_q_heads, D, dev, "q_out", n)
            _check(_lib.pnmix_kv4_append_qkv(self._refs[0], ctypes.byref(rope), ctypes.byref(batch.c),
                                             ctypes.byref(rq), ctypes.byref(rk), ctypes.byref(rv), wq, wk, pos,
                                             ctypes.byref(ro), self._refs[1], s), "pnmix_kv4_append_qkv")
        return q_out

    def read(self, batch: KV4Batch, k_out: torch.Tensor | None = None, v_out: torch.Tensor | None = None,
             stream=None):
        """The batch's rows as the cache holds them: (k, v) bf16 [n][Hkv][head_dim]."""
        H, D, n, dev = self.cfg.n_kv_heads, self.cfg.head_dim, batch.n_tokens, self.device
        with self._on(batch, stream) as s:
            k_out = torch.empty((n, H, D), dtype=torch.bfloat16, device=dev) if k_out is None else k_out
            v_out = torch.empty((n, H, D), dtype=torch.bfloat16, device=dev) if v_out is None else v_out
            rk, rv = _rows(k_out, H, D, dev, "k_out", n), _rows(v_out, H, D, dev, "v_out", n)
            _check(_lib.pnmix_kv4_read(self._refs[0], ctypes.byref(batch.c), self._refs[1], ctypes.byref(rk),
                                       ctypes.byref(rv), s), "pnmix_kv4_read")
        return k_out, v_out

    def attend(self, batch: KV4Batch, q: torch.Tensor, out: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """Causal attention of q bf16 [n][Hq][head_dim] over the pages -> bf16, same shape.
        The workspace (kv4_workspace_bytes) is taken from torch's allocator for the call unless
        one is given."""
        c, n, dev = self.cfg, batch.n_tokens, self.device
        rq = _rows(q, c.n_q_heads, c.head_dim, dev, "q", n)
        need = _lib.pnmix_kv4_workspace_bytes(self._refs[0], ctypes.byref(batch.c))
        with self._on(batch, stream) as s:
            if out is None:
                out = torch.empty((n, c.n_q_heads, c.head_dim), dtype=q.dtype, device=dev)
            ro = _rows(out, c.n_q_heads, c.head_dim, dev, "out", n)
            if workspace is None:
                workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
            elif not workspace.is_cuda or workspace.device != dev or workspace.dtype != torch.uint8 \
                    or not workspace.is_contiguous():
                raise TypeError(f"workspace must be contiguous uint8 on {dev}")
            _check(_lib.pnmix_kv4_attention(self._refs[0], ctypes.byref(batch.c), ctypes.byref(rq), self._refs[1],
                                            ctypes.byref(ro), workspace.data_ptr(), workspace.numel(), s),
                   "pnmix_kv4_attention")
        return out

    def pages(self) -> torch.Tensor:
        """uint8 view [n_pages][Hkv][blocks][20 * head_dim] (for tests and inspection)."""
        c = self.cfg
        n = self.n_pages * c.n_kv_heads * (c.page_tokens // 16) * 20 * c.head_dim
        return self.buffer[:n].view(self.n_pages, c.n_kv_heads, c.page_tokens // 16, 20 * c.head_dim)

    def read_error(self, clear: bool = True) -> int:
        """The device error word (waits for the device)."""
        val = ctypes.c_uint32(0)
        with torch.cuda.device(self.device):
            torch.cuda.current_stream().synchronize()
            st = _lib.pnmix_kv4_read_error(self._refs[1], 1 if clear else 0, ctypes.byref(val))
        if st not in (OK, ERR_DEVICE):
            raise PNMixError(st, "pnmix_kv4_read_error")
        return int(val.value)


def kv4_cache_bytes(cfg: KV4Config, n_pages: int) -> int:
    out = _sz(0)
    _check(_lib.pnmix_kv4_cache_bytes(ctypes.byref(cfg), n_pages, ctypes.byref(out)), "pnmix_kv4_cache_bytes")
    return int(out.value)


def kv4_workspace_bytes(cfg: KV4Config, batch: KV4Batch) -> int:
    return int(_lib.pnmix_kv4_workspace_bytes(ctypes.byref(cfg), ctypes.byref(batch.c)))
