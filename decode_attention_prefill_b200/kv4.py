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

import contextlib
import ctypes
import struct

import torch

from . import OK, ERR_DEVICE, PNMixError, _check, _lib

_vp, _i, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t


def _count(x, name: str) -> int:
    """A size that the C structures hold: ctypes would keep its low 32 bits without a word."""
    if not -(1 << 31) <= x < 1 << 31:
        raise ValueError(f"{name} must fit 32 bits, got {x}")
    return x


class KV4Config(ctypes.Structure):
    """pnmix_kv4_config: heads and pages of a 4-bit cache."""
    _fields_ = [("head_dim", ctypes.c_int32), ("n_q_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("page_tokens", ctypes.c_int32), ("softmax_scale", ctypes.c_float)]

    @classmethod
    def make(cls, n_q_heads: int, n_kv_heads: int, head_dim: int = 128, page_tokens: int = 64,
             softmax_scale: float = 0.0) -> "KV4Config":
        return cls(_count(head_dim, "head_dim"), _count(n_q_heads, "n_q_heads"), _count(n_kv_heads, "n_kv_heads"),
                   _count(page_tokens, "page_tokens"), softmax_scale)


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
        r = cls(_count(head_dim, "head_dim"), _count(rot_dim, "rot_dim"), int(interleaved), max(axes, default=0) + 1, eps)
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
    "pnmix_debug_kv4_stall": (_i, [_CP, _BP, _RP, _KP, _RP, _vp, _sz, _i, ctypes.c_uint32, _vp]),
    "pnmix_kv4_read_error": (_i, [_KP, _i, _P(ctypes.c_uint32)]),
}
for _name, (_res, _args) in SIGNATURES.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args
_byref = ctypes.byref


def _untyped(name: str):
    """The same call with its pointers to structures as plain addresses: a packed pnmix_rows passed as
    bytes costs a quarter of a ctypes structure, and a small call is bound by such things (the
    norm of one token 17.0 us a call, with structures and checks of its own outputs 20.6)."""
    fn = _lib[name]
    res, args = SIGNATURES[name]
    fn.restype, fn.argtypes = res, [_vp if a in (_RP, _BP, _KP, _CP, _OP) else a for a in args]
    return fn


_norm_rope, _append, _append_qkv, _read, _attention = (_untyped("pnmix_" + n) for n in (
    "norm_rope", "kv4_append", "kv4_append_qkv", "kv4_read", "kv4_attention"))
_pack = struct.Struct("Pqq").pack        # pnmix_rows


def _strides(t: torch.Tensor, shape: tuple, device, name: str) -> tuple:
    """The fields of pnmix_rows for a bf16 tensor [tokens][heads][head_dim] on `device`."""
    if isinstance(t, torch.Tensor) and t.dtype is torch.bfloat16 and t.shape == shape and t.device == device:
        s0, s1, s2 = t.stride()
        if s2 == 1:
            return t.data_ptr(), s0 if shape[0] > 1 else 0, s1 if shape[1] > 1 else 0
        raise ValueError(f"{name}: the channels of a head must be contiguous")
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


def _rows(t: torch.Tensor, shape: tuple, device, name: str) -> _Rows:
    return _Rows(*_strides(t, shape, device, name))


def _out(t, shape: tuple, like: torch.Tensor, device, name: str) -> tuple:
    """(tensor, its rows): the caller's output, checked, or a new one shaped like `like`."""
    if t is not None:
        return t, _byref(_rows(t, shape, device, name))
    t = torch.empty_like(like, memory_format=torch.contiguous_format)
    return t, _pack(t.data_ptr(), shape[1] * shape[2], shape[2])


def _ints(t: torch.Tensor, shape: tuple, device, name: str) -> int:
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.int32:
        raise TypeError(f"{name} must be an int32 tensor")
    if t.device != device or not t.is_cuda:
        raise ValueError(f"{name} is on {t.device}, not on {device}") if t.is_cuda else \
            TypeError(f"{name} must be a CUDA tensor")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {list(shape)}, got {list(t.shape)}")
    return t.data_ptr()


def _positions(t: torch.Tensor, axes: int, n: int, device) -> int:
    return _ints(t, (n,) if axes == 1 and isinstance(t, torch.Tensor) and t.dim() == 1 else (axes, n), device,
                 "positions")


def _weight(t, dim: int, device, name: str):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be a bfloat16 tensor")
    if t.device != device or t.shape != (dim,) or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous [{dim}] on {device}")
    return t.data_ptr()


_SAME = contextlib.nullcontext()


def _on(device, stream):
    """(context, raw stream, stream object or None): where a call on `device` goes.  Outputs made
    inside the context belong to that stream."""
    if stream is None:
        # the raw handle: a Stream object around it costs more than the rest of a small call
        ctx = _SAME if device.index == torch.cuda.current_device() else torch.cuda.device(device)
        return ctx, torch._C._cuda_getCurrentRawStream(device.index), None
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    if stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    return torch.cuda.stream(stream), stream.cuda_stream, stream


def _used_on(stream, *tensors):
    """Tells the allocator that a named stream uses these: their memory is not given out again
    before it is done with them."""
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


def norm_rope(rope: Rope, q: torch.Tensor | None, k: torch.Tensor | None, positions: torch.Tensor, q_weight=None,
              k_weight=None, q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None, stream=None):
    """Norm of every head of q and k (where a weight is given) and rotation by position.
    q, k bf16 [n][heads][head_dim], one of them may be None; positions int32 [n_axes][n] ([n]
    with one axis).  Returns (q_out, k_out), which may be the inputs themselves."""
    if not isinstance(rope, Rope):
        raise TypeError("rope must be a Rope")
    any_ = q if q is not None else k
    if not isinstance(any_, torch.Tensor) or any_.dim() != 3:
        raise TypeError("q and k are tensors [tokens][heads][head_dim], or one of them None")
    dev, n, D = any_.device, any_.shape[0], rope.head_dim
    pos = _positions(positions, rope.n_axes, n, dev)
    rq = rk = oq = ok = None
    hq = hk = 0
    ctx, s, named = _on(dev, stream)
    with ctx:
        if q is not None:
            hq = q.shape[1]
            shape = (n, hq, D)
            rq = _pack(*_strides(q, shape, dev, "q"))
            q_out, oq = _out(q_out, shape, q, dev, "q_out")
        if k is not None:
            if k.dim() != 3:
                raise ValueError("k must be [tokens][heads][head_dim]")
            hk = k.shape[1]
            shape = (n, hk, D)
            rk = _pack(*_strides(k, shape, dev, "k"))
            k_out, ok = _out(k_out, shape, k, dev, "k_out")
        _check(_norm_rope(_byref(rope), n, hq, hk, rq, rk, _weight(q_weight, D, dev, "q_weight"),
                          _weight(k_weight, D, dev, "k_weight"), pos, oq, ok, s), "pnmix_norm_rope")
    if named is not None:
        _used_on(named, q, k, positions, q_weight, k_weight, q_out, k_out)
    return q_out, k_out


class KV4Batch:
    """The sequences of one call (pnmix_kv4_batch).  The tensors are kept, not copied: their
    contents may change between calls (and between replays of a graph).  Which tensors they are
    and how many rows there are stays as it was made.

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
        c = _Batch(B, _count(n_tokens, "n_tokens"), page_table.shape[1], _count(max_q, "max_q"),
                   None if q_start is None else _ints(q_start, (B + 1,), dev, "q_start"),
                   _ints(kv_len, (B,), dev, "kv_len"),
                   _ints(page_table, (B, page_table.shape[1]), dev, "page_table"))
        self.__dict__.update(device=dev, n_tokens=n_tokens, kv_len=kv_len, page_table=page_table, q_start=q_start,
                             c=c, ref=ctypes.byref(c))

    def __setattr__(self, name, value):
        raise AttributeError(f"{name} of a KV4Batch stays as it was made; make another batch")


class KV4Cache:
    """The pages of one layer.  `buffer`: uint8 memory to use, 256-byte aligned and at least
    kv4_cache_bytes long (its contents stay); without it zeroed memory is taken.  What a cache was
    made with stays: `cfg` gives a copy."""

    def __init__(self, cfg: KV4Config, n_pages: int, device="cuda", buffer: torch.Tensor | None = None):
        if not isinstance(cfg, KV4Config):
            raise TypeError("cfg must be a KV4Config")
        cfg = KV4Config.from_buffer_copy(cfg)      # what the caller does with theirs later changes no call
        self._cfg, self.n_pages = cfg, n_pages
        nbytes = kv4_cache_bytes(cfg, n_pages)
        if buffer is None:
            buffer = torch.zeros(nbytes, dtype=torch.uint8, device=device)
        if not buffer.is_cuda or buffer.dtype != torch.uint8 or not buffer.is_contiguous():
            raise TypeError("buffer must be contiguous uint8 CUDA memory")
        self.buffer, self.device = buffer, buffer.device
        self.c = _Cache()
        _check(_lib.pnmix_kv4_cache_init(ctypes.byref(cfg), n_pages, buffer.data_ptr(), buffer.numel(),
                                         ctypes.byref(self.c)), "pnmix_kv4_cache_init")
        self._q, self._kv = (cfg.n_q_heads, cfg.head_dim), (cfg.n_kv_heads, cfg.head_dim)
        self._refs = (ctypes.byref(cfg), ctypes.byref(self.c))

    @property
    def cfg(self) -> KV4Config:
        return KV4Config.from_buffer_copy(self._cfg)

    def __setattr__(self, name, value):
        # the calls' pointers and the tensors' shapes belong together
        if "_refs" in self.__dict__ and (name in self.__dict__ or name == "cfg"):
            raise AttributeError(f"{name} of a KV4Cache stays as it was made; make another cache")
        super().__setattr__(name, value)

    def reset(self, stream=None):
        """Zero the pages and the error word."""
        ctx, s, named = _on(self.device, stream)
        with ctx:
            _check(_lib.pnmix_kv4_cache_reset(self._refs[1], s), "pnmix_kv4_cache_reset")
        if named is not None:
            _used_on(named, self.buffer)

    def _on(self, batch: KV4Batch, stream):
        if not isinstance(batch, KV4Batch):
            raise TypeError("batch must be a KV4Batch")
        if batch.device != self.device:
            raise ValueError(f"the batch is on {batch.device}, the cache on {self.device}")
        return _on(self.device, stream)

    def _used_on(self, stream, batch: KV4Batch, *tensors):
        _used_on(stream, self.buffer, batch.kv_len, batch.page_table, batch.q_start, *tensors)

    def append(self, batch: KV4Batch, k: torch.Tensor, v: torch.Tensor, stream=None):
        """Quantise rows k, v bf16 [n][Hkv][head_dim] (after RoPE) into the batch's places."""
        ctx, s, named = self._on(batch, stream)
        kv = (batch.n_tokens, *self._kv)
        rk, rv = _pack(*_strides(k, kv, self.device, "k")), _pack(*_strides(v, kv, self.device, "v"))
        with ctx:
            _check(_append(self._refs[0], batch.ref, rk, rv, self._refs[1], s), "pnmix_kv4_append")
        if named is not None:
            self._used_on(named, batch, k, v)

    def append_qkv(self, batch: KV4Batch, rope: Rope, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                   positions: torch.Tensor, q_weight=None, k_weight=None, q_out: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
        """norm_rope of q and k and append of the rotated k and v in one pass; returns q_out."""
        if not isinstance(rope, Rope):
            raise TypeError("rope must be a Rope")
        ctx, s, named = self._on(batch, stream)
        n, dev = batch.n_tokens, self.device
        qs, kv = (n, *self._q), (n, *self._kv)
        rq, rk, rv = _pack(*_strides(q, qs, dev, "q")), _pack(*_strides(k, kv, dev, "k")), _pack(*_strides(v, kv, dev, "v"))
        pos = _positions(positions, rope.n_axes, n, dev)
        D = qs[2]
        wq, wk = _weight(q_weight, D, dev, "q_weight"), _weight(k_weight, D, dev, "k_weight")
        with ctx:
            q_out, oq = _out(q_out, qs, q, dev, "q_out")
            _check(_append_qkv(self._refs[0], _byref(rope), batch.ref, rq, rk, rv, wq, wk, pos, oq, self._refs[1], s),
                   "pnmix_kv4_append_qkv")
        if named is not None:
            self._used_on(named, batch, q, k, v, positions, q_weight, k_weight, q_out)
        return q_out

    def read(self, batch: KV4Batch, k_out: torch.Tensor | None = None, v_out: torch.Tensor | None = None,
             stream=None):
        """The batch's rows as the cache holds them: (k, v) bf16 [n][Hkv][head_dim]."""
        ctx, s, named = self._on(batch, stream)
        kv, dev = (batch.n_tokens, *self._kv), self.device
        with ctx:
            if k_out is None:
                k_out = torch.empty(kv, dtype=torch.bfloat16, device=dev)
                ok = _pack(k_out.data_ptr(), kv[1] * kv[2], kv[2])
            else:
                k_out, ok = _out(k_out, kv, k_out, dev, "k_out")
            v_out, ov = _out(v_out, kv, k_out, dev, "v_out")
            _check(_read(self._refs[0], batch.ref, self._refs[1], ok, ov, s), "pnmix_kv4_read")
        if named is not None:
            self._used_on(named, batch, k_out, v_out)
        return k_out, v_out

    def attend(self, batch: KV4Batch, q: torch.Tensor, out: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """Causal attention of q bf16 [n][Hq][head_dim] over the pages -> bf16, same shape.
        The workspace (kv4_workspace_bytes) is taken from torch's allocator for the call unless
        one is given."""
        ctx, s, named = self._on(batch, stream)
        qs, dev = (batch.n_tokens, *self._q), self.device
        rq = _pack(*_strides(q, qs, dev, "q"))
        with ctx:
            out, oo = _out(out, qs, q, dev, "out")
            if workspace is None:
                need = _lib.pnmix_kv4_workspace_bytes(self._refs[0], batch.ref)
                workspace = self.buffer.new_empty(max(need, 256))
            elif workspace.device != dev or workspace.dtype is not torch.uint8 or not workspace.is_contiguous():
                raise TypeError(f"workspace must be contiguous uint8 on {dev}")
            _check(_attention(self._refs[0], batch.ref, rq, self._refs[1], oo, workspace.data_ptr(), workspace.numel(), s),
                   "pnmix_kv4_attention")
        if named is not None:
            self._used_on(named, batch, q, out, workspace)
        return out

    def pages(self) -> torch.Tensor:
        """uint8 view [n_pages][Hkv][blocks][20 * head_dim] (for tests and inspection)."""
        c = self._cfg
        n = self.n_pages * c.n_kv_heads * (c.page_tokens // 16) * 20 * c.head_dim
        return self.buffer[:n].view(self.n_pages, c.n_kv_heads, c.page_tokens // 16, 20 * c.head_dim)

    def read_error(self, clear: bool = True) -> int:
        """The device error word, once all work on the device is done, on whatever stream."""
        val = ctypes.c_uint32(0)
        with torch.cuda.device(self.device):
            st = _lib.pnmix_kv4_read_error(self._refs[1], 1 if clear else 0, ctypes.byref(val))
        if st not in (OK, ERR_DEVICE):
            raise PNMixError(st, "pnmix_kv4_read_error")
        return int(val.value)


def kv4_cache_bytes(cfg: KV4Config, n_pages: int) -> int:
    out = _sz(0)
    _check(_lib.pnmix_kv4_cache_bytes(ctypes.byref(cfg), _count(n_pages, "n_pages"), ctypes.byref(out)),
           "pnmix_kv4_cache_bytes")
    return int(out.value)


def kv4_workspace_bytes(cfg: KV4Config, batch: KV4Batch) -> int:
    return int(_lib.pnmix_kv4_workspace_bytes(_byref(cfg), batch.ref))
