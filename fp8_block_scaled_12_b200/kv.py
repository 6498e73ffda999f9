"""Paged FP8 key-value cache: its writers, its reader and decode attention.

Between the projections of a decoder's attention block (FP8 linear layers) stand the
norm and rotation of q and k, the cache, and the attention that reads it:

    cache = KVCache(num_pages=4096, page_size=64, heads=8, head_dim=128)
    table = rope_table(max_pos=131072, rotary_dim=128)
    q = qk_norm_rope_kv_write(q, k, v, positions, table, slots, cache, wq, wk)   # one pass
    o = paged_attention(q, cache, block_table, lens)                             # one new token each
    k, v = kv_read(cache, block_table, offsets, rows)                            # back as bf16

As in the rest of the binding, ``fp8_*`` functions take preallocated outputs and the
short names allocate them.  Tensors must live on one device; a call made while another
device is current switches to theirs.  Outputs that the short names allocate belong to the
stream the call runs on.
"""
from __future__ import annotations

import contextlib
import ctypes
import math

import torch

from . import E4M3, E5M2, SCALE_FP32, SCALE_UE8M0, _check, _expect, _u8, lib

__all__ = ["KVCache", "rope_table", "paged_attention_ws_bytes", "fp8_qk_norm_rope", "fp8_kv_write",
           "fp8_qk_norm_rope_kv_write", "fp8_kv_read", "fp8_paged_attention", "qk_norm_rope", "kv_write",
           "qk_norm_rope_kv_write", "kv_read", "paged_attention"]


class _CacheStruct(ctypes.Structure):
    """fp8_kv_cache of the C header."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale")] +
                [(n, ctypes.c_int64) for n in ("num_pages", "page_size", "heads", "head_dim", "page_stride",
                                               "head_stride", "token_stride")] +
                [("fmt", ctypes.c_int), ("scale_fmt", ctypes.c_int)])


def _declare() -> None:
    vp, i64, ci, fl = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
    rows = [vp, i64, i64]                          # pointer, token stride, head stride
    rope = [vp, vp, fl, vp, i64, i64, ci, vp]      # wq, wk, eps, cos_sin, max_pos, R, interleaved, pos
    lib.fp8_qk_norm_rope.argtypes = rows + rows + [i64] * 4 + rope + rows + rows + [vp]
    lib.fp8_kv_write.argtypes = rows + rows + [i64, vp, vp, vp]
    lib.fp8_qk_norm_rope_kv_write.argtypes = rows * 3 + [i64, i64] + rope + [vp, vp] + rows + [vp]
    lib.fp8_kv_read.argtypes = [vp, vp, i64, i64, vp, i64, i64, vp, vp, vp]
    lib.fp8_paged_attention_ws_bytes.argtypes = [i64, i64, vp]
    lib.fp8_paged_attention_ws_bytes.restype = i64
    lib.fp8_paged_attention.argtypes = rows + [i64, i64, vp, vp, i64, i64, vp, fl, i64, vp, vp, vp, i64, vp]
    for name in ("fp8_qk_norm_rope", "fp8_kv_write", "fp8_qk_norm_rope_kv_write", "fp8_kv_read",
                 "fp8_paged_attention"):
        getattr(lib, name).restype = ci


_declare()


class KVCache:
    """Device memory of a paged cache: codes `k`, `v` (uint8, logical shape [num_pages, heads,
    page_size, head_dim]) and scales `k_scale`, `v_scale` (fp32 [num_pages, heads, page_size]).
    `layout`: "HND" keeps a head's tokens of a page together, "NHD" a token's heads.  The
    memory is not initialised: readers use only what was written.  The tensors and formats may
    be replaced by others that fit (all checks of `wrap` again; sizes follow from them); the
    memory of those that are there has to stay in its place."""

    _PARTS = ("k", "v", "k_scale", "v_scale", "fmt", "scale_fmt")

    def __init__(self, num_pages: int, page_size: int, heads: int, head_dim: int, fmt: int = E4M3,
                 scale_fmt: int = SCALE_FP32, layout: str = "HND", device="cuda"):
        if layout not in ("HND", "NHD"):
            raise ValueError(f"layout must be HND or NHD, got {layout}")
        inner = (heads, page_size) if layout == "HND" else (page_size, heads)

        def codes():
            x = torch.empty((num_pages, *inner, head_dim), dtype=torch.uint8, device=device)
            return x if layout == "HND" else x.transpose(1, 2)

        def scales():
            return torch.empty((num_pages, heads, page_size), dtype=torch.float32, device=device)

        self._set(codes(), codes(), scales(), scales(), fmt, scale_fmt)

    @classmethod
    def wrap(cls, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor, fmt: int = E4M3,
             scale_fmt: int = SCALE_FP32) -> "KVCache":
        """A cache over memory that exists already (views of one allocation, say): k and v of
        the shape above with equal strides and contiguous channels."""
        c = cls.__new__(cls)
        c._set(k, v, k_scale, v_scale, fmt, scale_fmt)
        return c

    def _set(self, k, v, k_scale, v_scale, fmt, scale_fmt):
        k, v = _u8(k), _u8(v)
        if k.dim() != 4:
            raise ValueError(f"k has shape {tuple(k.shape)}, expected [num_pages, heads, page_size, head_dim]")
        _expect(v, tuple(k.shape), "v")
        if k.stride() != v.stride() or k.stride(3) != 1:
            raise ValueError(f"k and v need equal strides and contiguous channels, got {k.stride()} and {v.stride()}")
        if fmt not in (E4M3, E5M2) or scale_fmt not in (SCALE_FP32, SCALE_UE8M0):
            raise ValueError(f"unknown code format {fmt} or scale format {scale_fmt}")
        pages, heads, page, dim = k.shape
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            _expect(t, (pages, heads, page), name, torch.float32)
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
        if any(t.device != k.device for t in (v, k_scale, v_scale)):
            raise ValueError("the cache's tensors live on different devices")
        # a structure of its own each time: calls and copies of this object may hold the last one
        struct = _CacheStruct(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), pages, page, heads,
                              dim, k.stride(0), k.stride(1), k.stride(2), fmt, scale_fmt)
        vars(self).update(k=k, v=v, k_scale=k_scale, v_scale=v_scale, fmt=fmt, scale_fmt=scale_fmt, num_pages=pages,
                          heads=heads, page_size=page, head_dim=dim, device=k.device, index=k.get_device(),
                          _ref=ctypes.byref(struct))

    def __setattr__(self, name, value):
        if name in self._PARTS:
            self._set(**{n: value if n == name else getattr(self, n) for n in self._PARTS})
        elif name in vars(self):
            raise AttributeError(f"{name} of a cache follows from its tensors")
        else:
            super().__setattr__(name, value)


def rope_table(max_pos: int, rotary_dim: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """fp32 [max_pos, rotary_dim]: cosines, then sines, of p * base^(-2i / rotary_dim).  The angles
    are formed in 64 bits: in 32, those of far positions lose the turn's fraction."""
    freq = base ** (-torch.arange(0, rotary_dim, 2, dtype=torch.float64, device=device) / rotary_dim)
    a = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * freq
    return torch.cat([a.cos(), a.sin()], 1).float()


# ------------------------------------------------------------ argument checks
# A decode step makes these calls once a layer, so the checks touch every property of a tensor
# once and the current device and stream are read without building torch objects.
_BF16, _F32, _I64, _I32 = torch.bfloat16, torch.float32, torch.int64, torch.int32


def _check_devices(index: int, *tensors) -> None:
    """The tensors live on the CUDA device of that index (-1: not a CUDA device)."""
    if index < 0:
        raise ValueError("fp8 library tensors must live on a CUDA device")
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError(f"a tensor lives on {t.device}, the others on cuda:{index}")


def _call(name: str, fn, index: int, stream, args) -> None:
    """fn(*args, stream) with the device `index` current; the current stream unless one is given."""
    if torch._C._cuda_getDevice() != index:
        with torch.cuda.device(index):
            return _call(name, fn, index, stream, args)
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(index)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    code = fn(*args, stream)
    if code:
        _check(name, code)


def _alloc(device: torch.device, stream):
    """The context in which a short name allocates: the stream that will write the memory."""
    if stream is None:
        return contextlib.nullcontext()
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device)
    return torch.cuda.stream(stream)


def _rows(t: torch.Tensor, name: str, shape: tuple) -> tuple:
    """(pointer, token stride, head stride) of a bf16 [tokens, heads, D] view."""
    if t.dtype is not _BF16:
        raise TypeError(f"{name} has dtype {t.dtype}, expected torch.bfloat16")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    tok, head, one = t.stride()
    if one != 1:
        raise ValueError(f"{name} needs contiguous channels, got strides {t.stride()}")
    return t.data_ptr(), tok, head


def _vec(t: torch.Tensor, name: str, n: int, dtype) -> int:
    if t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected a contiguous ({n},)")
    return t.data_ptr()


def _rope(positions, cos_sin, T: int) -> tuple:
    """(cos_sin pointer, max_pos, R, pos pointer); no rotation without a table."""
    if cos_sin is None:
        return None, 0, 0, None
    if cos_sin.dtype is not _F32:
        raise TypeError(f"cos_sin has dtype {cos_sin.dtype}, expected torch.float32")
    if cos_sin.dim() != 2 or not cos_sin.is_contiguous():
        raise ValueError(f"cos_sin must be a contiguous [max_pos, R], got {tuple(cos_sin.shape)}")
    if positions is None:
        raise ValueError("a rotation needs positions")
    return cos_sin.data_ptr(), *cos_sin.shape, _vec(positions, "positions", T, _I64)


def _weight(w, name: str, D: int):
    return None if w is None else _vec(w, name, D, _BF16)


def _table(table: torch.Tensor, B: int) -> tuple:
    """(pointer, row stride, pages per row)."""
    if table.dtype is not _I32:
        raise TypeError(f"table has dtype {table.dtype}, expected torch.int32")
    if table.dim() != 2:
        raise ValueError(f"table must be [{B}, max_pages], got {tuple(table.shape)}")
    rows, pages = table.shape
    row, one = table.stride()
    if rows != B or (pages > 1 and one != 1):
        raise ValueError(f"table must be [{B}, max_pages] with contiguous rows, got {tuple(table.shape)}")
    # the row stride of one row, or of an empty one, may be anything: no second row is read
    return table.data_ptr(), max(row, pages) if B <= 1 else row, pages


# ---------------------------------------------------------------- C names
def fp8_qk_norm_rope(q, k, positions, cos_sin, q_out, k_out, wq=None, wk=None, eps: float = 1e-6,
                     interleaved: bool = False, stream=None) -> None:
    """RMS norm per head (weights wq, wk bf16 [D]; None: no norm) and rotation of bf16 q [T, Hq, D]
    and k [T, Hk, D] (views with any token and head strides) into q_out, k_out, which may be q
    and k.  cos_sin: rope_table's fp32 [max_pos, R], or None."""
    T, Hq, D = shape = q.shape
    Hk = k.shape[1]
    index = q.get_device()
    _check_devices(index, k, positions, cos_sin, q_out, k_out, wq, wk)
    table, max_pos, R, pos = _rope(positions, cos_sin, T)
    _call("fp8_qk_norm_rope", lib.fp8_qk_norm_rope, index, stream,
          (*_rows(q, "q", shape), *_rows(k, "k", (T, Hk, D)), T, Hq, Hk, D, _weight(wq, "wq", D),
           _weight(wk, "wk", D), eps, table, max_pos, R, 1 if interleaved else 0, pos,
           *_rows(q_out, "q_out", shape), *_rows(k_out, "k_out", (T, Hk, D))))


def fp8_kv_write(k, v, slots, cache: KVCache, stream=None) -> None:
    """bf16 k, v [T, heads, D] quantised into slots (int64 [T], page * page_size + row; one
    outside the cache, such as -1, is skipped; they must differ) of the cache."""
    T = k.shape[0]
    shape = (T, cache.heads, cache.head_dim)
    index = cache.index
    _check_devices(index, k, v, slots)
    _call("fp8_kv_write", lib.fp8_kv_write, index, stream,
          (*_rows(k, "k", shape), *_rows(v, "v", shape), T, _vec(slots, "slots", T, _I64), cache._ref))


def fp8_qk_norm_rope_kv_write(q, k, v, positions, cos_sin, slots, cache: KVCache, q_out, wq=None, wk=None,
                              eps: float = 1e-6, interleaved: bool = False, stream=None) -> None:
    """fp8_qk_norm_rope and fp8_kv_write in one pass: q into q_out, k (quantised from fp32) and v
    into the cache."""
    T, Hq, D = q_shape = q.shape
    shape = (T, cache.heads, cache.head_dim)
    if D != cache.head_dim:
        raise ValueError(f"q has head dimension {D}, the cache {cache.head_dim}")
    index = cache.index
    _check_devices(index, q, k, v, positions, cos_sin, slots, q_out, wq, wk)
    table, max_pos, R, pos = _rope(positions, cos_sin, T)
    _call("fp8_qk_norm_rope_kv_write", lib.fp8_qk_norm_rope_kv_write, index, stream,
          (*_rows(q, "q", q_shape), *_rows(k, "k", shape), *_rows(v, "v", shape), T, Hq, _weight(wq, "wq", D),
           _weight(wk, "wk", D), eps, table, max_pos, R, 1 if interleaved else 0, pos,
           _vec(slots, "slots", T, _I64), cache._ref, *_rows(q_out, "q_out", q_shape)))


def fp8_kv_read(cache: KVCache, table, offsets, k_out, v_out, stream=None) -> None:
    """The first tokens of each sequence back as bf16: rows [offsets[b], offsets[b + 1]) of k_out
    and v_out [rows, heads, D] are tokens 0, 1, ... of the pages table[b] (int32 [B, max_pages];
    offsets int32 [B + 1] on the device).  Rows outside every range are not written."""
    B = offsets.shape[0] - 1
    rows = k_out.shape[0]
    index = cache.index
    _check_devices(index, table, offsets, k_out, v_out)
    for t, n in ((k_out, "k_out"), (v_out, "v_out")):
        _expect(t, (rows, cache.heads, cache.head_dim), n, _BF16)
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    _call("fp8_kv_read", lib.fp8_kv_read, index, stream,
          (cache._ref, *_table(table, B), _vec(offsets, "offsets", B + 1, _I32), B, rows, k_out.data_ptr(),
           v_out.data_ptr()))


def paged_attention_ws_bytes(B: int, Hq: int, cache: KVCache) -> int:
    """Workspace of fp8_paged_attention for B sequences and Hq query heads, on the cache's device."""
    with torch.cuda.device(cache.index) if cache.index >= 0 else contextlib.nullcontext():
        n = lib.fp8_paged_attention_ws_bytes(B, Hq, cache._ref)
    if n == 0:
        raise ValueError(f"no attention of {Hq} query heads over this cache of {cache.heads} kv heads, "
                         f"head dimension {cache.head_dim} and pages of {cache.page_size}")
    return n


def fp8_paged_attention(q, cache: KVCache, table, lens, out, workspace, lse=None, scale: float | None = None,
                        window: int = 0, stream=None) -> None:
    """Attention of one new token per sequence: bf16 q [B, Hq, D] over tokens [0, lens[b]) (int32
    [B] on the device; the last `window` of them if window > 0) of the pages table[b] -> out bf16
    [B, Hq, D], and the log of the softmax's sum in lse (fp32 [B, Hq]) when given.  scale:
    1 / sqrt(D) unless given.  workspace: paged_attention_ws_bytes(B, Hq, cache) bytes; calls that
    share it must be ordered on one stream."""
    B, Hq, D = shape = q.shape
    if D != cache.head_dim:
        raise ValueError(f"q has head dimension {D}, the cache {cache.head_dim}")
    index = cache.index
    _check_devices(index, q, table, lens, out, workspace, lse)
    if out.dtype is not _BF16:
        raise TypeError(f"out has dtype {out.dtype}, expected torch.bfloat16")
    if out.shape != shape:
        raise ValueError(f"out has shape {tuple(out.shape)}, expected {tuple(shape)}")
    if not out.is_contiguous() or not workspace.is_contiguous():
        raise ValueError("out and workspace must be contiguous")
    if lse is not None:
        _expect(lse, (B, Hq), "lse", _F32)
        if not lse.is_contiguous():
            raise ValueError("lse must be contiguous")
    _call("fp8_paged_attention", lib.fp8_paged_attention, index, stream,
          (*_rows(q, "q", shape), B, Hq, cache._ref, *_table(table, B), _vec(lens, "lens", B, _I32),
           1.0 / math.sqrt(D) if scale is None else scale, window, out.data_ptr(),
           None if lse is None else lse.data_ptr(), workspace.data_ptr(), workspace.nbytes))


# ------------------------------------------------------ allocating wrappers
def qk_norm_rope(q, k, positions, cos_sin, wq=None, wk=None, eps: float = 1e-6, interleaved: bool = False,
                 stream=None):
    with _alloc(q.device, stream):
        qo, ko = (torch.empty(t.shape, dtype=torch.bfloat16, device=t.device) for t in (q, k))
    fp8_qk_norm_rope(q, k, positions, cos_sin, qo, ko, wq, wk, eps, interleaved, stream)
    return qo, ko


kv_write = fp8_kv_write


def qk_norm_rope_kv_write(q, k, v, positions, cos_sin, slots, cache: KVCache, wq=None, wk=None, eps: float = 1e-6,
                          interleaved: bool = False, stream=None):
    with _alloc(q.device, stream):
        qo = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    fp8_qk_norm_rope_kv_write(q, k, v, positions, cos_sin, slots, cache, qo, wq, wk, eps, interleaved, stream)
    return qo


def kv_read(cache: KVCache, table, offsets, rows: int, stream=None):
    """As fp8_kv_read with `rows` = offsets[-1], which the host has to know."""
    with _alloc(cache.device, stream):
        ko, vo = (torch.empty((rows, cache.heads, cache.head_dim), dtype=torch.bfloat16, device=cache.device)
                  for _ in range(2))
    fp8_kv_read(cache, table, offsets, ko, vo, stream)
    return ko, vo


def paged_attention(q, cache: KVCache, table, lens, scale: float | None = None, window: int = 0,
                    return_lse: bool = False, stream=None):
    with _alloc(cache.device, stream):
        out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
        ws = torch.empty((paged_attention_ws_bytes(q.shape[0], q.shape[1], cache),), dtype=torch.uint8,
                         device=q.device)
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device) if return_lse else None
    fp8_paged_attention(q, cache, table, lens, out, ws, lse, scale, window, stream)
    return (out, lse) if return_lse else out
