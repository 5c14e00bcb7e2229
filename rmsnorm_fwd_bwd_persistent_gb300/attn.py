"""The norms inside attention and the 4-bit cache: the tensor-level side of the entry points
``qk_norm_rope_*`` and ``kv4_*`` of ``include/rmsn.h`` (shapes, dtypes, devices and strides are
checked here or by the library, outputs and workspaces that the caller did not pass are
allocated, everything runs on the current stream of the tensors' device).
"""
from __future__ import annotations

import ctypes
import struct

import torch

_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_int = ctypes.c_int
_f32 = ctypes.c_float
_size = ctypes.c_size_t

KV4_GROUP = 32  # dims that share one scale and minimum
KV4_BLOCK = 16  # tokens per record


class _Heads(ctypes.Structure):
    _fields_ = [("data", _vp), ("batch_stride", _i64), ("token_stride", _i64),
                ("head_stride", _i64), ("heads", _i64)]


class _Rope(ctypes.Structure):
    _fields_ = [("cos", _vp), ("sin", _vp), ("rows", _i64), ("rot_dim", _i64),
                ("neighbours", _int), ("positions", _vp), ("pos_batch_stride", _i64),
                ("pos_token_stride", _i64)]


class _Kv4(ctypes.Structure):
    _fields_ = [("data", _vp), ("pages", _i64), ("kv_heads", _i64), ("page_size", _i64)]


def declare(L) -> None:
    """Result and argument types of the entry points."""
    hp, rp, cp = (ctypes.POINTER(t) for t in (_Heads, _Rope, _Kv4))
    types = {
        "qk_norm_rope_fwd": [hp, hp, _int, _vp, _vp, _int, rp, hp, hp, _i64, _i64, _i64, _f32, _vp],
        "qk_norm_rope_bwd": [hp, hp, hp, hp, _int, _vp, _vp, _int, rp, hp, hp, _vp, _vp, _i64,
                             _i64, _i64, _f32, _vp, _size, _vp],
        "qk_norm_rope_kv4_append": [hp, hp, hp, _vp, _vp, _int, rp, hp, cp, _vp, _i64, _i64, _f32,
                                    _vp],
        "kv4_read": [cp, _vp, hp, hp, _i64, _i64, _vp],
        "kv4_attention": [hp, cp, _vp, _i64, _i64, _vp, _vp, _i64, _i64, _i64, _i64, _f32, hp, _vp,
                          _vp, _size, _vp],
    }
    for name, args in types.items():
        f = getattr(L, name)
        f.restype, f.argtypes = _int, args
        # the wrappers' own handle: structs go in as packed bytes
        f = L[name]
        f.restype = _int
        f.argtypes = [_vp if issubclass(t, ctypes._Pointer) else t for t in args]
        _fast[name] = f
    L.qk_norm_rope_bwd_workspace_bytes.restype = _size
    L.qk_norm_rope_bwd_workspace_bytes.argtypes = [_i64, _int]
    L.kv4_attention_workspace_bytes.restype = _size
    L.kv4_attention_workspace_bytes.argtypes = [_i64, _i64, _int]


# The wrappers run before every launch of kernels that take a few microseconds, so they stay
# short: structs are packed bytes instead of ctypes objects, devices are compared as numbers, the
# current stream is taken as a plain handle, workspace sizes are looked up once.
_fast: dict = {}
_pack_heads = struct.Struct("@Pqqqq").pack
_pack_rope = struct.Struct("@PPqqiPqq").pack
_pack_kv4 = struct.Struct("@Pqqq").pack
_workspaces: dict = {}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda device: torch.cuda.current_stream(device).cuda_stream)
_current_device = torch.cuda.current_device
_DTYPES = {torch.float32: 0, torch.bfloat16: 1}
_F32, _BF16, _I32, _I64 = torch.float32, torch.bfloat16, torch.int32, torch.int64


def _lib():
    from . import load_library
    return load_library()


def _call(name: str, device: int, *args) -> None:
    f = _fast.get(name)
    if f is None:
        _lib()
        f = _fast[name]
    stream = _raw_stream(device)
    if _current_device() == device:
        status = f(*args, stream)
    else:
        with torch.cuda.device(device):
            status = f(*args, stream)
    if status:
        from . import RmsnError
        raise RmsnError(status, name)


def _device(names: str, *tensors) -> int:
    """The CUDA device of all the tensors (named in order in `names`)."""
    try:
        device = tensors[0].get_device()
        for t in tensors:
            if t.get_device() != device or device < 0:
                break
        else:
            return device
    except AttributeError:
        pass
    named = list(zip(names.split(), tensors))
    for name, t in named:
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
    for name, t in named:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor (got {t.device})")
    for name, t in named:
        if t.device != tensors[0].device:
            raise ValueError(f"{name} is on {t.device}, {named[0][0]} on {tensors[0].device}")
    raise AssertionError("unreachable")


def _dtype_code(t: torch.Tensor, name: str) -> int:
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: unsupported dtype {t.dtype} (float32 or bfloat16)")
    return code


def _heads(t: torch.Tensor, name: str) -> bytes:
    st = t.stride()
    if st[-1] != 1 and t.shape[-1] > 1 and t.numel() > 0:
        raise ValueError(f"{name}: the elements of a head must be next to each other")
    return _pack_heads(t.data_ptr(), st[0] if len(st) == 4 else 0, st[-3], st[-2], t.shape[-2])


def _rows(q: torch.Tensor, k: torch.Tensor, batched: bool) -> tuple[int, int, int]:
    """(B, T, D) of q and k; `batched`: they may have a batch axis."""
    a, b = q.shape, k.shape
    n = len(a)
    if len(b) != n or not (n == 3 or (n == 4 and batched)):
        raise ValueError("q and k must be [T, heads, D]" +
                         (" or [B, S, heads, D]" if batched else ""))
    if a[-1] != b[-1] or a[-3] != b[-3] or a[0] != b[0]:
        raise ValueError("q and k must have the same tokens and the same head size")
    if q.dtype is not k.dtype:
        raise TypeError("q and k must be of one dtype")
    return (a[0] if n == 4 else 1), a[-3], a[-1]


def _weights(wq: torch.Tensor, wk: torch.Tensor, D: int) -> int:
    for w, n in ((wq, "wq"), (wk, "wk")):
        if w.dim() != 1 or w.shape[0] != D or not w.is_contiguous():
            raise ValueError(f"{n} must be a contiguous [{D}]")
    if wq.dtype is not wk.dtype:
        raise TypeError("wq and wk must be of one dtype")
    return _dtype_code(wq, "wq")


def _rope(cos, sin, positions, interleaved: bool, B: int, T: int, batched: bool) -> bytes:
    shape = cos.shape
    if len(shape) != 2 or shape != sin.shape:
        raise ValueError("cos and sin must be [positions, rotated dims / 2]")
    if cos.dtype is not _F32 or sin.dtype is not _F32:
        raise TypeError("cos and sin must be float32")
    if not (cos.is_contiguous() and sin.is_contiguous()):
        raise ValueError("cos and sin must be contiguous")
    if positions.dtype is not _I64:
        raise TypeError("positions must be int64")
    p, st = positions.shape, positions.stride()
    if len(p) == 1 and p[0] == T:
        sb, st = 0, st[0]
    elif batched and len(p) == 2 and p[0] == B and p[1] == T:
        sb, st = st
    else:
        raise ValueError("positions must be [T] (or [B, S] beside q of [B, S, heads, D])")
    return _pack_rope(cos.data_ptr(), sin.data_ptr(), shape[0], 2 * shape[1], 1 if interleaved else 0,
                      positions.data_ptr(), sb, st)


def _like(out, t: torch.Tensor, name: str) -> torch.Tensor:
    if out is None:
        return t.new_empty(t.shape)
    _device("input " + name, t, out)
    if out.shape != t.shape or out.dtype is not t.dtype:
        raise ValueError(f"{name} must have the shape and dtype of its input")
    return out


def _buffer(out, shape, dtype, like: torch.Tensor, name: str) -> torch.Tensor:
    if out is None:
        return like.new_empty(shape, dtype=dtype)
    _device("input " + name, like, out)
    if out.shape != shape or out.dtype is not dtype or not out.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {shape}")
    return out


def _scratch(ws, need: int, like: torch.Tensor) -> tuple[torch.Tensor, int]:
    """The caller's workspace or a new one, and its bytes."""
    if ws is None:
        return like.new_empty((max(need, 16),), dtype=torch.uint8), max(need, 16)
    _device("input workspace", like, ws)
    if not ws.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return ws, ws.numel() * ws.element_size()


def _index(device) -> int:
    if device is None:
        return _current_device()
    if isinstance(device, int):
        return device
    device = torch.device(device)
    return device.index if device.index is not None else _current_device()


# --------------------------------------------------------------------------- training
def qk_norm_rope_fwd(q, k, wq, wk, cos, sin, positions, eps: float = 1e-6, *,
                     interleaved: bool = False, q_out=None, k_out=None):
    """RMS norm of every query and key head and the position rotation, in one pass.

    q, k        [T, heads, D] or [B, S, heads, D], float32 or bfloat16, any strides with unit
                stride in D (views of a fused projection, [B, H, S, D].transpose(1, 2), ...)
    wq, wk      [D], shared by the heads
    cos, sin    float32 [positions, rd/2]: the first rd dims of a head turn, in pairs (i, i + rd/2),
                or (2i, 2i + 1) with interleaved=True
    positions   int64 [T] or [B, S]: the table row of every token
    q_out and k_out may be q and k themselves.  Returns (q_out, k_out)."""
    dev = _device("q k wq wk cos sin positions", q, k, wq, wk, cos, sin, positions)
    B, T, D = _rows(q, k, True)
    wd = _weights(wq, wk, D)
    rope = _rope(cos, sin, positions, interleaved, B, T, q.dim() == 4)
    q_out, k_out = _like(q_out, q, "q_out"), _like(k_out, k, "k_out")
    _call("qk_norm_rope_fwd", dev, _heads(q, "q"), _heads(k, "k"), _dtype_code(q, "q"),
          wq.data_ptr(), wk.data_ptr(), wd, rope, _heads(q_out, "q_out"), _heads(k_out, "k_out"),
          B, T, D, eps)
    return q_out, k_out


def qk_norm_rope_bwd_workspace_bytes(D: int, device=None) -> int:
    key = (D, _index(device))
    if key not in _workspaces:
        _workspaces[key] = int(_lib().qk_norm_rope_bwd_workspace_bytes(*key))
    return _workspaces[key]


def qk_norm_rope_bwd(gq, gk, q, k, wq, wk, cos, sin, positions, eps: float = 1e-6, *,
                     interleaved: bool = False, workspace=None, dq=None, dk=None, dwq=None,
                     dwk=None):
    """Gradients of qk_norm_rope_fwd at (q, k) for the gradients gq and gk of its outputs.
    Returns (dq, dk, dwq, dwk); dwq and dwk are float32 [D] (overwritten)."""
    dev = _device("gq gk q k wq wk cos sin positions", gq, gk, q, k, wq, wk, cos, sin, positions)
    B, T, D = _rows(q, k, True)
    for g, x, n in ((gq, q, "gq"), (gk, k, "gk")):
        if g.shape != x.shape or g.dtype is not x.dtype:
            raise ValueError(f"{n} must have the shape and dtype of its input")
    wd = _weights(wq, wk, D)
    rope = _rope(cos, sin, positions, interleaved, B, T, q.dim() == 4)
    dq, dk = _like(dq, q, "dq"), _like(dk, k, "dk")
    dwq = _buffer(dwq, (D,), _F32, q, "dwq")
    dwk = _buffer(dwk, (D,), _F32, q, "dwk")
    ws, ws_bytes = _scratch(workspace, qk_norm_rope_bwd_workspace_bytes(D, dev), q)
    _call("qk_norm_rope_bwd", dev, _heads(gq, "gq"), _heads(gk, "gk"), _heads(q, "q"),
          _heads(k, "k"), _dtype_code(q, "q"), wq.data_ptr(), wk.data_ptr(), wd, rope,
          _heads(dq, "dq"), _heads(dk, "dk"), dwq.data_ptr(), dwk.data_ptr(), B, T, D, eps,
          ws.data_ptr(), ws_bytes)
    return dq, dk, dwq, dwk


# ---------------------------------------------------------------------------- serving
def kv4_cache_shape(pages: int, kv_heads: int, page_size: int, D: int) -> tuple[int, int, int, int]:
    """Shape of the uint8 tensor that holds a 4-bit cache; page_size is a multiple of 16, D is
    64, 128 or 256.  Its contents need no preparation."""
    if page_size < KV4_BLOCK or page_size % KV4_BLOCK or D not in (64, 128, 256):
        raise ValueError("page_size must be a multiple of 16 and D 64, 128 or 256")
    return pages, kv_heads, page_size // KV4_BLOCK, 20 * D


def _cache(cache: torch.Tensor) -> tuple[bytes, int, int]:
    """The packed description, the head size and the kv heads."""
    s = cache.shape
    if len(s) != 4 or cache.dtype is not torch.uint8 or not cache.is_contiguous() or s[3] % 20:
        raise ValueError("cache must be a contiguous uint8 tensor of kv4_cache_shape(...)")
    return _pack_kv4(cache.data_ptr(), s[0], s[1], s[2] * KV4_BLOCK), s[3] // 20, s[1]


def _slots(slots: torch.Tensor, T: int | None):
    if slots.dtype is not _I64 or slots.dim() != 1 or not slots.is_contiguous() or \
            (T is not None and slots.shape[0] != T):
        raise ValueError("slots must be a contiguous int64 [T]")


def qk_norm_rope_kv4_append(q, k, v, wq, wk, cos, sin, positions, cache, slots,
                            eps: float = 1e-6, *, interleaved: bool = False, q_out=None):
    """qk_norm_rope_fwd for serving: returns the normed and rotated q, and stores the normed and
    rotated k and the v as they are to `cache` in 4 bits at `slots` (int64 [T]: page * page_size +
    place in the page; negative: the token is padding and nothing is done for it, its q_out row
    included).  q, k, v are bfloat16 [T, heads, D] by any strides; q_out may be q."""
    dev = _device("q k v wq wk cos sin positions cache slots", q, k, v, wq, wk, cos, sin, positions,
                  cache, slots)
    _, T, D = _rows(q, k, False)
    if q.dtype is not _BF16 or v.dtype is not _BF16:
        raise TypeError("q, k and v must be bfloat16")
    if v.shape != k.shape:
        raise ValueError("v must have k's shape")
    wd = _weights(wq, wk, D)
    rope = _rope(cos, sin, positions, interleaved, 1, T, False)
    kv, cache_d, cache_heads = _cache(cache)
    if cache_d != D or cache_heads != k.shape[1]:
        raise ValueError("the cache is for other heads than k")
    _slots(slots, T)
    q_out = _like(q_out, q, "q_out")
    _call("qk_norm_rope_kv4_append", dev, _heads(q, "q"), _heads(k, "k"), _heads(v, "v"),
          wq.data_ptr(), wk.data_ptr(), wd, rope, _heads(q_out, "q_out"), kv, slots.data_ptr(), T,
          D, eps)
    return q_out


def kv4_read(cache, slots, k=None, v=None):
    """The K and V stored at `slots` (int64 [T]) as bfloat16 [T, kv heads, D]: (k, v).  Rows of a
    negative slot stay as they were."""
    dev = _device("cache slots", cache, slots)
    kv, D, heads = _cache(cache)
    _slots(slots, None)
    shape = (slots.shape[0], heads, D)
    outs = []
    for t, n in ((k, "k"), (v, "v")):
        if t is None:
            t = cache.new_empty(shape, dtype=_BF16)
        else:
            _device("cache " + n, cache, t)
            if t.shape != shape or t.dtype is not _BF16:
                raise ValueError(f"{n} must be bfloat16 [T, kv heads, D]")
        outs.append(t)
    _call("kv4_read", dev, kv, slots.data_ptr(), _heads(outs[0], "k"), _heads(outs[1], "v"),
          shape[0], D)
    return tuple(outs)


def kv4_attention_workspace_bytes(seqs: int, D: int, device=None) -> int:
    key = (seqs, D, _index(device))
    if key not in _workspaces:
        if len(_workspaces) > 4096:  # many batch sizes: start over
            _workspaces.clear()
        _workspaces[key] = int(_lib().kv4_attention_workspace_bytes(*key))
    return _workspaces[key]


def kv4_attention(q, cache, page_table, kv_lens, *, cu_q=None, max_q: int = 1,
                  scale: float | None = None, out=None, lse=None, workspace=None):
    """Attention of the last tokens of every sequence over the 4-bit cache.

    q           bfloat16 [T, heads, D]; heads a multiple of the cache's kv heads
    page_table  int32 [seqs, width]: the pages of every sequence in order
    kv_lens     int32 [seqs]: cached tokens, the query tokens' own included
    cu_q        int32 [seqs + 1]: sequence b has the query tokens cu_q[b] .. cu_q[b+1]-1, its last
                tokens, each of which sees itself and what is before it; None: one each (T = seqs)
    max_q       about the most query tokens of a sequence (for speed; results are right for any)
    scale       of the scores, 1/sqrt(D) where None
    Returns (out bfloat16 [T, heads, D], lse float32 [T, heads]); a query that sees no token gives
    0 and -inf, rows that no sequence has stay as they were."""
    dev = _device("q cache page_table kv_lens", q, cache, page_table, kv_lens)
    if q.dim() != 3 or q.dtype is not _BF16:
        raise ValueError("q must be bfloat16 [T, heads, D]")
    kv, D, kv_heads = _cache(cache)
    T, heads, q_d = q.shape
    if q_d != D or heads % kv_heads != 0:
        raise ValueError("the cache is for other heads than q")
    if page_table.dtype is not _I32 or page_table.dim() != 2 or \
            (page_table.shape[1] > 1 and page_table.stride(1) != 1):
        raise ValueError("page_table must be int32 [seqs, width] with unit stride in the width")
    seqs, width = page_table.shape
    if kv_lens.dtype is not _I32 or kv_lens.shape != (seqs,) or not kv_lens.is_contiguous():
        raise ValueError("kv_lens must be a contiguous int32 [seqs]")
    cu = None
    if cu_q is None:
        if T != seqs:
            raise ValueError("without cu_q there is one query token per sequence")
    else:
        _device("q cu_q", q, cu_q)
        if cu_q.dtype is not _I32 or cu_q.shape != (seqs + 1,) or not cu_q.is_contiguous():
            raise ValueError("cu_q must be a contiguous int32 [seqs + 1]")
        cu = cu_q.data_ptr()
    out = _like(out, q, "out")
    lse = _buffer(lse, (T, heads), _F32, q, "lse")
    ws, ws_bytes = _scratch(workspace, kv4_attention_workspace_bytes(seqs, D, dev), q)
    _call("kv4_attention", dev, _heads(q, "q"), kv, page_table.data_ptr(), width,
          page_table.stride(0) if seqs > 1 else width, kv_lens.data_ptr(), cu, max_q, seqs, T, D,
          D ** -0.5 if scale is None else scale, _heads(out, "out"), lse.data_ptr(), ws.data_ptr(),
          ws_bytes)
    return out, lse
