"""The norms inside attention and the 4-bit cache: the tensor-level side of the entry points
``qk_norm_rope_*`` and ``kv4_*`` of ``include/rmsn.h`` (shapes, dtypes, devices and strides are
checked here or by the library, outputs and workspaces that the caller did not pass are
allocated, everything runs on the current stream of the tensors' device).
"""
from __future__ import annotations

import ctypes

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
    L.qk_norm_rope_fwd.restype = _int
    L.qk_norm_rope_fwd.argtypes = [hp, hp, _int, _vp, _vp, _int, rp, hp, hp, _i64, _i64, _i64,
                                   _f32, _vp]
    L.qk_norm_rope_bwd_workspace_bytes.restype = _size
    L.qk_norm_rope_bwd_workspace_bytes.argtypes = [_i64, _int]
    L.qk_norm_rope_bwd.restype = _int
    L.qk_norm_rope_bwd.argtypes = [hp, hp, hp, hp, _int, _vp, _vp, _int, rp, hp, hp, _vp, _vp,
                                   _i64, _i64, _i64, _f32, _vp, _size, _vp]
    L.qk_norm_rope_kv4_append.restype = _int
    L.qk_norm_rope_kv4_append.argtypes = [hp, hp, hp, _vp, _vp, _int, rp, hp, cp, _vp, _i64, _i64,
                                          _f32, _vp]
    L.kv4_read.restype = _int
    L.kv4_read.argtypes = [cp, _vp, hp, hp, _i64, _i64, _vp]
    L.kv4_attention_workspace_bytes.restype = _size
    L.kv4_attention_workspace_bytes.argtypes = [_i64, _i64, _int]
    L.kv4_attention.restype = _int
    L.kv4_attention.argtypes = [hp, cp, _vp, _i64, _i64, _vp, _vp, _i64, _i64, _i64, _i64, _f32,
                                hp, _vp, _vp, _size, _vp]


def _lib():
    from . import load_library
    return load_library()


def _check(status: int, what: str):
    from . import _check as check
    check(status, what)


def _on_gpu(first: torch.Tensor, **others):
    """Every tensor is a CUDA tensor on the device of `first`."""
    for name, t in others.items():
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
    for name, t in others.items():
        if t.device.type != "cuda":
            raise ValueError(f"{name} must be a CUDA tensor (got {t.device})")
        if t.device != first.device:
            raise ValueError(f"{name} is on {t.device}, the first tensor on {first.device}")


def _dtype_code(t: torch.Tensor, name: str) -> int:
    from . import RMSN_BF16, RMSN_F32
    if t.dtype == torch.float32:
        return RMSN_F32
    if t.dtype == torch.bfloat16:
        return RMSN_BF16
    raise TypeError(f"{name}: unsupported dtype {t.dtype} (float32 or bfloat16)")


def _ptr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _stream(t: torch.Tensor) -> int:
    return torch.cuda.current_stream(t.device).cuda_stream


def _heads(t: torch.Tensor, name: str) -> _Heads:
    if t.stride(-1) != 1 and t.shape[-1] > 1 and t.numel() > 0:
        raise ValueError(f"{name}: the elements of a head must be next to each other")
    sb = t.stride(0) if t.dim() == 4 else 0
    return _Heads(t.data_ptr(), sb, t.stride(-3), t.stride(-2), t.shape[-2])


def _rows(q: torch.Tensor, k: torch.Tensor, dims) -> tuple[int, int, int]:
    """(B, T, D) of q and k; `dims`: how many dimensions they may have."""
    if q.dim() not in dims or k.dim() != q.dim():
        raise ValueError("q and k must be [T, heads, D]" +
                         (" or [B, S, heads, D]" if 4 in dims else ""))
    if k.shape[:-2] != q.shape[:-2] or k.shape[-1] != q.shape[-1]:
        raise ValueError("q and k must have the same tokens and the same head size")
    if k.dtype != q.dtype:
        raise TypeError("q and k must be of one dtype")
    return (q.shape[0] if q.dim() == 4 else 1), q.shape[-3], q.shape[-1]


def _weights(wq: torch.Tensor, wk: torch.Tensor, D: int) -> int:
    for w, n in ((wq, "wq"), (wk, "wk")):
        if w.shape != (D,) or not w.is_contiguous():
            raise ValueError(f"{n} must be a contiguous [{D}]")
    if wq.dtype != wk.dtype:
        raise TypeError("wq and wk must be of one dtype")
    return _dtype_code(wq, "wq")


def _rope(cos, sin, positions, interleaved: bool, B: int, T: int, batched: bool) -> _Rope:
    if cos.dim() != 2 or cos.shape != sin.shape:
        raise ValueError("cos and sin must be [positions, rotated dims / 2]")
    for t, n in ((cos, "cos"), (sin, "sin")):
        if t.dtype != torch.float32:
            raise TypeError(f"{n} must be float32")
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    if positions.dtype != torch.int64:
        raise TypeError("positions must be int64")
    if batched and positions.dim() == 2 and positions.shape == (B, T):
        sb, st = positions.stride()
    elif positions.shape == (T,):
        sb, st = 0, positions.stride(0)
    else:
        raise ValueError("positions must be [T] (or [B, S] beside q of [B, S, heads, D])")
    return _Rope(cos.data_ptr(), sin.data_ptr(), cos.shape[0], 2 * cos.shape[1],
                 int(bool(interleaved)), positions.data_ptr(), sb, st)


def _like(out, t: torch.Tensor, name: str) -> torch.Tensor:
    if out is None:
        return torch.empty(t.shape, device=t.device, dtype=t.dtype)
    _on_gpu(t, **{name: out})
    if out.shape != t.shape or out.dtype != t.dtype:
        raise ValueError(f"{name} must have the shape and dtype of its input")
    return out


def _buffer(out, shape, dtype, like: torch.Tensor, name: str) -> torch.Tensor:
    if out is None:
        return torch.empty(shape, device=like.device, dtype=dtype)
    _on_gpu(like, **{name: out})
    if out.shape != tuple(shape) or out.dtype != dtype or not out.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {tuple(shape)}")
    return out


def _scratch(ws, need: int, like: torch.Tensor) -> torch.Tensor:
    if ws is None:
        return torch.empty(max(need, 16), device=like.device, dtype=torch.uint8)
    _on_gpu(like, workspace=ws)
    if not ws.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return ws


def _bytes(t: torch.Tensor) -> int:
    return t.numel() * t.element_size()


def _index(device) -> int:
    if device is None:
        return torch.cuda.current_device()
    if isinstance(device, int):
        return device
    device = torch.device(device)
    return device.index if device.index is not None else torch.cuda.current_device()


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
    _on_gpu(q, q=q, k=k, wq=wq, wk=wk, cos=cos, sin=sin, positions=positions)
    B, T, D = _rows(q, k, (3, 4))
    wd = _weights(wq, wk, D)
    rope = _rope(cos, sin, positions, interleaved, B, T, q.dim() == 4)
    q_out, k_out = _like(q_out, q, "q_out"), _like(k_out, k, "k_out")
    with torch.cuda.device(q.device):
        st = _lib().qk_norm_rope_fwd(_heads(q, "q"), _heads(k, "k"), _dtype_code(q, "q"), _ptr(wq),
                                     _ptr(wk), wd, rope, _heads(q_out, "q_out"),
                                     _heads(k_out, "k_out"), B, T, D, float(eps), _stream(q))
    _check(st, "qk_norm_rope_fwd")
    return q_out, k_out


def qk_norm_rope_bwd_workspace_bytes(D: int, device=None) -> int:
    return int(_lib().qk_norm_rope_bwd_workspace_bytes(int(D), _index(device)))


def qk_norm_rope_bwd(gq, gk, q, k, wq, wk, cos, sin, positions, eps: float = 1e-6, *,
                     interleaved: bool = False, workspace=None, dq=None, dk=None, dwq=None,
                     dwk=None):
    """Gradients of qk_norm_rope_fwd at (q, k) for the gradients gq and gk of its outputs.
    Returns (dq, dk, dwq, dwk); dwq and dwk are float32 [D] (overwritten)."""
    _on_gpu(q, gq=gq, gk=gk, q=q, k=k, wq=wq, wk=wk, cos=cos, sin=sin, positions=positions)
    B, T, D = _rows(q, k, (3, 4))
    for g, x, n in ((gq, q, "gq"), (gk, k, "gk")):
        if g.shape != x.shape or g.dtype != x.dtype:
            raise ValueError(f"{n} must have the shape and dtype of its input")
    wd = _weights(wq, wk, D)
    rope = _rope(cos, sin, positions, interleaved, B, T, q.dim() == 4)
    dq, dk = _like(dq, q, "dq"), _like(dk, k, "dk")
    dwq = _buffer(dwq, (D,), torch.float32, q, "dwq")
    dwk = _buffer(dwk, (D,), torch.float32, q, "dwk")
    with torch.cuda.device(q.device):
        ws = _scratch(workspace, qk_norm_rope_bwd_workspace_bytes(D, q.device), q)
        st = _lib().qk_norm_rope_bwd(_heads(gq, "gq"), _heads(gk, "gk"), _heads(q, "q"),
                                     _heads(k, "k"), _dtype_code(q, "q"), _ptr(wq), _ptr(wk), wd,
                                     rope, _heads(dq, "dq"), _heads(dk, "dk"), _ptr(dwq),
                                     _ptr(dwk), B, T, D, float(eps), _ptr(ws), _bytes(ws),
                                     _stream(q))
    _check(st, "qk_norm_rope_bwd")
    return dq, dk, dwq, dwk


# ---------------------------------------------------------------------------- serving
def kv4_cache_shape(pages: int, kv_heads: int, page_size: int, D: int) -> tuple[int, int, int, int]:
    """Shape of the uint8 tensor that holds a 4-bit cache; page_size is a multiple of 16, D is
    64, 128 or 256.  Its contents need no preparation."""
    if page_size < KV4_BLOCK or page_size % KV4_BLOCK or D not in (64, 128, 256):
        raise ValueError("page_size must be a multiple of 16 and D 64, 128 or 256")
    return pages, kv_heads, page_size // KV4_BLOCK, 20 * D


def _cache(cache: torch.Tensor) -> tuple[_Kv4, int]:
    if cache.dim() != 4 or cache.dtype != torch.uint8 or not cache.is_contiguous() or \
            cache.shape[3] % 20 != 0:
        raise ValueError("cache must be a contiguous uint8 tensor of kv4_cache_shape(...)")
    return (_Kv4(cache.data_ptr(), cache.shape[0], cache.shape[1], cache.shape[2] * KV4_BLOCK),
            cache.shape[3] // 20)


def _slots(slots: torch.Tensor, T: int | None):
    if slots.dtype != torch.int64 or slots.dim() != 1 or not slots.is_contiguous() or \
            (T is not None and slots.shape[0] != T):
        raise ValueError("slots must be a contiguous int64 [T]")


def qk_norm_rope_kv4_append(q, k, v, wq, wk, cos, sin, positions, cache, slots,
                            eps: float = 1e-6, *, interleaved: bool = False, q_out=None):
    """qk_norm_rope_fwd for serving: returns the normed and rotated q, and stores the normed and
    rotated k and the v as they are to `cache` in 4 bits at `slots` (int64 [T]: page * page_size +
    place in the page; negative: the token is padding and nothing is done for it, its q_out row
    included).  q, k, v are bfloat16 [T, heads, D] by any strides; q_out may be q."""
    _on_gpu(q, q=q, k=k, v=v, wq=wq, wk=wk, cos=cos, sin=sin, positions=positions, cache=cache,
            slots=slots)
    _, T, D = _rows(q, k, (3,))
    if q.dtype != torch.bfloat16 or v.dtype != torch.bfloat16:
        raise TypeError("q, k and v must be bfloat16")
    if v.shape != k.shape:
        raise ValueError("v must have k's shape")
    wd = _weights(wq, wk, D)
    rope = _rope(cos, sin, positions, interleaved, 1, T, False)
    kv, cache_d = _cache(cache)
    if cache_d != D or cache.shape[1] != k.shape[1]:
        raise ValueError("the cache is for other heads than k")
    _slots(slots, T)
    q_out = _like(q_out, q, "q_out")
    with torch.cuda.device(q.device):
        st = _lib().qk_norm_rope_kv4_append(_heads(q, "q"), _heads(k, "k"), _heads(v, "v"),
                                            _ptr(wq), _ptr(wk), wd, rope, _heads(q_out, "q_out"),
                                            kv, _ptr(slots), T, D, float(eps), _stream(q))
    _check(st, "qk_norm_rope_kv4_append")
    return q_out


def kv4_read(cache, slots, k=None, v=None):
    """The K and V stored at `slots` (int64 [T]) as bfloat16 [T, kv heads, D]: (k, v).  Rows of a
    negative slot stay as they were."""
    _on_gpu(cache, cache=cache, slots=slots)
    kv, D = _cache(cache)
    _slots(slots, None)
    shape = (slots.shape[0], cache.shape[1], D)
    outs = []
    for t, n in ((k, "k"), (v, "v")):
        if t is None:
            t = torch.empty(shape, device=cache.device, dtype=torch.bfloat16)
        _on_gpu(cache, **{n: t})
        if t.shape != shape or t.dtype != torch.bfloat16:
            raise ValueError(f"{n} must be bfloat16 [T, kv heads, D]")
        outs.append(t)
    with torch.cuda.device(cache.device):
        st = _lib().kv4_read(kv, _ptr(slots), _heads(outs[0], "k"), _heads(outs[1], "v"),
                             shape[0], D, _stream(cache))
    _check(st, "kv4_read")
    return tuple(outs)


def kv4_attention_workspace_bytes(seqs: int, D: int, device=None) -> int:
    return int(_lib().kv4_attention_workspace_bytes(int(seqs), int(D), _index(device)))


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
    _on_gpu(q, q=q, cache=cache, page_table=page_table, kv_lens=kv_lens)
    if q.dim() != 3 or q.dtype != torch.bfloat16:
        raise ValueError("q must be bfloat16 [T, heads, D]")
    kv, D = _cache(cache)
    T, heads = q.shape[0], q.shape[1]
    if q.shape[2] != D or heads % cache.shape[1] != 0:
        raise ValueError("the cache is for other heads than q")
    if page_table.dtype != torch.int32 or page_table.dim() != 2 or \
            (page_table.shape[1] > 1 and page_table.stride(1) != 1):
        raise ValueError("page_table must be int32 [seqs, width] with unit stride in the width")
    seqs, width = page_table.shape
    if kv_lens.dtype != torch.int32 or kv_lens.shape != (seqs,) or not kv_lens.is_contiguous():
        raise ValueError("kv_lens must be a contiguous int32 [seqs]")
    if cu_q is None:
        if T != seqs:
            raise ValueError("without cu_q there is one query token per sequence")
    else:
        _on_gpu(q, cu_q=cu_q)
        if cu_q.dtype != torch.int32 or cu_q.shape != (seqs + 1,) or not cu_q.is_contiguous():
            raise ValueError("cu_q must be a contiguous int32 [seqs + 1]")
    out = _like(out, q, "out")
    lse = _buffer(lse, (T, heads), torch.float32, q, "lse")
    stride = page_table.stride(0) if seqs > 1 else width
    with torch.cuda.device(q.device):
        ws = _scratch(workspace, kv4_attention_workspace_bytes(seqs, D, q.device), q)
        st = _lib().kv4_attention(_heads(q, "q"), kv, _ptr(page_table), width, stride,
                                  _ptr(kv_lens), _ptr(cu_q), int(max_q), seqs, T, D,
                                  float(D ** -0.5 if scale is None else scale),
                                  _heads(out, "out"), _ptr(lse), _ptr(ws), _bytes(ws), _stream(q))
    _check(st, "kv4_attention")
    return out, lse
