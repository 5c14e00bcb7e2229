"""The norms inside attention and the 4-bit cache: the entry points ``qk_norm_rope_*`` and
``kv4_*`` of ``include/rmsn.h`` for tensors.  The compiled module ``_binding`` checks shapes,
dtypes, devices and strides, allocates the outputs and workspaces that the caller did not pass,
and calls the library on the current stream of the tensors' device; arguments that it refuses
raise TypeError or ValueError, those that the library refuses RmsnError.
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
    """Result and argument types of the entry points (for callers of the C ABI)."""
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
    L.qk_norm_rope_bwd_workspace_bytes.restype = _size
    L.qk_norm_rope_bwd_workspace_bytes.argtypes = [_i64, _int]
    L.kv4_attention_workspace_bytes.restype = _size
    L.kv4_attention_workspace_bytes.argtypes = [_i64, _i64, _int]


_module = None


def load_binding():
    """The compiled module (``csrc/rmsn_binding.cpp``); raises if it was not built."""
    global _module
    if _module is None:
        _lib()  # the library it is linked against
        try:
            from . import _binding
        except ImportError as e:
            raise RuntimeError(
                "the compiled module _binding.so is missing or does not fit this torch: build it "
                "with `python -m rmsnorm_fwd_bwd_persistent_gb300.build`") from e
        _module = _binding
    return _module


def _lib():
    from . import load_library
    return load_library()


def _done(result, what: str):
    """The tensors of a call, or its status raised."""
    if type(result) is int:
        from . import RmsnError
        raise RmsnError(result, what)
    return result


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
    return _done(load_binding().qk_norm_rope_fwd(q, k, wq, wk, cos, sin, positions, eps, interleaved,
                                            q_out, k_out), "qk_norm_rope_fwd")


def qk_norm_rope_bwd_workspace_bytes(D: int, device=None) -> int:
    return int(_lib().qk_norm_rope_bwd_workspace_bytes(D, _index(device)))


def qk_norm_rope_bwd(gq, gk, q, k, wq, wk, cos, sin, positions, eps: float = 1e-6, *,
                     interleaved: bool = False, workspace=None, dq=None, dk=None, dwq=None,
                     dwk=None):
    """Gradients of qk_norm_rope_fwd at (q, k) for the gradients gq and gk of its outputs.
    Returns (dq, dk, dwq, dwk); dwq and dwk are float32 [D] (overwritten)."""
    return _done(load_binding().qk_norm_rope_bwd(gq, gk, q, k, wq, wk, cos, sin, positions, eps,
                                            interleaved, workspace, dq, dk, dwq, dwk),
                 "qk_norm_rope_bwd")


# ---------------------------------------------------------------------------- serving
def kv4_cache_shape(pages: int, kv_heads: int, page_size: int, D: int) -> tuple[int, int, int, int]:
    """Shape of the uint8 tensor that holds a 4-bit cache; page_size is a multiple of 16, D is
    64, 128 or 256.  Its contents need no preparation."""
    if page_size < KV4_BLOCK or page_size % KV4_BLOCK or D not in (64, 128, 256):
        raise ValueError("page_size must be a multiple of 16 and D 64, 128 or 256")
    return pages, kv_heads, page_size // KV4_BLOCK, 20 * D


def qk_norm_rope_kv4_append(q, k, v, wq, wk, cos, sin, positions, cache, slots,
                            eps: float = 1e-6, *, interleaved: bool = False, q_out=None):
    """qk_norm_rope_fwd for serving: returns the normed and rotated q, and stores the normed and
    rotated k and the v as they are to `cache` in 4 bits at `slots` (int64 [T]: page * page_size +
    place in the page; negative: the token is padding and nothing is done for it, its q_out row
    included).  q, k, v are bfloat16 [T, heads, D] by any strides; q_out may be q."""
    return _done(load_binding().qk_norm_rope_kv4_append(q, k, v, wq, wk, cos, sin, positions, cache, slots,
                                                   eps, interleaved, q_out),
                 "qk_norm_rope_kv4_append")[0]


def kv4_read(cache, slots, k=None, v=None):
    """The K and V stored at `slots` (int64 [T]) as bfloat16 [T, kv heads, D]: (k, v).  Rows of a
    negative slot stay as they were."""
    return _done(load_binding().kv4_read(cache, slots, k, v), "kv4_read")


def kv4_attention_workspace_bytes(seqs: int, D: int, device=None) -> int:
    return int(_lib().kv4_attention_workspace_bytes(seqs, D, _index(device)))


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
    return _done(load_binding().kv4_attention(q, cache, page_table, kv_lens, cu_q, max_q, scale, out, lse,
                                         workspace), "kv4_attention")
