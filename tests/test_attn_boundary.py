"""The entry points of the norms inside attention and of the 4-bit cache without a GPU: argument
checks return their status before anything touches CUDA, the tensor-level wrappers refuse what the
library cannot take, and the cache's address arithmetic (the header the kernels include, compiled
for the host) covers every byte of a record exactly once and never leaves the cache."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import _attn_ref as R
import rmsnorm_fwd_bwd_persistent_gb300 as rmsn
from rmsnorm_fwd_bwd_persistent_gb300 import attn
from rmsnorm_fwd_bwd_persistent_gb300 import build as rbuild

OK, INVALID, SHAPE, MISALIGNED, WS_SMALL, CUDA = 0, 1, 2, 3, 4, 5
A = 1 << 20  # a fake, aligned "device" address: never dereferenced by these calls
F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def lib():
    rbuild.build()
    return rmsn.load_library()


def heads(n=4, D=64, p=A, sb=None, st=None, sh=None):
    return attn._Heads(p, 0 if sb is None else sb, n * D if st is None else st, D if sh is None else sh, n)


def rope(p=A, rows=10, rd=64, sin=A, pos=A, sb=0, st=1):
    return attn._Rope(p, sin, rows, rd, 0, pos, sb, st)


def cache(p=A, pages=4, hk=2, ps=32):
    return attn._Kv4(p, pages, hk, ps)


def fwd(lib, q=None, k=None, dt=BF16, wq=A, wk=A, wd=F32, r=None, yq=None, yk=None, B=1, T=0, D=64, eps=1e-6):
    q, k = q or heads(), k or heads(2)
    return lib.qk_norm_rope_fwd(q, k, dt, wq, wk, wd, r or rope(rd=min(D, 64)), yq or q, yk or k, B, T, D, eps, None)


def test_fwd_refusals(lib):
    assert fwd(lib) == OK                                        # T == 0: nothing to do
    assert fwd(lib, q=heads(p=None), T=0) == OK
    assert fwd(lib, q=heads(p=None), T=1) == INVALID
    for D in (0, 8, 24, 72, 272, 512, -16):
        assert fwd(lib, D=D) == SHAPE
    for dt in (-1, 2):
        assert fwd(lib, dt=dt) == INVALID
        assert fwd(lib, wd=dt) == INVALID
    for eps in (-1.0, float("nan"), float("inf")):
        assert fwd(lib, eps=eps) == INVALID
    assert fwd(lib, T=-1) == INVALID and fwd(lib, B=-1) == INVALID
    assert fwd(lib, B=1 << 16, T=1 << 15) == SHAPE               # 2^31 tokens
    assert fwd(lib, B=1 << 62, T=4) == SHAPE
    assert fwd(lib, q=heads(0)) == INVALID and fwd(lib, q=heads(4097)) == INVALID
    assert fwd(lib, yq=heads(3)) == INVALID                      # other heads out than in
    assert fwd(lib, q=heads(p=A + 8), T=2) == MISALIGNED
    assert fwd(lib, q=heads(st=260), T=2) == MISALIGNED          # not a multiple of 16 bytes
    assert fwd(lib, dt=F32, q=heads(st=258), T=2) == MISALIGNED
    assert fwd(lib, q=heads(sh=-64), yq=heads(), T=2) == INVALID
    assert fwd(lib, wq=None, T=2) == INVALID and fwd(lib, wk=A + 4, T=2) == MISALIGNED
    # outputs that overlap themselves: heads on each other, tokens on each other, batches too
    assert fwd(lib, yq=heads(sh=0), T=2) == INVALID
    assert fwd(lib, yq=heads(sh=32), T=2) == INVALID
    assert fwd(lib, yq=heads(st=64), T=2) == INVALID
    assert fwd(lib, yk=heads(2, st=0), T=2) == INVALID
    assert fwd(lib, yq=heads(sb=256), B=2, T=2) == INVALID


def test_strides_that_would_leave_64_bits_are_refused(lib):
    far = (1 << 40) - 8
    assert fwd(lib, q=heads(st=far), yq=heads(), T=1 << 30) == INVALID
    assert fwd(lib, yq=heads(st=far), T=1 << 30) == INVALID
    assert fwd(lib, q=heads(sb=far), yq=heads(sb=512), yk=heads(2, sb=256), B=1 << 20, T=2) == INVALID
    assert fwd(lib, q=heads(st=(1 << 40) + 8), yq=heads(), T=2) == INVALID


def test_rope_refusals(lib):
    for rd in (0, 8, 24, 80, -16):
        assert fwd(lib, r=rope(rd=rd)) == SHAPE
    assert fwd(lib, r=rope(rows=0)) == INVALID
    assert fwd(lib, r=rope(st=-1), T=2) == INVALID
    assert fwd(lib, r=rope(p=None), T=2) == INVALID
    assert fwd(lib, r=rope(sin=A + 8), T=2) == MISALIGNED
    assert fwd(lib, r=rope(pos=None), T=2) == INVALID
    assert fwd(lib, r=rope(pos=A + 4), T=2) == MISALIGNED


def test_bwd_refusals(lib):
    def bwd(gq=None, q=None, dq=None, dwq=A, dwk=A, T=2, D=64, ws=A, n=1 << 30):
        q = q or heads()
        return lib.qk_norm_rope_bwd(gq or q, heads(2), q, heads(2), BF16, A, A, F32, rope(), dq or q,
                                    heads(2), dwq, dwk, 1, T, D, 1e-6, ws, n, None)
    assert bwd(gq=heads(5)) == INVALID and bwd(dq=heads(5)) == INVALID
    assert bwd(dwq=None) == INVALID and bwd(dwk=A + 2) == MISALIGNED
    assert bwd(ws=None, n=0) == WS_SMALL and bwd(ws=None) == INVALID and bwd(ws=A + 8) == MISALIGNED
    assert bwd(dq=heads(sh=0)) == INVALID
    assert bwd(D=40) == SHAPE
    assert lib.qk_norm_rope_bwd_workspace_bytes(40, 0) == 0
    assert lib.qk_norm_rope_bwd_workspace_bytes(64, -1) == 0


def test_cache_refusals(lib):
    def append(c=None, k=None, v=None, slots=A, T=2, D=64):
        return lib.qk_norm_rope_kv4_append(heads(), k or heads(2), v or heads(2), A, A, F32, rope(), heads(),
                                           c or cache(), slots, T, D, 1e-6, None)
    assert append(T=0) == OK and append(c=cache(p=None), slots=None, T=0) == OK
    for D in (32, 96, 192):
        assert append(D=D) == SHAPE
    assert append(c=cache(ps=8)) == SHAPE and append(c=cache(ps=24)) == SHAPE
    assert append(c=cache(pages=0)) == INVALID and append(c=cache(hk=0)) == INVALID
    assert append(c=cache(pages=1 << 30, ps=64)) == SHAPE        # 2^31 records or more
    assert append(c=cache(pages=1 << 62, ps=1 << 40)) == SHAPE
    assert append(c=cache(p=None)) == INVALID and append(c=cache(p=A + 8)) == MISALIGNED
    assert append(c=cache(hk=3)) == INVALID                      # other heads than k
    assert append(v=heads(1)) == INVALID
    assert append(slots=None) == INVALID and append(slots=A + 4) == MISALIGNED

    def read(c=None, k=None, v=None, slots=A, T=2, D=64):
        return lib.kv4_read(c or cache(), slots, k or heads(2), v or heads(2), T, D, None)
    assert read(T=0) == OK
    assert read(D=48) == SHAPE and read(k=heads(3)) == INVALID and read(v=heads(2, sh=0)) == INVALID
    assert read(slots=None) == INVALID and read(k=heads(2, p=A + 2)) == MISALIGNED


def test_attention_refusals(lib):
    def att(q=None, c=None, table=A, width=3, stride=3, lens=A, cu=A, max_q=1, seqs=2, T=5, D=64, scale=1.0,
            out=None, lse=A, ws=A, n=1 << 30):
        q = q or heads(4)
        return lib.kv4_attention(q, c or cache(), table, width, stride, lens, cu, max_q, seqs, T, D, scale,
                                 out or heads(4), lse, ws, n, None)
    assert att(T=0) == OK and att(seqs=0) == OK
    assert att(D=96) == SHAPE
    assert att(q=heads(3), out=heads(3)) == INVALID              # 3 heads over 2 kv heads
    assert att(out=heads(2)) == INVALID
    assert att(cu=None) == INVALID                               # then T must be seqs
    assert att(max_q=0) == INVALID and att(seqs=-1) == INVALID
    for s in (float("nan"), float("inf")):
        assert att(scale=s) == INVALID
    assert att(stride=2) == INVALID and att(width=-1) == INVALID
    assert att(width=1 << 30, stride=1 << 30) == SHAPE           # longer than 2^30 tokens
    assert att(width=(1 << 25) + 1, stride=1 << 30) == SHAPE     # the shortest such table
    assert att(T=1 << 29) == SHAPE                               # 2^31 (token, head) columns
    assert att(table=None) == INVALID and att(lens=None) == INVALID
    assert att(lens=A + 2) == MISALIGNED and att(cu=A + 1) == MISALIGNED and att(lse=A + 2) == MISALIGNED
    assert att(ws=None, n=0) == WS_SMALL and att(ws=A + 8) == MISALIGNED
    assert att(out=heads(4, st=64)) == INVALID
    assert lib.kv4_attention_workspace_bytes(2, 96, 0) == 0
    assert lib.kv4_attention_workspace_bytes(-1, 64, 0) == 0


def test_wrappers_refuse_cpu_tensors_and_wrong_types():
    q, k, w = torch.zeros(2, 4, 64), torch.zeros(2, 2, 64), torch.ones(64)
    cs, pos = torch.zeros(8, 32), torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        rmsn.qk_norm_rope_fwd(q, k, w, w, cs, cs, pos)
    with pytest.raises(TypeError, match="Tensor"):
        rmsn.qk_norm_rope_fwd(q, k, w, None, cs, cs, pos)
    with pytest.raises(ValueError, match="CUDA"):
        rmsn.kv4_read(torch.zeros(rmsn.kv4_cache_shape(1, 1, 16, 64), dtype=torch.uint8), pos)
    for bad in ((1, 1, 8, 64), (1, 1, 40, 64), (1, 1, 16, 96)):
        with pytest.raises(ValueError):
            rmsn.kv4_cache_shape(*bad)


# ------------------------------------------------------------------ the cache's addresses
HARNESS = r"""
#include "rmsn_kv4_layout.h"
using namespace rmsn;
extern "C" {
int k_word(int D, int r, int w) { return kv4_k_word(D, r, w); }
int v_unit(int D, int r, int g) { return kv4_v_unit(D, r, g); }
int k_scale(int D, int r, int j) { return kv4_k_scale(D, r, j); }
int v_scale(int D, int r, int j) { return kv4_v_scale(D, r, j); }
int record_bytes(int D) { return kv4_record_bytes(D); }
long long record(long long slot, long long pages, int nb, int hk, int h) {
    return kv4_record(slot, pages, nb, hk, h);
}
}
"""


@pytest.fixture(scope="module")
def layout(tmp_path_factory):
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("layout")
    (d / "h.cpp").write_text(HARNESS)
    csrc = os.path.join(os.path.dirname(rmsn.library_path()), "csrc")
    subprocess.run([cxx, "-O1", "-shared", "-fPIC", "-I", csrc, "-o", str(d / "h.so"), str(d / "h.cpp")],
                   check=True)
    L = ctypes.CDLL(str(d / "h.so"))
    L.record.restype = ctypes.c_longlong
    L.record.argtypes = [ctypes.c_longlong, ctypes.c_longlong, ctypes.c_int, ctypes.c_int, ctypes.c_int]
    return L


@pytest.mark.parametrize("D", [64, 128, 256])
def test_record_bytes_are_covered_once(layout, D):
    n = layout.record_bytes(D)
    assert n == 20 * D and n % 16 == 0
    seen = [0] * n
    for r in range(16):
        for w in range(D // 8):
            at = layout.k_word(D, r, w)
            assert at % 4 == 0
            for i in range(4):
                seen[at + i] += 1
            for d in range(8 * w, 8 * w + 8):
                assert R.k_place(D, r, d) == (at + d % 8 // 2, 4 * (d % 2))
        for g in range(8):
            at, size = layout.v_unit(D, r, g), D // 16
            assert at % size == 0
            for i in range(size):
                seen[at + i] += 1
            for e in range(D // 8):
                assert R.v_place(D, r, g * D // 8 + e) == (at + e // 2, 4 * (e % 2))
        for j in range(D // 32):
            for at in R.k_scale(D, r, j) + R.v_scale(D, r, j):
                seen[at] += 1
                seen[at + 1] += 1
            assert layout.k_scale(D, r, j) == R.k_scale(D, r, j)[0]
            assert layout.v_scale(D, r, j) == R.v_scale(D, r, j)[0]
    assert seen == [1] * n


@pytest.mark.parametrize("D", [64, 128, 256])
def test_fragment_loads_are_whole_and_free_of_bank_conflicts(layout, D):
    """A lane's K words (one per group) lie in aligned pieces of up to 16 bytes, and each phase of a
    shared-memory access (128 bytes) touches every bank once."""
    def phases(addr, size):  # addr: lane -> byte address of its access of `size` bytes
        per = 128 // size if size > 4 else 32
        for p in range(0, 32, per):
            words = set()
            for lane in range(p, p + per):
                words |= {addr[lane] // 4 + i for i in range(size // 4)}
            banks = [w % 32 for w in words]
            assert len(banks) == len(set(banks))

    lanes = [(i // 4, i % 4) for i in range(32)]
    step = min(D // 32, 4)
    for half in (0, 8):
        for u in range(D // 32 // step):
            at = [layout.k_word(D, g + half, t + 4 * step * u) for g, t in lanes]
            for (g, t), a in zip(lanes, at):
                assert a % (4 * step) == 0
                for j in range(step):
                    assert layout.k_word(D, g + half, t + 4 * (step * u + j)) == a + 4 * j
            phases(at, 4 * step)
    for r in (0, 1, 8, 9):
        phases([layout.v_unit(D, 2 * t + r, g) for g, t in lanes], D // 16)


def test_records_stay_inside(layout):
    for pages, nb, hk in ((1, 1, 1), (3, 2, 5), (7, 16, 2)):
        seen = set()
        for slot in range(pages * nb * 16):
            for h in range(hk):
                rec = layout.record(slot, pages, nb, hk, h)
                assert 0 <= rec < pages * nb * hk
                seen.add((rec, slot % 16))
        assert len(seen) == pages * nb * hk * 16
        for slot in (-1, -(1 << 62), pages * nb * 16, (1 << 62)):
            assert layout.record(slot, pages, nb, hk, 0) == -1
    # beyond 32 bits
    assert layout.record((1 << 35) + 5, 1 << 32, 4, 3, 2) == ((1 << 29) * 3 + 2) * 4
