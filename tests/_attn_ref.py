"""64-bit references of the per-head norm + rotation and of attention over the 4-bit cache, the
cache's format written out dim by dim, and the error bounds the GPU tests hold the kernels to.
Everything runs on CPU tensors and shares nothing with the package.

Bounds.  u = 2^-24 is half a step of FP32, half(t) half a step of the output type.  They follow
the kernels' evaluation term by term and are worst cases, element by element:
  sum of squares   at most D/LPR + log2 LPR + 2 <= 22 roundings on a path: 22 u, so rstd 14 u
  n = x rstd w     16 u;  rotation: two products and a sum, 18 u (|na cos| + |nb sin|)
"""
import math

import torch

U = 2.0 ** -24
F64 = torch.float64


def half(dtype):
    return torch.finfo(dtype).eps / 2


# --------------------------------------------------------------------- norm + rotation
def pairs(rd, interleaved):
    i = torch.arange(rd // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rd // 2)


def turn(x, cos, sin, interleaved, back=False, absolute=False):
    """x [..., H, D] with the angles [..., rd/2] of its tokens; `absolute`: of magnitudes."""
    y = x.clone()
    rd = 2 * cos.shape[-1]
    a, b = pairs(rd, interleaved)
    c, s = cos.unsqueeze(-2), sin.unsqueeze(-2)
    if absolute:
        c, s, x = c.abs(), s.abs(), x.abs()
        y = x.clone()
        y[..., a] = x[..., a] * c + x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
        return y
    if back:
        s = -s
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def fwd(x, w, cos, sin, pos, eps, interleaved):
    """(y, bound without the output's rounding)."""
    x, w, c, s = x.to(F64), w.to(F64), cos.to(F64)[pos], sin.to(F64)[pos]
    n = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w
    return turn(n, c, s, interleaved), 20 * U * turn(n, c, s, interleaved, absolute=True)


def bwd(gy, x, w, cos, sin, pos, eps, interleaved):
    """((dx, bound), (dw, bound)) without the output's rounding."""
    gy, x, w, c, s = gy.to(F64), x.to(F64), w.to(F64), cos.to(F64)[pos], sin.to(F64)[pos]
    D = x.shape[-1]
    r = 1 / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    h = turn(gy, c, s, interleaved, back=True)
    ha = turn(gy, c, s, interleaved, absolute=True)
    g, ga = h * w, ha * w.abs()
    dx = r * (g - x * r * r * (g * x).mean(-1, keepdim=True))
    # r 14 u, h 2 u, h w 3 u, the dot 22 u + 3 u, r^2 28 u, and the few products around them
    da = r * (8 * U * ga + 64 * U * x.abs() * r * r * (ga * x.abs()).mean(-1, keepdim=True))
    da = da + 18 * U * dx.abs()
    over = tuple(range(x.dim() - 1))
    return (dx, da), ((h * x * r).sum(over), 24 * U * (ha * x.abs() * r).sum(over))


def assert_within(got, ref, bound, dtype, what=""):
    got = got.detach().cpu().to(F64)
    lim = bound + half(dtype) * (ref.abs() + bound) + 2.0 ** -130
    bad = ~((got - ref).abs() <= lim)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst "
                           f"{float(((got - ref).abs() / lim).nan_to_num(nan=math.inf).max()):.3g} "
                           f"of the bound at {tuple(int(v) for v in bad.nonzero()[0])}")


# --------------------------------------------------------------------------- the cache
def k_place(D, r, d):
    """(byte, shift) in its record of the K code of dim d of token r."""
    j, t = d // 32, d % 32 // 8
    word = t * (D // 32) + j
    if D == 256 and r % 2:
        word ^= 4
    return r * (D // 2) + 4 * word + d % 8 // 2, 4 * (d % 2)


def v_place(D, r, d):
    row = r // 8 * 8 + r % 8 // 2 + r % 2 * 4
    unit = d // (D // 8)
    if D == 128:
        unit ^= row // 2 % 2 * 4
    if D == 256:
        unit ^= row % 4 * 2
    return 8 * D + row * (D // 2) + unit * (D // 16) + d % (D // 8) // 2, 4 * (d % 2)


def k_scale(D, r, j):
    """Bytes of the scale and of the minimum."""
    at = 16 * D + r * (D // 8) + 4 * j
    return at, at + 2


def v_scale(D, r, j):
    at = 18 * D + r // 2 * (D // 4) + 8 * j + 2 * (r % 2)
    return at, at + 4


_tables = {}


def tables(D):
    """Index tables: code bytes and shifts [16, D], scale positions in bf16s [16, D/32, 2], of K and V."""
    if D not in _tables:
        out = []
        for place, scale in ((k_place, k_scale), (v_place, v_scale)):
            p = torch.tensor([[place(D, r, d) for d in range(D)] for r in range(16)])
            s = torch.tensor([[scale(D, r, j) for j in range(D // 32)] for r in range(16)])
            out.append((p[..., 0], p[..., 1], s // 2))
        _tables[D] = out
    return _tables[D]


def quantise(x):
    """bf16 [..., D] -> codes [..., D] (int64), scale and minimum bf16 [..., D/32], in binary32."""
    g = x.float().unflatten(-1, (-1, 32))
    z, top = g.amin(-1), g.amax(-1)
    fifteen = torch.tensor(15.0)
    s = (top / fifteen - z / fifteen).to(torch.bfloat16)
    sf = s.float()[..., None]
    c = ((g - z[..., None]) / sf).round().clamp(0, 15)
    c = torch.where(sf > 0, c, torch.zeros(()))
    bad = ~torch.isfinite(g).all(-1)
    c = torch.where(bad[..., None], torch.zeros(()), c)
    nan = torch.tensor(math.nan, dtype=torch.bfloat16)
    return (c.long().flatten(-2), torch.where(bad, nan, s), torch.where(bad, nan, z.to(torch.bfloat16)))


def store(cache, slots, k, v):
    """Writes bf16 k, v [T, Hk, D] at slots into a copy of the cache (CPU uint8)."""
    cache = cache.clone()
    D, Hk, nb = cache.shape[3] // 20, cache.shape[1], cache.shape[2]
    halves = cache.view(torch.int16)
    for t, slot in enumerate(slots.tolist()):
        if slot < 0 or slot >= cache.shape[0] * nb * 16:
            continue
        page, blk, r = slot // (16 * nb), slot // 16 % nb, slot % 16
        for (byte, shift, sc), x in zip(tables(D), (k[t], v[t])):
            c, s, z = quantise(x)
            for h in range(Hk):
                rec = cache[page, h, blk]
                even, odd = c[h, 0::2], c[h, 1::2]
                rec[byte[r, 0::2]] = (even | (odd << 4)).to(torch.uint8)
                halves[page, h, blk][sc[r, :, 0]] = s[h].view(torch.int16)
                halves[page, h, blk][sc[r, :, 1]] = z[h].view(torch.int16)
    return cache


def cached(cache, slots):
    """FP32 values (c s + z, one rounding) of K and V at slots: [T, Hk, D] each."""
    D, nb = cache.shape[3] // 20, cache.shape[2]
    rec = cache[slots // (16 * nb), :, slots // 16 % nb]
    r = slots % 16
    out = []
    for byte, shift, sc in tables(D):
        at = byte[r][:, None].expand(-1, rec.shape[1], -1)
        c = (rec.gather(-1, at).long() >> shift[r][:, None]) & 15
        s = sc[r].flatten(1)[:, None].expand(-1, rec.shape[1], -1)
        sz = rec.view(torch.bfloat16).gather(-1, s).unflatten(-1, (-1, 2)).to(F64)
        sz = sz.repeat_interleave(32, -2)
        out.append((c.to(F64) * sz[..., 0] + sz[..., 1]).float())
    return out


def cached_parts(cache, slots):
    """|scale * code| + |minimum| of K, as magnitudes for the score's bound (FP64 [T, Hk, D])."""
    D, nb = cache.shape[3] // 20, cache.shape[2]
    rec = cache[slots // (16 * nb), :, slots // 16 % nb]
    r = slots % 16
    byte, shift, sc = tables(D)[0]
    c = (rec.gather(-1, byte[r][:, None].expand(-1, rec.shape[1], -1)).long() >> shift[r][:, None]) & 15
    s = sc[r].flatten(1)[:, None].expand(-1, rec.shape[1], -1)
    sz = rec.view(torch.bfloat16).gather(-1, s).unflatten(-1, (-1, 2)).to(F64).repeat_interleave(32, -2)
    return (c.to(F64) * sz[..., 0]).abs() + sz[..., 1].abs()


# --------------------------------------------------------------------------- attention
def attention(q, cache, table, lens, cu, scale, skip=None):
    """(o, lse, bound of o, bound of lse) in 64 bits; `skip`: page ids whose tokens are left out.

    Scores: 2^-18 of scale sum |q| (s c + |z|): at most 40 FP32 additions, some of them truncated,
    on a path.  The probabilities and V's values are rounded to bf16 once each."""
    T, H, D = q.shape
    Hk, ps, pages = cache.shape[1], cache.shape[2] * 16, cache.shape[0]
    o = torch.zeros(T, H, D, dtype=F64)
    lse = torch.full((T, H), -math.inf, dtype=F64)
    ob, lb = torch.zeros_like(o), torch.zeros_like(lse)
    seen_rows = torch.zeros(T, dtype=torch.bool)
    for b in range(len(lens)):
        q0, q1 = (b, b + 1) if cu is None else (int(cu[b]), int(cu[b + 1]))
        n, L = q1 - q0, min(max(int(lens[b]), 0), table.shape[1] * ps)
        seen_rows[q0:q1] = True
        t = torch.arange(L)
        page = table[b].long()[t // ps] if L else t
        ok = (page >= 0) & (page < pages)
        slots = torch.where(ok, page, 0) * ps + t % ps
        if L:
            K, V = (x.to(F64) for x in cached(cache, slots))
            A = cached_parts(cache, slots)
        for i in range(n):
            m = L - n + 1 + i
            if m <= 0 or not ok[:m].any():
                continue
            keep = ok[:m]
            x = q[q0 + i].to(F64).view(Hk, H // Hk, D)
            s = scale * torch.einsum("hgd,thd->hgt", x, K[:m])[..., keep]
            a = abs(scale) * torch.einsum("hgd,thd->hgt", x.abs(), A[:m])[..., keep]
            delta = 2.0 ** -18 * a.amax(-1)
            p = torch.softmax(s, -1)
            o[q0 + i] = torch.einsum("hgt,thd->hgd", p, V[:m][keep]).reshape(H, D)
            lse[q0 + i] = torch.logsumexp(s, -1).flatten()
            pv = torch.einsum("hgt,thd->hgd", p, V[:m][keep].abs())
            ob[q0 + i] = (pv * (2.0 ** -7 + 2.0 ** -14 + 2 * delta[..., None])).reshape(H, D)
            lb[q0 + i] = (delta + 2.0 ** -20).flatten() + 4 * U * lse[q0 + i].abs()
    return o, lse, ob, lb, seen_rows
