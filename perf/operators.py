"""Cases of the attention-side operators: the per-head norm and rotation of queries and keys (forward, backward,
and the serving form that stores K and V in 4 bits), reading the 4-bit cache back, and attention over it.

``run`` computes them in plain torch operations, or, where ``own`` is true, with this package's entry points.
"""
import math

import torch

own = False

DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-6
GROUP = 32  # dims that share one (scale, minimum) in the cache


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # the smallest training call: 64 tokens of 4 query heads of 64 (hidden 256) in fp32, where latency counts
        dict(name="fwd_small_fp32", op="fwd", B=1, T=64, Hq=4, Hk=1, D=64, rd=64, dtype="fp32", wdtype="fp32",
             layout="packed", interleaved=False),
        # one training micro-batch at hidden 4096: q and k as views of the fused projection's output
        dict(name="fwd_train", op="fwd", B=1, T=8192, Hq=32, Hk=8, D=128, rd=128, dtype="bf16", wdtype="bf16",
             layout="packed", interleaved=False),
        # head-major [B, H, S, D] tensors of odd length, heads of 96 of which 48 rotate, neighbouring pairs
        dict(name="fwd_heads_first", op="fwd", B=3, T=683, Hq=16, Hk=4, D=96, rd=48, dtype="bf16", wdtype="fp32",
             layout="bhsd", interleaved=True),
        # the backward of a long training batch
        dict(name="bwd_train", op="bwd", B=1, T=32768, Hq=32, Hk=8, D=128, rd=128, dtype="bf16", wdtype="fp32",
             layout="packed", interleaved=False),
        # the backward in fp32, an odd token count, heads of 80
        dict(name="bwd_fp32_odd", op="bwd", B=1, T=1021, Hq=12, Hk=2, D=80, rd=80, dtype="fp32", wdtype="fp32",
             layout="dense", interleaved=True),
        # one decoding step of 64 sequences: one new token each, stored to 64 pages
        dict(name="append_decode", op="append", T=64, Hq=32, Hk=8, D=128, rd=128, page=16, seqs=64, wdtype="bf16",
             interleaved=False),
        # prompts of together 4096 tokens stored to the cache
        dict(name="append_prompt", op="append", T=4096, Hq=32, Hk=8, D=128, rd=128, page=64, seqs=3, wdtype="bf16",
             interleaved=False),
        # a short cached prefix read back, heads of 64
        dict(name="read_short", op="read", T=77, Hk=4, D=64, page=32, seqs=2),
        # a long cached prefix read back for a dense attention
        dict(name="read_prefix", op="read", T=32768, Hk=8, D=128, page=64, seqs=1),
        # one sequence with a long history: few rows, a long axis
        dict(name="attend_one_long", op="attend", B=1, n=1, longest=131072, ragged=False, Hq=32, Hk=8, D=128,
             page=64),
        # a serving batch of 64 sequences of mixed lengths
        dict(name="attend_batch", op="attend", B=64, n=1, longest=16384, ragged=True, Hq=32, Hk=8, D=128, page=64),
        # four drafted tokens a sequence checked at once, small pages, heads of 64
        dict(name="attend_drafts", op="attend", B=16, n=4, longest=2000, ragged=True, Hq=24, Hk=8, D=64, page=16),
    ]


def _log(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "append", "read", "attend", "attend"])
    Hq, Hk = rng.choice([(1, 1), (4, 1), (8, 8), (12, 2), (14, 2), (16, 4), (20, 4), (24, 8), (32, 8), (32, 32),
                         (40, 8), (64, 8)])
    if op in ("fwd", "bwd"):
        D = rng.choice([32, 64, 64, 80, 96, 128, 128, 128, 192, 256])
        c = dict(op=op, B=rng.choice([1, 1, 2, 3]), T=_log(rng, 1, 32768), Hq=Hq, Hk=Hk, D=D,
                 rd=rng.choice([D, D, D, 16 * max(1, D // 32)]), dtype=rng.choice(["bf16", "bf16", "fp32"]),
                 wdtype=rng.choice(["bf16", "fp32"]), layout=rng.choice(["packed", "dense", "bhsd"]),
                 interleaved=rng.random() < 0.4)
        c["T"] = max(1, c["T"] // c["B"])
        key = "T"
    else:
        D = rng.choice([64, 128, 128, 256])
        page = rng.choice([16, 32, 64, 128, 256])
        if op == "append":
            c = dict(op=op, T=_log(rng, 1, 16384), Hq=Hq, Hk=Hk, D=D, rd=rng.choice([D, D, D // 2]), page=page, seqs=1,
                     wdtype=rng.choice(["bf16", "fp32"]), interleaved=rng.random() < 0.4)
            c["seqs"] = rng.choice([1, c["T"], _log(rng, 1, c["T"])])
            key = "T"
        elif op == "read":
            c = dict(op=op, T=_log(rng, 1, 131072), Hk=Hk, D=D, page=page, seqs=1)
            c["seqs"] = _log(rng, 1, c["T"])
            key = "T"
        else:
            c = dict(op=op, B=_log(rng, 1, 128), n=rng.choice([1, 1, 1, 2, 3, 5, 8]), longest=_log(rng, 1, 131072),
                     ragged=rng.random() < 0.7, Hq=Hq, Hk=Hk, D=D, page=page)
            key = "longest"
    most = 600e6  # below the largest listed case
    while work(c)["bytes"] > most:
        c[key] = max(1, c[key] * 2 // 3)
    return c


def _lens(case):
    """Cached tokens of each sequence of an "attend" case: fixed by the case, so that its work is."""
    B, top = case["B"], case["longest"]
    if not case["ragged"]:
        return [top] * B
    # spread over [0, longest] in a mixed order; the first is the longest
    return [top if b == 0 else (b * 7919 % B) * top // B for b in range(B)]


def work(case):
    op, D = case["op"], case["D"]
    if op in ("fwd", "bwd"):
        e = 2 if case["dtype"] == "bf16" else 4
        tok = case["B"] * case["T"]
        n = tok * (case["Hq"] + case["Hk"]) * D
        return {"bytes": n * e * (2 if op == "fwd" else 3) + tok * 8 + case["T"] * case["rd"] * 4,
                "flops": n * (8 if op == "fwd" else 16)}
    record = 5 * D // 4  # bytes of one token and head of the cache
    if op == "append":
        tok = case["T"]
        return {"bytes": tok * ((2 * case["Hq"] + 2 * case["Hk"]) * D * 2 + case["Hk"] * (2 * record + 4 * D)
                                + 16 + case["rd"] * 4),
                "flops": tok * (case["Hq"] + 2 * case["Hk"]) * D * 8}
    if op == "read":
        return {"bytes": case["T"] * (case["Hk"] * (record + 4 * D) + 8), "flops": case["T"] * case["Hk"] * D * 4}
    tok, kv = case["B"] * case["n"], sum(_lens(case))
    return {"bytes": kv * case["Hk"] * record + tok * case["Hq"] * (4 * D + 4) + kv // case["page"] * 4,
            "flops": 4 * kv * case["n"] * case["Hq"] * D}


# ------------------------------------------------------------------- the cache's format
# cache: uint8 [pages, kv heads, page / 16, 20 D]; a record of 20 D bytes holds 16 consecutive tokens of one head:
#   [0, 8D) K codes, [8D, 16D) V codes, [16D, 18D) K's (scale, minimum), [18D, 20D) V's.  Two dims a byte, the even one low.
def _k_bytes(D):
    """[16, D/2]: where in a record the byte of dims (2m, 2m+1) of K of token r is."""
    r = torch.arange(16, device=DEV)[:, None]
    m = torch.arange(D // 2, device=DEV)[None, :]
    word = (m // 4 % 4) * (D // 32) + m // 16
    if D == 256:
        word = word ^ ((r & 1) * 4)
    return r * (D // 2) + word * 4 + m % 4


def _v_bytes(D):
    r = torch.arange(16, device=DEV)[:, None]
    m = torch.arange(D // 2, device=DEV)[None, :]
    row = (r & 8) + ((r & 7) >> 1) + 4 * (r & 1)
    part = D // 16
    unit = m // part
    if D == 128:
        unit = unit ^ (((row >> 1) & 1) * 4)
    if D == 256:
        unit = unit ^ ((row & 3) * 2)
    return 8 * D + row * (D // 2) + unit * part + m % part


def _k_scales(D):
    """[16, D/32, 2]: which bf16 of a record is (scale, minimum) of group j of K of token r."""
    r, j, w = (torch.arange(n, device=DEV) for n in (16, D // 32, 2))
    return 8 * D + r[:, None, None] * (D // 16) + j[None, :, None] * 2 + w[None, None, :]


def _v_scales(D):
    r, j, w = (torch.arange(n, device=DEV) for n in (16, D // 32, 2))
    return (9 * D + (r >> 1)[:, None, None] * (D // 8) + j[None, :, None] * 4 + w[None, None, :] * 2
            + (r & 1)[:, None, None])


def _places(D):
    """The tables above, for K and for V: what a program that works on the cache's bytes keeps."""
    return (_k_bytes(D), _k_scales(D)), (_v_bytes(D), _v_scales(D))


def _quantise(x):
    """bf16 [..., D] -> codes uint8 [..., D], (scale, minimum) bf16 [..., D/32, 2]."""
    g = x.float().unflatten(-1, (-1, GROUP))
    z, top = g.amin(-1), g.amax(-1)
    s = (top / 15 - z / 15).to(BF16).float()
    c = ((g - z[..., None]) / s[..., None]).round().clamp(0, 15)
    c = torch.where(s[..., None] > 0, c, 0.0)
    return c.to(torch.uint8).flatten(-2), torch.stack([s, z], -1).to(BF16)


def _value(codes, scales):
    """fp32 values of codes uint8 [..., D/2] and scales bf16 [..., D/32, 2]."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float().unflatten(-1, (-1, GROUP))
    s = scales.float()
    return (c * s[..., 0, None] + s[..., 1, None]).flatten(-2)


def _filled_cache(pages, Hk, page, D, g):
    """A cache whose every slot holds quantised values: keys about as a per-head norm leaves them, values N(0, 1)."""
    nb, D2 = page // 16, D // 2
    cache = torch.empty(pages, Hk, nb, 20 * D, dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 28) // (Hk * page * D))
    for a in range(0, pages, step):
        rec = cache[a:a + step]
        for byte, scale in _places(D):
            x = torch.randn(rec.shape[0], Hk, nb, 16, D, generator=g, device=DEV, dtype=BF16)
            c, sz = _quantise(x)
            rec[..., byte.flatten()] = (c[..., 0::2] | (c[..., 1::2] << 4)).flatten(-2)
            rec.view(BF16)[..., scale.flatten()] = sz.flatten(-3)
    return cache


# ------------------------------------------------------------------------------ inputs
def _angles(P, rd):
    """cos and sin tables, made in 64 bits: fp32 [P, rd/2]."""
    f = 10000.0 ** (-torch.arange(rd // 2, device=DEV, dtype=torch.float64) * 2 / rd)
    a = torch.arange(P, device=DEV, dtype=torch.float64)[:, None] * f
    return a.cos().float(), a.sin().float()


def _heads(case, g, std=1.0):
    """q and k [B, T, H, D] ([T, H, D] where B is 1) in the case's memory layout."""
    B, T, Hq, Hk, D = (case[x] for x in ("B", "T", "Hq", "Hk", "D"))
    dt = BF16 if case["dtype"] == "bf16" else F32

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV, dtype=dt).mul_(std)

    if case["layout"] == "packed":  # [tokens, (q heads, k heads, v heads)], as one projection writes it
        x = normal(B, T, Hq + 2 * Hk, D)
        q, k = x[:, :, :Hq], x[:, :, Hq:Hq + Hk]
    elif case["layout"] == "bhsd":
        q, k = normal(B, Hq, T, D).transpose(1, 2), normal(B, Hk, T, D).transpose(1, 2)
    else:
        q, k = normal(B, T, Hq, D), normal(B, T, Hk, D)
    return (q, k) if B > 1 else (q[0], k[0])


def _weights(case, g):
    dt = BF16 if case["wdtype"] == "bf16" else F32
    return [(1 + 0.1 * torch.randn(case["D"], generator=g, device=DEV)).to(dt) for _ in range(2)]


def _split(T, seqs):
    """T tokens over `seqs` sequences: lengths as equal as they get."""
    return [T // seqs + (1 if i < T % seqs else 0) for i in range(seqs)]


def _slots(case, g, past):
    """Cache pages and, for each token, its slot and position: sequence after sequence; the pages in a random order.
    `past`: tokens that each sequence has already."""
    page = case["page"]
    n = torch.tensor(_split(case["T"], case["seqs"]), device=DEV)
    total = (n + past + page - 1) // page
    first = torch.cumsum(total, 0) - total
    pages = torch.randperm(int(total.sum()) + 3, generator=g, device=DEV)
    seq = torch.repeat_interleave(torch.arange(n.numel(), device=DEV), n)
    pos = torch.arange(case["T"], device=DEV) - (torch.cumsum(n, 0) - n)[seq] + past[seq]
    slot = pages[first[seq] + pos // page] * page + pos % page
    return pages.numel(), slot, pos


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, D = case["op"], case["D"]
    s = {"op": op, "D": D}
    if op in ("fwd", "bwd"):
        s["q"], s["k"] = _heads(case, g)
        if op == "bwd":
            s["gq"], s["gk"] = _heads(dict(case, layout="dense"), g)
        s["wq"], s["wk"] = _weights(case, g)
        # two documents packed into the batch: the positions start again in the middle
        T = case["T"]
        s["pos"] = torch.cat([torch.arange(T - T // 2, device=DEV), torch.arange(T // 2, device=DEV)])
        if case["B"] > 1:
            s["pos"] = s["pos"].expand(case["B"], T).contiguous()
        s["cos"], s["sin"] = _angles(T, case["rd"])
        s["interleaved"] = case["interleaved"]
        return s
    s["places"] = _places(D)
    if op in ("append", "read"):
        n = case["seqs"]
        past = torch.randint(0, 1000 if op == "append" else 1, (n,), generator=g, device=DEV)
        count, s["slots"], s["pos"] = _slots(case, g, past)
        s["page"] = case["page"]
        if op == "read":
            s["cache"] = _filled_cache(count, case["Hk"], case["page"], D, g)
        else:
            s["cache"] = torch.zeros(count, case["Hk"], case["page"] // 16, 20 * D, dtype=torch.uint8, device=DEV)
            x = torch.randn(case["T"], case["Hq"] + 2 * case["Hk"], D, generator=g, device=DEV, dtype=BF16)
            s["q"], s["k"], s["v"] = x.split([case["Hq"], case["Hk"], case["Hk"]], 1)
            s["wq"], s["wk"] = _weights(case, g)
            s["cos"], s["sin"] = _angles(1000 + case["T"], case["rd"])
            s["interleaved"] = case["interleaved"]
    else:
        B, page = case["B"], case["page"]
        lens = torch.tensor(_lens(case), device=DEV)
        need = (lens + page - 1) // page
        count = int(need.sum()) + 2
        width = int(need.max()) + 1
        s["cache"] = _filled_cache(count, case["Hk"], page, D, g)
        pages = torch.randperm(count, generator=g, device=DEV)
        first = torch.cumsum(need, 0) - need
        col = torch.arange(width, device=DEV)
        used = col[None, :] < need[:, None]
        s["table"] = torch.where(used, pages[(first[:, None] + col[None, :]).clamp(max=count - 1)], 0).int()
        s["lens"] = lens.int()
        s["longest"], s["n"] = case["longest"], case["n"]
        s["q"] = torch.randn(B * case["n"], case["Hq"], D, generator=g, device=DEV, dtype=BF16)
        s["cu"] = None if case["n"] == 1 else (torch.arange(B + 1, device=DEV) * case["n"]).int()
    return s


# ------------------------------------------------------------------------- plain forms
def _norm(x, w):
    x = x.float()
    return x * (1 / (x.square().mean(-1, keepdim=True) + EPS).sqrt()) * w.float()


def _turn(n, cos, sin, interleaved):
    """Rotates the first 2 * cos.shape[-1] dims of n [..., H, D] by the angles of its token."""
    cos, sin = cos.unsqueeze(-2), sin.unsqueeze(-2)
    h = cos.shape[-1]
    if interleaved:
        a, b = n[..., 0:2 * h:2], n[..., 1:2 * h:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = n[..., :h], n[..., h:2 * h]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, n[..., 2 * h:]], -1)


def _grad(gy, x, w, cos, sin, interleaved):
    x, g = x.float(), _turn(gy.float(), cos, -sin, interleaved)  # the rotation's transpose turns back
    r = 1 / (x.square().mean(-1, keepdim=True) + EPS).sqrt()
    xh = x * r
    gw = g * w.float()
    dx = r * (gw - xh * (gw * xh).mean(-1, keepdim=True))
    return dx.to(gy.dtype), (g * xh).sum(tuple(range(x.dim() - 1)))




def _read(cache, places, slots, page):
    rec = cache[slots // page, :, slots % page // 16]  # [T, Hk, 20 D]
    r = slots % 16

    def at(byte, scale):
        b = byte[r][:, None].expand(-1, rec.shape[1], -1)
        z = scale.flatten(1)[r][:, None].expand(-1, rec.shape[1], -1)
        return _value(rec.gather(-1, b), rec.view(BF16).gather(-1, z).unflatten(-1, (-1, 2))).to(BF16)

    return at(*places[0]), at(*places[1])


def _store(cache, places, slots, page, k, v):
    D = cache.shape[-1] // 20
    nb, Hk = cache.shape[2], cache.shape[1]
    head = torch.arange(Hk, device=DEV)
    rec = ((slots // page)[:, None] * Hk + head) * nb + (slots % page // 16)[:, None]  # [T, Hk]
    r = slots % 16
    bytes_, halves = cache.view(-1), cache.view(BF16).view(-1)
    for x, (byte, scale) in zip((k, v), places):
        c, sz = _quantise(x)
        bytes_[rec[..., None] * (20 * D) + byte[r][:, None]] = c[..., 0::2] | (c[..., 1::2] << 4)
        halves[rec[..., None, None] * (10 * D) + scale[r][:, None]] = sz


def _attend(s):
    cache, D, n, q = s["cache"], s["D"], s["n"], s["q"]
    B, Hk, Hq, page = s["lens"].numel(), cache.shape[1], q.shape[1], cache.shape[2] * 16
    width = -(-s["longest"] // page)
    rec = cache[s["table"][:, :width].long()]  # [B, pages, Hk, page/16, 20 D]

    def all_of(byte, scale):
        c = rec[..., byte.flatten()].unflatten(-1, (16, -1))
        z = rec.view(BF16)[..., scale.flatten()].unflatten(-1, (16, -1, 2))
        return _value(c, z).permute(0, 2, 1, 3, 4, 5).flatten(2, 4)  # [B, Hk, L, D]

    q = q.float().view(B, n, Hk, Hq // Hk, D).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [B, Hk, n G, D]
    t = q @ all_of(*s["places"][0]).transpose(-1, -2) / math.sqrt(D)
    most = s["lens"][:, None] - n + 1 + torch.arange(n, device=DEV)  # tokens that query i sees
    seen = torch.arange(t.shape[-1], device=DEV) < most.repeat_interleave(Hq // Hk, 1)[:, None, :, None]
    t = torch.where(seen, t, -math.inf)
    m = t.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = (t - m).exp()
    l = p.sum(-1, keepdim=True)
    o = (p @ all_of(*s["places"][1])) / torch.where(l > 0, l, 1.0)
    lse = (m + l.log())[..., 0]
    o = o.view(B, Hk, n, Hq // Hk, D).permute(0, 2, 1, 3, 4).reshape(B * n, Hq, D)
    return o.to(BF16), lse.view(B, Hk, n, Hq // Hk).permute(0, 2, 1, 3).reshape(B * n, Hq)


def run(s):
    op = s["op"]
    if own:
        import rmsnorm_fwd_bwd_persistent_gb300 as rmsn
        if op == "fwd":
            return rmsn.qk_norm_rope_fwd(s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"], s["pos"], EPS,
                                         interleaved=s["interleaved"])
        if op == "bwd":
            return rmsn.qk_norm_rope_bwd(s["gq"], s["gk"], s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"],
                                         s["pos"], EPS, interleaved=s["interleaved"])
        if op == "append":
            q = rmsn.qk_norm_rope_kv4_append(s["q"], s["k"], s["v"], s["wq"], s["wk"], s["cos"], s["sin"], s["pos"],
                                             s["cache"], s["slots"], EPS, interleaved=s["interleaved"])
            return (q, *rmsn.kv4_read(s["cache"], s["slots"]))
        if op == "read":
            return rmsn.kv4_read(s["cache"], s["slots"])
        return rmsn.kv4_attention(s["q"], s["cache"], s["table"], s["lens"], cu_q=s["cu"], max_q=s["n"])
    if op == "read":
        return _read(s["cache"], s["places"], s["slots"], s["page"])
    if op == "attend":
        return _attend(s)
    cos, sin = s["cos"][s["pos"]], s["sin"][s["pos"]]
    if op == "bwd":
        dq, dwq = _grad(s["gq"], s["q"], s["wq"], cos, sin, s["interleaved"])
        dk, dwk = _grad(s["gk"], s["k"], s["wk"], cos, sin, s["interleaved"])
        return dq, dk, dwq, dwk
    q = _turn(_norm(s["q"], s["wq"]), cos, sin, s["interleaved"]).to(s["q"].dtype)
    k = _turn(_norm(s["k"], s["wk"]), cos, sin, s["interleaved"]).to(s["k"].dtype)
    if op == "fwd":
        return q, k
    _store(s["cache"], s["places"], s["slots"], s["page"], k, s["v"])
    return (q, *_read(s["cache"], s["places"], s["slots"], s["page"]))


# -------------------------------------------------------------- from the definitions, in 64 bits
def _exact_head(x, w, cos, sin, interleaved, gy=None):
    """The normed and rotated x, or, with the gradient gy of that, dx and dw: rotations as complex products."""
    x, w = x.double(), w.double()
    half = cos.shape[-1]
    turn = torch.complex(cos.double(), sin.double()).unsqueeze(-2)
    D = x.shape[-1]
    i = torch.arange(half, device=x.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)

    def rotate(v, by):
        z = torch.complex(v[..., a], v[..., b]) * by
        v = v.clone()
        v[..., a], v[..., b] = z.real, z.imag
        return v

    rms = (x.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt()
    if gy is None:
        return rotate(x / rms * w, turn)
    g = rotate(gy.double(), turn.conj())
    dw = torch.einsum("...d,...d->d", g, x / rms)
    g = g * w
    return g / rms - x * (g * x).sum(-1, keepdim=True) / (D * rms.pow(3)), dw


def _exact_cached(cache, slots):
    """K and V [T, Hk, D] of slots in 64 bits, dim by dim from the format's description."""
    D, page = cache.shape[-1] // 20, cache.shape[2] * 16
    dev = cache.device
    rec = cache[torch.div(slots, page, rounding_mode="floor")]
    rec = rec[torch.arange(slots.numel(), device=dev), :, (slots % page) >> 4]
    r = (slots & 15)[:, None]
    d = torch.arange(D, device=dev)[None, :]
    j, t = d // 32, d % 32 // 8
    kword = t * (D // 32) + j
    row = (r // 8) * 8 + (r % 8) // 2 + (r % 2) * 4
    chunk = d // (D // 8)
    if D == 256:
        kword = torch.where(r % 2 == 1, torch.bitwise_xor(kword, torch.full_like(kword, 4)), kword)
        chunk = torch.bitwise_xor(chunk, row % 4 * 2)
    elif D == 128:
        chunk = torch.bitwise_xor(chunk, row // 2 % 2 * 4)
    kat = r * (D // 2) + kword * 4 + d % 8 // 2
    vat = 8 * D + row * (D // 2) + chunk * (D // 16) + d % (D // 8) // 2
    ksc = 8 * D + r * (D // 16) + j * 2
    vsc = 9 * D + (r // 2) * (D // 8) + j * 4 + r % 2
    half = rec.view(BF16)
    out = []
    for at, s, z in ((kat, ksc, ksc + 1), (vat, vsc, vsc + 2)):
        def pick(src, i):
            return src.gather(-1, i[:, None, :].expand(-1, src.shape[1], -1))
        c = torch.bitwise_right_shift(pick(rec, at).long(), 4 * (d % 2)[:, None, :]) % 16
        out.append(c.double() * pick(half, s).double() + pick(half, z).double())
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op, D = s["op"], s["D"]
    if op in ("fwd", "bwd", "append"):
        cos, sin, il = s["cos"][s["pos"]], s["sin"][s["pos"]], s["interleaved"]
    if op == "fwd":
        return tuple(_exact_head(s[x], s["w" + x], cos, sin, il) for x in ("q", "k"))
    if op == "bwd":
        (dq, dwq), (dk, dwk) = (_exact_head(s[x], s["w" + x], cos, sin, il, s["g" + x]) for x in ("q", "k"))
        return dq, dk, dwq, dwk
    if op == "append":
        # what 16 levels between the bounds of each group of 32 (the step and the lower bound held in bf16) leave
        def levels(x):
            x = x.double().to(BF16).double().unflatten(-1, (D // 32, 32))
            low = x.min(-1, keepdim=True).values
            step = ((x.max(-1, keepdim=True).values - low) / 15).to(BF16).double()
            c = torch.where(step > 0, ((x - low) / step.clamp(min=1e-300)).round().clamp(0, 15), 0.0)
            return (low + c * step).flatten(-2)
        return (_exact_head(s["q"], s["wq"], cos, sin, il), levels(_exact_head(s["k"], s["wk"], cos, sin, il)),
                levels(s["v"]))
    if op == "read":
        return tuple(_exact_cached(s["cache"], s["slots"]))
    n, Hq, Hk, page = s["n"], s["q"].shape[1], s["cache"].shape[1], s["cache"].shape[2] * 16
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    for b, length in enumerate(s["lens"].tolist()):
        if length == 0:
            continue
        t = torch.arange(length, device=DEV)
        K, V = _exact_cached(s["cache"], s["table"][b].long()[t // page] * page + t % page)
        for i in range(n):
            m = length - n + 1 + i
            if m <= 0:
                continue
            q = s["q"][b * n + i].double().view(Hk, Hq // Hk, D)
            a = torch.einsum("hgd,thd->hgt", q, K[:m]) / math.sqrt(D)
            lse[b * n + i] = torch.logsumexp(a, -1).flatten()
            o[b * n + i] = torch.einsum("hgt,thd->hgd", torch.softmax(a, -1), V[:m]).reshape(Hq, D)
    return o, lse
