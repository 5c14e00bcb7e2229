"""The 4-bit cache: what the append stores (bit by bit), what is read back, and attention over it
against 64 bits: head sizes and groups, lengths from none to long, pages, several query tokens, empty
rows, NaN where it may and may not reach, bad indices, graphs and shared workspaces."""
import math

import pytest
import torch

import _attn_ref as R
import rmsnorm_fwd_bwd_persistent_gb300 as rmsn

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-6
ERR_INDEX = 8


def angles(P, rd):
    f = 10000.0 ** (-torch.arange(rd // 2, dtype=torch.float64) * 2 / rd)
    a = torch.arange(P, dtype=torch.float64)[:, None] * f
    return a.cos().float(), a.sin().float()


def empty_cache(pages, Hk, ps, D, fill=0xAB):
    return torch.full(rmsn.kv4_cache_shape(pages, Hk, ps, D), fill, dtype=torch.uint8, device=DEV)


def append_inputs(T, Hq, Hk, D, rd, seed, wd=F32):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, Hq + 2 * Hk, D, generator=g).to(BF16)
    w = [(1 + 0.1 * torch.randn(D, generator=g)).to(wd) for _ in range(2)]
    pos = torch.randint(0, 50, (T,), generator=g)
    return x, w, angles(50, rd), pos, g


@pytest.mark.parametrize("T,Hq,Hk,D,rd,ps,nb", [
    (1, 1, 1, 64, 64, 16, False), (1, 32, 8, 128, 128, 16, False), (37, 8, 2, 128, 128, 32, False),
    (37, 8, 2, 128, 64, 48, True), (50, 5, 5, 64, 32, 16, False), (33, 4, 1, 256, 256, 64, False),
    (20, 3, 3, 256, 64, 16, True), (200, 32, 8, 128, 128, 256, True), (70, 14, 2, 64, 64, 16, True),
    (9, 16, 1, 128, 16, 16, False)])
def test_append_and_read(T, Hq, Hk, D, rd, ps, nb):
    x, (wq, wk), (cos, sin), pos, g = append_inputs(T, Hq, Hk, D, rd, seed=T + D)
    pages = -(-T // ps) + 2
    slots = torch.randperm(pages * ps, generator=g)[:T]
    if T > 8:
        slots[3] = slots[T - 1] = -1  # padding
    cache = empty_cache(pages, Hk, ps, D)
    before = cache.cpu()
    xd = x.to(DEV)
    q, k, v = xd.split([Hq, Hk, Hk], 1)
    rest = [t.to(DEV) for t in (wq, wk, cos, sin, pos)]
    yq, yk = rmsn.qk_norm_rope_fwd(q, k, *rest, EPS, interleaved=nb)
    out = rmsn.qk_norm_rope_kv4_append(q, k, v, *rest, cache, slots.to(DEV), EPS, interleaved=nb,
                                       q_out=torch.full_like(yq, 7.0))
    used = slots >= 0
    assert torch.equal(out[used.to(DEV)], yq[used.to(DEV)]) and (out[~used.to(DEV)] == 7).all()
    # the cache's bytes are the quantised bf16 values, and nothing else was touched
    assert torch.equal(cache.cpu(), R.store(before, slots, yk.cpu(), x[:, Hq + Hk:]))
    ko, vo = (torch.full((T, Hk, D), 7.0, dtype=BF16, device=DEV) for _ in range(2))
    rmsn.kv4_read(cache, slots.to(DEV), ko, vo)
    for got, ref in zip((ko, vo), R.cached(cache.cpu(), slots.clamp(min=0))):
        assert torch.equal(got.cpu()[used], ref.to(BF16)[used])
        assert (got.cpu()[~used] == 7).all()
    # and what is read is within half a step of what was stored: s/2, and 15 s 2^-9 by the scale's rounding
    for got, src in ((ko, yk.cpu()), (vo, x[:, Hq + Hk:])):
        _, s, _ = R.quantise(src[used])
        lim = s.float().repeat_interleave(32, -1) * (0.5 + 15 * 2.0 ** -8) + 2.0 ** -8 * src[used].float().abs() + 1e-2
        assert ((got.cpu()[used].float() - src[used].float()).abs() <= lim).all()
    assert rmsn.rmsn_device_status() == 0


@pytest.mark.parametrize("D", [64, 128, 256])
def test_read_into_strided_rows(D):
    """Rows that start on 16 bytes but not on 32, and rows with gaps: the same values, the gaps untouched."""
    cache, table, g = filled([40], 3, 16, D, seed=D)
    slots = torch.cat([table[0, :3].long()[torch.arange(40) // 16] * 16 + torch.arange(40) % 16, torch.tensor([-1])])
    k, v = rmsn.kv4_read(cache.to(DEV), slots.to(DEV), *(torch.zeros(41, 3, D, dtype=BF16, device=DEV) for _ in "kv"))
    for off, gap in ((8, 0), (0, 8), (16, 16)):
        buf = torch.full((2, 41 * 3 * (D + gap) + 32), 7.0, dtype=BF16, device=DEV)
        ko, vo = (b[off:off + 41 * 3 * (D + gap)].view(41, 3, D + gap)[..., :D] for b in buf)
        rmsn.kv4_read(cache.to(DEV), slots.to(DEV), ko, vo)
        assert torch.equal(ko[:40], k[:40]) and torch.equal(vo[:40], v[:40])
        ko[:40] = 7
        vo[:40] = 7
        assert (buf == 7).all()
    assert rmsn.rmsn_device_status() == 0


def test_append_in_place_and_overwriting():
    T, Hq, Hk, D = 24, 4, 2, 128
    cache = empty_cache(3, Hk, 16, D)
    ref = cache.cpu()
    for seed in (1, 2):  # the same slots twice: tokens are stored independently
        x, (wq, wk), (cos, sin), pos, _ = append_inputs(T, Hq, Hk, D, D, seed)
        n = T if seed == 1 else 7
        slots = torch.arange(5, 5 + T)[:n] * (1 if seed == 1 else 3)
        xd = x[:n].to(DEV)
        q, k, v = xd.split([Hq, Hk, Hk], 1)
        rest = [t.to(DEV) for t in (wq, wk, cos, sin, pos[:n])]
        yq, yk = rmsn.qk_norm_rope_fwd(q, k, *rest, EPS)
        assert rmsn.qk_norm_rope_kv4_append(q, k, v, *rest, cache, slots.to(DEV), EPS, q_out=q) is q
        assert torch.equal(q, yq)
        ref = R.store(ref, slots, yk.cpu(), x[:n, Hq + Hk:])
        assert torch.equal(cache.cpu(), ref)


def test_quantiser_edges():
    """Constant groups, one huge element, tiny ranges, signed zeros, infinities and NaN, through V."""
    Hk, D = 1, 64
    rows = [torch.zeros(D), torch.full((D,), -3.25), torch.randn(D, generator=torch.Generator().manual_seed(0))]
    rows.append(torch.where(torch.arange(D) == 5, 1e30, rows[2]))
    rows.append(1.0 + torch.arange(D) % 2 * 2.0 ** -7)
    rows.append(torch.arange(D) * 1e-40)
    rows.append(torch.where(torch.arange(D) % 2 == 0, -0.0, 0.0))
    rows.append(torch.where(torch.arange(D) == 40, math.inf, rows[2]))
    rows.append(torch.where(torch.arange(D) == 3, math.nan, rows[2]))
    rows.append(torch.where(torch.arange(D) == 3, -math.inf, rows[2]))
    rows.append(rows[2] * 1e38)
    v = torch.stack(rows).to(BF16)[:, None]
    T = v.shape[0]
    x, (wq, wk), (cos, sin), pos, _ = append_inputs(T, 1, 1, D, D, 3)
    cache = empty_cache(1, Hk, 16, D)
    rest = [t.to(DEV) for t in (wq, wk, cos, sin, pos)]
    slots = torch.arange(T)
    k = x[:, 1:2].to(DEV)
    yk = rmsn.qk_norm_rope_fwd(x[:, :1].to(DEV), k, *rest, EPS)[1]
    before = cache.cpu()
    rmsn.qk_norm_rope_kv4_append(x[:, :1].to(DEV), k, v.to(DEV), *rest, cache, slots.to(DEV), EPS)
    assert torch.equal(cache.cpu(), R.store(before, slots, yk.cpu(), v))
    got = rmsn.kv4_read(cache, slots.to(DEV))[1].cpu().float()[:, 0]
    assert (got[0] == 0).all() and (got[1] == -3.25).all() and (got[6] == 0).all()
    assert torch.equal(got[4], v[4, 0].float())
    for row, group in ((7, 1), (8, 0), (9, 0)):
        assert torch.isnan(got[row, 32 * group:32 * group + 32]).all()
        assert torch.isfinite(got[row, 32 - 32 * group:64 - 32 * group]).all()
    # the last row: its second group holds an infinity in bf16 (a draw above 3.4 times 1e38), its first none
    fine = torch.isfinite(v[10, 0].float()).view(2, 32).all(1)
    assert fine.tolist() == [True, False]
    assert torch.isfinite(got[10, :32]).all() and torch.isnan(got[10, 32:]).all()


@pytest.mark.parametrize("bad", [96, 1 << 40, (1 << 62)])
def test_append_and_read_bad_slots(bad):
    T, Hq, Hk, D = 12, 4, 2, 64
    x, (wq, wk), (cos, sin), pos, _ = append_inputs(T, Hq, Hk, D, D, 5)
    cache = empty_cache(3, Hk, 32, D)
    slots = torch.arange(T) * 7
    slots[4] = bad
    pos[6] = 50  # not a table row: the token is left out, its V too
    before = cache.cpu()
    q, k, v = x.to(DEV).split([Hq, Hk, Hk], 1)
    rest = [t.to(DEV) for t in (wq, wk, cos, sin, pos)]
    assert rmsn.rmsn_device_status() == 0
    yq = torch.full((T, Hq, D), 7.0, dtype=BF16, device=DEV)
    rmsn.qk_norm_rope_kv4_append(q, k, v, *rest, cache, slots.to(DEV), EPS, q_out=yq)
    assert rmsn.rmsn_device_status() == ERR_INDEX
    assert (yq[4] == 7).all() and (yq[6] == 7).all() and not (yq[5] == 7).all()
    rest[-1] = pos.clamp(max=49).to(DEV)
    yk = rmsn.qk_norm_rope_fwd(q, k, *rest, EPS)[1]
    slots[6] = -1
    assert torch.equal(cache.cpu(), R.store(before, slots, yk.cpu(), x[:, Hq + Hk:]))
    ko, vo = (torch.full((T, Hk, D), 7.0, dtype=BF16, device=DEV) for _ in range(2))
    rmsn.kv4_read(cache, slots.to(DEV), ko, vo)
    assert rmsn.rmsn_device_status() == ERR_INDEX
    assert (ko[4] == 7).all() and (vo[4] == 7).all()
    assert rmsn.rmsn_device_status() == 0


# ----------------------------------------------------------------------------- attention
def filled(lens, Hk, ps, D, seed, spare=2, std=1.0):
    """A cache with K and V of sequences of these lengths, pages in a random order (CPU tensors)."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-max(n, 0) // ps) for n in lens]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=g)
    table = torch.full((len(lens), max(need + [1]) + 1), 2 ** 31 - 1, dtype=torch.int32)  # unread entries
    cache = torch.randint(0, 256, rmsn.kv4_cache_shape(pages, Hk, ps, D), generator=g, dtype=torch.uint8)
    at = 0
    slots = []
    for b, n in enumerate(lens):
        table[b, :need[b]] = order[at:at + need[b]].int()
        t = torch.arange(max(n, 0))
        slots.append(order[at + t // ps] * ps + t % ps)
        at += need[b]
    slots = torch.cat(slots)
    # every 16-token record quantised at once: codes and scales by the tables
    T = slots.numel()
    k, v = ((torch.randn(T, Hk, D, generator=g) * std).to(BF16) for _ in range(2))
    rec = slots // (16 * (ps // 16)), slots // 16 % (ps // 16), slots % 16
    flat, half = cache.view(-1), cache.view(torch.int16).view(-1)
    for (byte, shift, sc), x in zip(R.tables(D), (k, v)):
        c, s, z = R.quantise(x)
        for h in range(Hk):
            base = ((rec[0] * Hk + h) * (ps // 16) + rec[1]) * 20 * D
            flat[(base[:, None] + byte[rec[2]][:, 0::2])] = (c[:, h, 0::2] | (c[:, h, 1::2] << 4)).to(torch.uint8)
            half[(base[:, None] // 2 + sc[rec[2]][..., 0])] = s[:, h].view(torch.int16)
            half[(base[:, None] // 2 + sc[rec[2]][..., 1])] = z[:, h].view(torch.int16)
    return cache, table, g


def check(q, cache, table, lens, cu=None, max_q=1, scale=None, rms=True, status=0):
    D = q.shape[-1]
    lens = torch.as_tensor(lens, dtype=torch.int32)
    cud = None if cu is None else torch.as_tensor(cu, dtype=torch.int32)
    o0 = torch.full(q.shape, 7.0, dtype=BF16, device=DEV)
    l0 = torch.full(q.shape[:2], 7.0, device=DEV)
    o, lse = rmsn.kv4_attention(q.to(DEV), cache.to(DEV), table.to(DEV), lens.to(DEV),
                                cu_q=None if cu is None else cud.to(DEV), max_q=max_q, scale=scale, out=o0, lse=l0)
    assert rmsn.rmsn_device_status() == status
    ro, rl, ob, lb, rows = R.attention(q, cache, table, lens, cud, D ** -0.5 if scale is None else scale)
    assert (o.cpu()[~rows] == 7).all() and (lse.cpu()[~rows] == 7).all()
    R.assert_within(o[rows.to(DEV)], ro[rows], ob[rows], BF16, "o")
    got, want = lse.cpu()[rows].double(), rl[rows]
    assert torch.equal(torch.isinf(got), torch.isinf(want))
    f = torch.isfinite(want)
    assert ((got[f] - want[f]).abs() <= lb[rows][f] + 2.0 ** -22 * want[f].abs()).all()
    if rms and float(ro.norm()) > 0:
        # three roundings to bf16 (p, v, o), each of rms at most 2^-8 / sqrt(3) of its value
        assert float((o.cpu()[rows].double() - ro[rows]).norm() / ro[rows].norm()) <= 2.0 ** -8
    return o, lse


@pytest.mark.parametrize("Hq,Hk,D", [(8, 1, 128), (8, 8, 128), (32, 8, 128), (14, 2, 64), (12, 2, 256), (20, 4, 128),
                                     (10, 1, 64), (40, 1, 128), (24, 1, 256), (3, 3, 64)])
@pytest.mark.parametrize("lens,ps", [([1], 16), ([17, 0, 5, 160, 1], 16), ([300, 64, 65, 63], 64), ([1000], 32)])
def test_one_token_each(Hq, Hk, D, lens, ps):
    cache, table, g = filled(lens, Hk, ps, D, seed=len(lens) + D + Hq)
    check(torch.randn(len(lens), Hq, D, generator=g).to(BF16), cache, table, lens, max_q=1)


@pytest.mark.parametrize("max_q", [1, 3, 9])
@pytest.mark.parametrize("Hq,Hk,D", [(8, 1, 128), (6, 3, 64), (4, 1, 256), (16, 2, 64)])
def test_several_tokens(Hq, Hk, D, max_q):
    """Sequences with none to nine query tokens, one with more queries than tokens, rows that no
    sequence has before, between (none) and behind."""
    lens, counts, ps = [100, 33, 4, 0, 250, 16], [4, 1, 9, 2, 0, 3], 16
    cu = [2]
    for n in counts:
        cu.append(cu[-1] + n)
    cache, table, g = filled(lens, Hk, ps, D, seed=D + Hq)
    q = torch.randn(cu[-1] + 5, Hq, D, generator=g).to(BF16)
    check(q, cache, table, lens, cu, max_q)


@pytest.mark.parametrize("Hq,Hk,D,n", [(8, 1, 128, 3), (4, 1, 128, 5), (14, 2, 128, 3), (8, 1, 128, 4), (8, 2, 128, 13),
                                       (8, 1, 64, 3), (10, 2, 64, 4), (8, 1, 64, 5), (8, 1, 256, 2), (3, 1, 256, 3),
                                       (6, 2, 256, 6)])
@pytest.mark.parametrize("lens", [[60, 400, 17], [700, 90, 2000]])
def test_columns_of_every_width(Hq, Hk, D, n, lens):
    """9 to 52 (query token, head) columns of a kv head: one to several tiles and blocks of them."""
    cu = [n * i for i in range(len(lens) + 1)]
    cache, table, g = filled(lens, Hk, 32, D, seed=D + n)
    check(torch.randn(cu[-1], Hq, D, generator=g).to(BF16), cache, table, lens, cu, max_q=n)


@pytest.mark.parametrize("max_q", [1, 4])
@pytest.mark.parametrize("Hq,Hk,D", [(8, 1, 128), (12, 4, 64), (16, 4, 128), (4, 1, 256)])
def test_several_tokens_of_long_and_short_sequences(Hq, Hk, D, max_q):
    """Long enough that items are split over CTAs, beside short and empty sequences."""
    lens, counts, ps = [700, 33, 4, 0, 1250, 16, 513], [4, 1, 9, 2, 3, 0, 5], 32
    cu = [1]
    for n in counts:
        cu.append(cu[-1] + n)
    cache, table, g = filled(lens, Hk, ps, D, seed=D + Hk)
    check(torch.randn(cu[-1] + 2, Hq, D, generator=g).to(BF16), cache, table, lens, cu, max_q)


@pytest.mark.parametrize("longest", [0, 1, 480, 512, 513, 544])
@pytest.mark.parametrize("width", [None, 64])
def test_around_the_length_from_which_items_are_split(longest, width):
    """No sequence above 512 tokens, in page tables that hold more or not (without cu_q and with)."""
    lens, ps = [longest, 40, 0, min(longest, 300)], 32
    cache, table, g = filled(lens, 2, ps, 128, seed=longest)
    table = table[:, :max(-(-n // ps) for n in lens)]
    if width:
        table = torch.cat([table, torch.full((4, width - table.shape[1]), -1, dtype=torch.int32)], 1)
    table = table.contiguous()
    check(torch.randn(4, 8, 128, generator=g).to(BF16), cache, table, lens)
    check(torch.randn(10, 8, 128, generator=g).to(BF16), cache, table, lens, [1, 4, 6, 7, 9], max_q=3)


@pytest.mark.parametrize("Hq,Hk,D,ps", [(8, 1, 128, 256), (32, 8, 128, 64), (4, 4, 64, 16), (2, 1, 256, 128)])
def test_long_and_ragged(Hq, Hk, D, ps):
    lens = [5000, 1, 777, 2048, 0, 16, 3001]
    cache, table, g = filled(lens, Hk, ps, D, seed=D)
    check(torch.randn(len(lens), Hq, D, generator=g).to(BF16), cache, table, lens)


def test_a_chunk_of_a_prompt():
    """Far more query tokens than max_q says, in many blocks of columns, beside single ones."""
    lens, cu = [333, 40, 200], [0, 200, 201, 250]
    for Hq, Hk, D in ((8, 2, 128), (6, 2, 64), (2, 1, 256)):
        cache, table, g = filled(lens, Hk, 16, D, seed=D)
        check(torch.randn(250, Hq, D, generator=g).to(BF16), cache, table, lens, cu, max_q=1)


def test_calls_on_two_streams():
    """Two calls at once, each with its own buffers: the bits of the calls alone."""
    lens = [4000, 300, 77]
    cache, table, g = filled(lens, 4, 32, 128, seed=21)
    c, t, n = cache.to(DEV), table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    q = [torch.randn(3, 16, 128, generator=g).to(BF16).to(DEV) for _ in range(2)]
    alone = [rmsn.kv4_attention(x, c, t, n) for x in q]
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(side[i]):
                outs[i].append(rmsn.kv4_attention(q[i], c, t, n))
    torch.cuda.synchronize()
    for i in range(2):
        for o in outs[i]:
            assert torch.equal(o[0], alone[i][0]) and torch.equal(o[1], alone[i][1])
    assert rmsn.rmsn_device_status() == 0


def test_graphs_that_share_a_workspace():
    """Two graphs captured over one workspace and replayed in turn: what one leaves does not reach the other."""
    long, short = filled([3000], 2, 16, 64, seed=22), filled([50, 0, 700], 2, 16, 64, seed=23)
    runs = []
    ws = torch.empty(rmsn.kv4_attention_workspace_bytes(3, 64), dtype=torch.uint8, device=DEV)
    for (cache, table, g), lens in ((long, [3000]), (short, [50, 0, 700])):
        a = (torch.randn(len(lens), 8, 64, generator=g).to(BF16).to(DEV), cache.to(DEV), table.to(DEV),
             torch.tensor(lens, dtype=torch.int32, device=DEV))
        eager = rmsn.kv4_attention(*a)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = rmsn.kv4_attention(*a, workspace=ws)
        runs.append((graph, out, eager, a))
    for _ in range(3):
        for graph, out, eager, _ in runs:
            graph.replay()
        torch.cuda.synchronize()
        for _, out, eager, _ in runs:
            assert torch.equal(out[0], eager[0]) and torch.equal(out[1], eager[1])


def test_many_sequences():
    """More sequences than the threads of a CTA (two tiles of the work split's prefix sums)."""
    lens = [(i * 37) % 40 for i in range(300)]
    cache, table, g = filled(lens, 2, 16, 64, seed=1)
    check(torch.randn(300, 4, 64, generator=g).to(BF16), cache, table, lens)


@pytest.mark.parametrize("Hq,Hk,D,longest,n", [(4, 4, 128, 100, 1), (8, 8, 64, 480, 1), (4, 4, 256, 300, 1),
                                               (16, 4, 128, 128, 3), (12, 4, 64, 300, 3)])
def test_more_short_items_than_ctas(Hq, Hk, D, longest, n):
    """Thousands of short items, some empty, in page tables of at most 512 tokens."""
    lens = [(i * 53) % (longest + 1) for i in range(420)]
    cache, table, g = filled(lens, Hk, 32, D, seed=D + n)
    table = table[:, :-(-longest // 32)].contiguous()
    cu = [n * i for i in range(len(lens) + 1)]
    check(torch.randn(cu[-1], Hq, D, generator=g).to(BF16), cache, table, lens, cu if n > 1 else None, max_q=n)


@pytest.mark.parametrize("std", [1e-3, 1.0, 40.0])
@pytest.mark.parametrize("scale", [None, 0.0, -0.3, 3.0])
def test_score_ranges(std, scale):
    """From flat to one-hot softmaxes, negative scale, large and tiny queries."""
    lens = [500, 200]
    cache, table, g = filled(lens, 2, 32, 128, seed=3)
    q = (torch.randn(2, 8, 128, generator=g) * std).to(BF16)
    q[0, 1] = 0
    check(q, cache, table, lens, scale=scale, rms=False)


def test_queries_near_the_ends_of_the_range():
    """Large queries over small keys and the other way round: the scores are ordinary, the
    factors between them (2^(exponent + 24)) are not.  The scale is a power of two, so every
    product is that of the ordinary case, and K's codes are the same."""
    for e in (118, 80, -70):
        cache, table, g = filled([300, 40], 2, 32, 128, seed=5, std=1.0)
        half = cache.view(BF16)
        for t in range(cache.shape[0] * cache.shape[2] * 16):
            rec = half[t // 32, :, t // 16 % 2]
            at = R.tables(128)[0][2][t % 16].flatten()
            rec[:, at] = rec[:, at] * 2.0 ** -e
        q = torch.randn(2, 8, 128, generator=g).to(BF16)
        check((q.float() * 2.0 ** e).to(BF16), cache, table, [300, 40])


def test_rising_scores():
    """Keys that grow along the sequence: the running maximum moves all the time."""
    lens = [640]
    cache, table, g = filled(lens, 1, 16, 128, seed=4)
    half = cache.view(BF16)
    _, _, sc = R.tables(128)[0]
    for t in range(640):
        rec = half[table[0, t // 16], 0, 0]
        rec[sc[t % 16].flatten()] = rec[sc[t % 16].flatten()] * (1 + t / 40)
    check(torch.randn(1, 8, 128, generator=g).to(BF16), cache, table, lens, rms=False)


def test_nan_reaches_only_who_sees_it():
    """NaN in K or V of a drafted token: earlier queries do not see it; behind the end anything may be."""
    Hk, D, n, L = 2, 128, 4, 53
    cache, table, g = filled([L], Hk, 16, D, seed=6)
    q = torch.randn(n, 4, D, generator=g).to(BF16)
    args = (q.to(DEV), table.to(DEV), torch.tensor([L], dtype=torch.int32, device=DEV))
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)

    def run(c):
        o, lse = rmsn.kv4_attention(args[0], c.to(DEV), *args[1:], cu_q=cu, max_q=n)
        return o.cpu().float(), lse.cpu()

    clean, lse0 = run(cache)
    assert torch.isfinite(clean).all()
    half = cache.view(BF16)

    def poke(which, tok, group, value=math.nan):
        c = cache.clone()
        sc = R.tables(D)[which][2]
        c.view(BF16)[table[0, tok // 16], 1, 0, sc[tok % 16, group]] = torch.tensor([value, value], dtype=BF16)
        return c

    # V of token 51 (seen by queries 2 and 3 of 4), kv head 1, group 2
    o, lse = run(poke(1, 51, 2))
    hit = torch.zeros_like(clean, dtype=torch.bool)
    hit[2:, 2:, 64:96] = True
    assert torch.isnan(o[hit]).all() and torch.equal(o[~hit], clean[~hit]) and torch.equal(lse, lse0)
    # V of an old token: every query of that kv head
    o, _ = run(poke(1, 3, 0, math.inf))
    hit[:] = False
    hit[:, 2:, 0:32] = True
    assert not torch.isfinite(o[hit]).any() and torch.equal(o[~hit], clean[~hit])
    # K of token 52: the last query only
    o, lse = run(poke(0, 52, 1))
    assert torch.isnan(o[3, 2:]).all() and torch.isnan(lse[3, 2:]).all()
    assert torch.equal(o[:3], clean[:3]) and torch.equal(o[3, :2], clean[3, :2]) and torch.equal(lse[:3], lse0[:3])
    # behind the end
    for tok in (53, 60, 63):
        for which in (0, 1):
            o, lse = run(poke(which, tok, 3))
            assert torch.equal(o, clean) and torch.equal(lse, lse0)
    # a query's own NaN or infinity stays in its row
    for bad in (math.nan, math.inf):
        q2 = q.clone()
        q2[1, 0, 7] = bad
        args = (q2.to(DEV), *args[1:])
        o, lse = run(cache)
        assert torch.isnan(o[1, 0]).all() and torch.isnan(lse[1, 0])
        o[1, 0], lse[1, 0] = clean[1, 0], lse0[1, 0]
        assert torch.equal(o, clean) and torch.equal(lse, lse0)
    assert rmsn.rmsn_device_status() == 0


def test_bad_pages_and_lengths():
    Hk, D, ps = 2, 64, 16
    lens = [100, 40, 16]
    cache, table, g = filled(lens, Hk, ps, D, seed=7)
    q = torch.randn(3, 4, D, generator=g).to(BF16)
    assert rmsn.rmsn_device_status() == 0
    table[0, 2], table[1, 0], table[2, 0] = cache.shape[0], -1, 2 ** 31 - 1  # tokens left out, one row empty
    check(q, cache, table, lens, status=ERR_INDEX)
    cache, table, g = filled(lens, Hk, ps, D, seed=8)
    table = table[:, :5].contiguous()  # 80 tokens: the first length is too long, one is negative
    check(q, cache, table, [100, -5, 16], status=ERR_INDEX)
    # lengths of cu_q outside the rows are cut, not followed
    cu = torch.tensor([0, 2, 9, -4], dtype=torch.int32, device=DEV)
    rmsn.kv4_attention(q.to(DEV), cache.to(DEV), table.to(DEV), torch.tensor([64, 40, 16], dtype=torch.int32, device=DEV),
                       cu_q=cu, max_q=2)
    rmsn.rmsn_device_status()


def test_strided_q_out_and_table():
    Hk, D, lens = 2, 128, [90, 33, 200]
    cache, table, g = filled(lens, Hk, 16, D, seed=9)
    q = torch.randn(3, 8, D, generator=g).to(BF16)
    plain = check(q, cache, table, lens)[0]
    wide = torch.zeros(3, 12, D + 8, dtype=BF16, device=DEV)
    wide[:, 2:10, :D] = q.to(DEV)
    big = torch.zeros(3, table.shape[1] + 5, dtype=torch.int32, device=DEV)
    big[:, :table.shape[1]] = table.to(DEV)
    out = torch.zeros(8, 3, D, dtype=BF16, device=DEV)
    rmsn.kv4_attention(wide[:, 2:10, :D], cache.to(DEV), big[:, :table.shape[1]],
                       torch.tensor(lens, dtype=torch.int32, device=DEV), out=out.transpose(0, 1))
    assert torch.equal(out.transpose(0, 1), plain)


def test_same_bits_and_dirty_workspace():
    lens = [3000, 10, 1234]
    cache, table, g = filled(lens, 8, 64, 128, seed=10)
    q = torch.randn(3, 32, 128, generator=g).to(BF16).to(DEV)
    a = (q, cache.to(DEV), table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV))
    o, lse = rmsn.kv4_attention(*a)
    ws = torch.empty(rmsn.kv4_attention_workspace_bytes(3, 128), dtype=torch.uint8, device=DEV)
    for fill in (0, 255, 0x7f):
        ws.fill_(fill)
        o2, l2 = rmsn.kv4_attention(*a, workspace=ws)
        assert torch.equal(o, o2) and torch.equal(lse, l2)
    with pytest.raises(rmsn.RmsnError) as e:
        rmsn.kv4_attention(*a, workspace=ws[:1024])
    assert e.value.status == 4


def test_refusals():
    cache, table, g = filled([20, 20], 2, 16, 64, seed=11)
    q = torch.randn(2, 4, 64).to(BF16).to(DEV)
    c, t, n = cache.to(DEV), table.to(DEV), torch.tensor([20, 20], dtype=torch.int32, device=DEV)
    f = rmsn.kv4_attention
    for bad in ((q.float(), c, t, n), (q[:1], c, t, n), (q[:, :3], c, t, n), (q, c.int(), t, n),
                (q, c[..., :1000], t, n), (q, c, t.long(), n), (q, c, t, n.long()), (q, c, t, n[:1]),
                (torch.zeros(2, 4, 128, dtype=BF16, device=DEV), c, t, n)):
        with pytest.raises((ValueError, TypeError)):
            f(*bad)
    with pytest.raises(ValueError):
        f(q, c, t, n, cu_q=n)
    with pytest.raises(ValueError):
        f(q, c.cpu(), t, n)
    with pytest.raises(rmsn.RmsnError):
        f(q, c, t, n, max_q=0)
    with pytest.raises(rmsn.RmsnError):
        f(q, c, t, n, scale=math.inf)


def test_serving_path_in_a_graph():
    """Prompts stored, then decoding steps of append and attention replayed from a graph whose buffers
    are refilled: every step against 64 bits over the cache that it left."""
    Hq, Hk, D, ps, B = 8, 2, 128, 16, 3
    prompt = [5, 30, 17]
    steps, width = 20, 4
    pages = B * width
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(0)).view(B, width).int()
    cache = empty_cache(pages, Hk, ps, D)
    cos, sin = (t.to(DEV) for t in angles(64, D))
    g = torch.Generator().manual_seed(1)
    w = [(1 + 0.1 * torch.randn(D, generator=g)).to(DEV) for _ in range(2)]

    def slots_of(b, t):
        return table[b].long()[t // ps] * ps + t % ps

    # prompts in one call
    pos = torch.cat([torch.arange(n) for n in prompt])
    slots = torch.cat([slots_of(b, torch.arange(n)) for b, n in enumerate(prompt)])
    x = torch.randn(sum(prompt), Hq + 2 * Hk, D, generator=g).to(BF16).to(DEV)
    q, k, v = x.split([Hq, Hk, Hk], 1)
    rmsn.qk_norm_rope_kv4_append(q, k, v, *w, cos, sin, pos.to(DEV), cache, slots.to(DEV), EPS)

    bx = torch.zeros(B + 1, Hq + 2 * Hk, D, dtype=BF16, device=DEV)  # one padding row
    bpos = torch.zeros(B + 1, dtype=torch.int64, device=DEV)
    bslots = torch.full((B + 1,), -1, dtype=torch.int64, device=DEV)
    lens = torch.tensor([*prompt, 0], dtype=torch.int32, device=DEV)
    tab = torch.cat([table, torch.zeros(1, width, dtype=torch.int32)]).to(DEV)

    def step():
        q, k, v = bx.split([Hq, Hk, Hk], 1)
        rmsn.qk_norm_rope_kv4_append(q, k, v, *w, cos, sin, bpos, cache, bslots, EPS, q_out=q)
        return rmsn.kv4_attention(q, cache, tab, lens)

    keep = cache.clone()
    step()
    torch.cuda.synchronize()
    assert torch.equal(cache, keep)  # all padding: nothing stored
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = step()
    for i in range(steps):
        at = torch.tensor([n + i for n in prompt])
        bx.copy_(torch.randn(bx.shape, generator=g).to(BF16))
        bpos[:B] = at.to(DEV)
        bslots[:B] = torch.stack([slots_of(b, at[b]) for b in range(B)]).to(DEV)
        lens[:B] = (at + 1).int().to(DEV)
        graph.replay()
        torch.cuda.synchronize()
        ro, rl, ob, lb, _ = R.attention(bx.cpu()[:B, :Hq], cache.cpu(), table, lens.cpu()[:B], None, D ** -0.5)
        R.assert_within(out[:B], ro, ob, BF16, f"step {i}")
        assert ((lse[:B].cpu().double() - rl).abs() <= lb + 2.0 ** -22 * rl.abs()).all()
        assert (out[B] == 0).all() and torch.isinf(lse[B]).all()
    assert rmsn.rmsn_device_status() == 0


@pytest.mark.parametrize("T,nb", [(5000, False), (9000, True)])
def test_long_append_streams(T, nb):
    """Enough tokens for the streaming kernel, padding and a bad slot among them: the bytes of the small one."""
    Hq, Hk, D, ps = 6, 2, 128, 16
    x, (wq, wk), (cos, sin), pos, g = append_inputs(T, Hq, Hk, D, D, seed=T)
    pages = -(-T // ps) + 1
    slots = torch.randperm(pages * ps, generator=g)[:T]
    slots[::97] = -1
    slots[1234] = pages * ps
    q, k, v = x.to(DEV).split([Hq, Hk, Hk], 1)
    rest = [t.to(DEV) for t in (wq, wk, cos, sin)]
    big, small = empty_cache(pages, Hk, ps, D), empty_cache(pages, Hk, ps, D)
    yq = torch.full((T, Hq, D), 7.0, dtype=BF16, device=DEV)
    rmsn.qk_norm_rope_kv4_append(q, k, v, *rest, pos.to(DEV), big, slots.to(DEV), EPS, interleaved=nb, q_out=yq)
    assert rmsn.rmsn_device_status() == ERR_INDEX
    zq = torch.full((T, Hq, D), 7.0, dtype=BF16, device=DEV)
    for a in range(0, T, 100):
        b = slice(a, a + 100)
        rmsn.qk_norm_rope_kv4_append(q[b], k[b], v[b], *rest, pos[b].to(DEV), small, slots[b].to(DEV), EPS,
                                     interleaved=nb, q_out=zq[b])
    assert rmsn.rmsn_device_status() == ERR_INDEX
    assert torch.equal(big, small) and torch.equal(yq, zq)
    assert (yq[0] == 7).all() and (yq[1234] == 7).all()


def test_cache_beyond_4_gib():
    """Records whose byte offsets pass 2^32."""
    Hk, D, ps = 1, 128, 16
    pages = (1 << 32) // (20 * D) + 40
    cache = torch.zeros(rmsn.kv4_cache_shape(pages, Hk, ps, D), dtype=torch.uint8, device=DEV)
    T = 40
    x, (wq, wk), (cos, sin), pos, g = append_inputs(T, 8, Hk, D, D, 12)
    table = torch.tensor([[pages - 1, pages - 20, 3]], dtype=torch.int32)
    t = torch.arange(T)
    slots = table[0].long()[t // ps] * ps + t % ps
    q, k, v = x.to(DEV).split([8, Hk, Hk], 1)
    rmsn.qk_norm_rope_kv4_append(q, k, v, *(a.to(DEV) for a in (wq, wk, cos, sin, pos)), cache, slots.to(DEV), EPS)
    o, _ = rmsn.kv4_attention(q[:1].contiguous(), cache, table.to(DEV), torch.tensor([T], dtype=torch.int32, device=DEV))
    small = cache[table[0].long()].cpu()
    ro, _, ob, _, _ = R.attention(x[:1, :8], small, torch.tensor([[0, 1, 2]]), [T], None, D ** -0.5)
    R.assert_within(o, ro, ob, BF16)
    assert rmsn.rmsn_device_status() == 0
