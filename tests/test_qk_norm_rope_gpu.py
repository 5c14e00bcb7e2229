"""qk_norm_rope_fwd and qk_norm_rope_bwd against the 64-bit formulas: types, head layouts, partial and
neighbouring rotations, strides, odd sizes, positions outside the table, in-place use, graphs, streams."""
import pytest
import torch

import _attn_ref as R
import rmsnorm_fwd_bwd_persistent_gb300 as rmsn

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-6
ERR_INDEX = 8


def gen(seed):
    return torch.Generator().manual_seed(seed)


def angles(P, rd):
    f = 10000.0 ** (-torch.arange(rd // 2, dtype=torch.float64) * 2 / rd)
    a = torch.arange(P, dtype=torch.float64)[:, None] * f
    return a.cos().float(), a.sin().float()


def make(B, T, Hq, Hk, D, rd, dtype, wd, layout, seed=0, P=None, std=1.0):
    """q, k, gq, gk (CPU, [B, T, H, D]; [T, H, D] where B is None), weights, tables, positions, and a
    function that lays a CPU tensor out on the device."""
    g = gen(seed)
    lead = (T,) if B is None else (B, T)
    q, k, gq, gk = ((torch.randn(*lead, H, D, generator=g) * std).to(dtype) for H in (Hq, Hk, Hq, Hk))
    wq, wk = ((1 + 0.1 * torch.randn(D, generator=g)).to(wd) for _ in range(2))
    P = P or T + 7
    cos, sin = angles(P, rd)
    pos = torch.randint(0, P, lead, generator=g)
    return q, k, gq, gk, wq, wk, cos, sin, pos


def place(q, k, layout):
    """q and k on the device in a memory layout."""
    if layout == "packed":
        x = torch.cat([q, k, torch.zeros_like(k)], -2).to(DEV)
        return x[..., :q.shape[-2], :], x[..., q.shape[-2]:q.shape[-2] + k.shape[-2], :]
    if layout == "bhsd":
        return tuple(t.transpose(-2, -3).contiguous().to(DEV).transpose(-2, -3) for t in (q, k))
    if layout == "padded":  # rows and heads with gaps
        out = []
        for t in (q, k):
            buf = torch.full((*t.shape[:-1], t.shape[-1] + 8), 3.0, dtype=t.dtype, device=DEV)
            buf[..., :t.shape[-1]] = t.to(DEV)
            out.append(buf[..., :t.shape[-1]])
        return tuple(out)
    return q.to(DEV), k.to(DEV)


CASES = [
    # B, T, Hq, Hk, D, rd, x, w, layout, neighbours
    (None, 1, 1, 1, 64, 64, BF16, F32, "dense", False),
    (None, 1, 32, 8, 128, 128, BF16, BF16, "packed", False),
    (None, 67, 32, 8, 128, 128, BF16, F32, "packed", False),
    (None, 67, 32, 8, 128, 128, BF16, F32, "dense", True),
    (None, 33, 5, 3, 128, 64, BF16, F32, "packed", False),
    (None, 33, 5, 3, 128, 32, F32, F32, "packed", True),
    (None, 40, 4, 1, 64, 64, F32, F32, "dense", False),
    (None, 129, 9, 1, 64, 16, BF16, BF16, "bhsd", False),
    (3, 21, 16, 4, 96, 48, BF16, F32, "bhsd", True),
    (3, 21, 16, 4, 96, 96, BF16, F32, "bhsd", False),
    (2, 1, 7, 7, 80, 80, F32, BF16, "packed", True),
    (2, 50, 3, 2, 80, 32, BF16, F32, "padded", False),
    (2, 19, 2, 1, 256, 256, BF16, BF16, "dense", False),
    (1, 19, 2, 1, 256, 128, F32, F32, "packed", True),
    (None, 23, 3, 2, 192, 192, BF16, F32, "dense", False),
    (None, 45, 6, 2, 16, 16, BF16, F32, "dense", False),
    (None, 45, 6, 2, 16, 16, F32, F32, "padded", True),
    (None, 31, 11, 2, 32, 16, BF16, F32, "packed", True),
    (None, 31, 40, 33, 48, 48, F32, F32, "dense", False),
    (None, 1200, 12, 2, 112, 96, BF16, BF16, "packed", False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v).replace("torch.", "") for v in c))
def test_forward(case):
    B, T, Hq, Hk, D, rd, dt, wd, layout, nb = case
    q, k, _, _, wq, wk, cos, sin, pos = make(*case[:9], seed=1)
    dq, dk = place(q, k, layout)
    yq, yk = rmsn.qk_norm_rope_fwd(dq, dk, *(t.to(DEV) for t in (wq, wk, cos, sin, pos)), EPS, interleaved=nb)
    assert yq.is_contiguous() and yq.dtype == dt
    for y, x, w, n in ((yq, q, wq, "q"), (yk, k, wk, "k")):
        R.assert_within(y, *R.fwd(x, w, cos, sin, pos, EPS, nb), dt, n)
    # in place, through the same views
    zq, zk = rmsn.qk_norm_rope_fwd(dq, dk, *(t.to(DEV) for t in (wq, wk, cos, sin, pos)), EPS, interleaved=nb,
                                   q_out=dq, k_out=dk)
    assert zq is dq and torch.equal(zq, yq) and torch.equal(zk, yk)
    assert rmsn.rmsn_device_status() == 0


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v).replace("torch.", "") for v in c))
def test_backward(case):
    B, T, Hq, Hk, D, rd, dt, wd, layout, nb = case
    q, k, gq, gk, wq, wk, cos, sin, pos = make(*case[:9], seed=2)
    x, g = place(q, k, layout), place(gq, gk, "padded" if layout == "packed" else layout)
    rest = [t.to(DEV) for t in (wq, wk, cos, sin, pos)]
    dq, dk, dwq, dwk = rmsn.qk_norm_rope_bwd(*g, *x, *rest, EPS, interleaved=nb)
    for d, dw, y, v, w, n in ((dq, dwq, gq, q, wq, "q"), (dk, dwk, gk, k, wk, "k")):
        (dx, bx), (dwr, bw) = R.bwd(y, v, w, cos, sin, pos, EPS, nb)
        R.assert_within(d, dx, bx, dt, "d" + n)
        R.assert_within(dw, dwr, bw, F32, "dw" + n)
    # the same bits again, in place over the gradients, with a caller's workspace
    ws = torch.full((rmsn.qk_norm_rope_bwd_workspace_bytes(D),), 255, dtype=torch.uint8, device=DEV)
    again = rmsn.qk_norm_rope_bwd(*g, *x, *rest, EPS, interleaved=nb, workspace=ws, dq=g[0], dk=g[1])
    for a, b in zip(again, (dq, dk, dwq, dwk)):
        assert torch.equal(a, b)
    assert rmsn.rmsn_device_status() == 0


@pytest.mark.parametrize("nb", [False, True])
def test_gradients_against_differences(nb):
    """Central differences of sum(gy y) in 64 bits over the formula's forward, in every input of a row,
    against the kernel's fp32 gradients: step 1e-5, so the differences are off by about 1e-10 x the third
    derivative (below 1e-6 here), the kernel by its bound."""
    q, k, gq, gk, wq, wk, cos, sin, pos = make(None, 3, 2, 1, 32, 32, F32, F32, "dense", seed=3)
    out = rmsn.qk_norm_rope_bwd(*(t.to(DEV) for t in (gq, gk, q, k, wq, wk, cos, sin, pos)), EPS, interleaved=nb)
    out = [t.cpu().double() for t in out]

    def loss(q, k, wq, wk):
        return sum((R.fwd(x, w, cos, sin, pos, EPS, nb)[0] * g.double()).sum() for x, w, g in ((q, wq, gq), (k, wk, gk)))

    args = [t.double() for t in (q, k, wq, wk)]
    for i, name in enumerate(("dq", "dk", "dwq", "dwk")):
        flat = args[i].reshape(-1)
        for e in range(0, flat.numel(), 7):
            v = flat[e].item()
            flat[e] = v + 1e-5
            up = loss(*args)
            flat[e] = v - 1e-5
            down = loss(*args)
            flat[e] = v
            d = float((up - down) / 2e-5)
            assert abs(float(out[i].reshape(-1)[e]) - d) <= 2e-5 * (1 + abs(d)), (name, e)


def test_zero_and_extreme_rows():
    q, k, gq, gk, wq, wk, cos, sin, pos = make(None, 12, 4, 2, 128, 128, F32, F32, "dense", seed=4)
    q[0], k[1] = 0, 0
    q[2] *= 1e15
    q[3] *= 1e-12  # mean square far below eps
    rest = [t.to(DEV) for t in (wq, wk, cos, sin, pos)]
    yq, yk = rmsn.qk_norm_rope_fwd(q.to(DEV), k.to(DEV), *rest, EPS)
    R.assert_within(yq, *R.fwd(q, wq, cos, sin, pos, EPS, False), F32)
    R.assert_within(yk, *R.fwd(k, wk, cos, sin, pos, EPS, False), F32)
    out = rmsn.qk_norm_rope_bwd(gq.to(DEV), gk.to(DEV), q.to(DEV), k.to(DEV), *rest, EPS)
    (dx, bx), (dw, bw) = R.bwd(gq, q, wq, cos, sin, pos, EPS, False)
    R.assert_within(out[0], dx, bx, F32)
    R.assert_within(out[2], dw, bw, F32)
    assert (yq[0] == 0).all()


def test_rounding_of_the_reciprocal_root():
    """One nonzero element per head, no rotation (cos = 1, sin = 0), w = 1: y = x (1 / sqrt(x^2 / 16 + eps)) with
    every operation rounded once, so torch's IEEE square root and division on the CPU give the same bits."""
    T, D = 20000, 16
    g = gen(11)
    v = torch.randn(T, 1, generator=g) * 10.0 ** torch.empty(T, 1).uniform_(-6, 6, generator=g)
    x = torch.zeros(T, 1, D)
    x[..., 3] = v
    one, zero = torch.ones(1, 8, device=DEV), torch.zeros(1, 8, device=DEV)
    for eps in (1e-6, 1e-5, 0.0):
        y, _ = rmsn.qk_norm_rope_fwd(x.to(DEV), x.to(DEV), torch.ones(D, device=DEV), torch.ones(D, device=DEV), one,
                                     zero, torch.zeros(T, dtype=torch.int64, device=DEV), eps)
        m = v * v * (1.0 / D) + torch.tensor(eps, dtype=F32)
        ref = v * (1.0 / m.sqrt())
        normal = m > 1e-30
        assert torch.equal(y.cpu()[..., 3][normal], ref[normal])


def test_long_sum_of_weight_gradients():
    """Many rows into the 64 columns of dw: the bound does not grow with their number."""
    q, k, gq, gk, wq, wk, cos, sin, pos = make(None, 6000, 24, 3, 64, 64, BF16, F32, "dense", seed=5)
    out = rmsn.qk_norm_rope_bwd(*(t.to(DEV) for t in (gq, gk, q, k, wq, wk, cos, sin, pos)), EPS)
    for dw, g, x, w in ((out[2], gq, q, wq), (out[3], gk, k, wk)):
        _, (ref, bound) = R.bwd(g, x, w, cos, sin, pos, EPS, False)
        R.assert_within(dw, ref, bound, F32)
        # what the bound is made of is the terms' rounding; the sum itself adds less than one step
        assert float((dw.cpu().double() - ref).norm() / ref.norm()) < 2e-6


@pytest.mark.parametrize("bad", [-1, 50, 1 << 40, -(1 << 62)])
def test_positions_outside_the_table(bad):
    q, k, gq, gk, wq, wk, cos, sin, pos = make(None, 40, 6, 2, 64, 64, BF16, F32, "dense", seed=6, P=50)
    ok = torch.ones(40, dtype=torch.bool)
    for t in (0, 17, 39):
        pos[t], ok[t] = bad, False
    rest = [t.to(DEV) for t in (wq, wk, cos, sin, pos)]
    yq, yk = torch.full_like(q, 7.0).to(DEV), torch.full_like(k, 7.0).to(DEV)
    assert rmsn.rmsn_device_status() == 0
    rmsn.qk_norm_rope_fwd(q.to(DEV), k.to(DEV), *rest, EPS, q_out=yq, k_out=yk)
    assert rmsn.rmsn_device_status() == ERR_INDEX
    safe = torch.where(ok, pos, 0)
    for y, x, w in ((yq, q, wq), (yk, k, wk)):
        assert (y[~ok] == 7).all()
        ref, bound = R.fwd(x, w, cos, sin, safe, EPS, False)
        R.assert_within(y[ok], ref[ok], bound[ok], BF16)
    dq, dk = torch.full_like(q, 7.0).to(DEV), torch.full_like(k, 7.0).to(DEV)
    out = rmsn.qk_norm_rope_bwd(gq.to(DEV), gk.to(DEV), q.to(DEV), k.to(DEV), *rest, EPS, dq=dq, dk=dk)
    assert rmsn.rmsn_device_status() == ERR_INDEX
    for d, dw, g, x, w in ((dq, out[2], gq, q, wq), (dk, out[3], gk, k, wk)):
        assert (d[~ok] == 7).all()
        (dx, bx), (dwr, bw) = R.bwd(g[ok], x[ok], w, cos, sin, safe[ok], EPS, False)
        R.assert_within(d[ok], dx, bx, BF16)
        R.assert_within(dw, dwr, bw, F32)
    assert rmsn.rmsn_device_status() == 0


def test_positions_broadcast_and_strided():
    q, k, _, _, wq, wk, cos, sin, _ = make(3, 10, 4, 2, 64, 64, BF16, F32, "dense", seed=7, P=40)
    pos = torch.arange(20, device=DEV)[::2]  # [S], for all batches, stride 2
    rest = [t.to(DEV) for t in (wq, wk, cos, sin)]
    y, _ = rmsn.qk_norm_rope_fwd(q.to(DEV), k.to(DEV), *rest, pos, EPS)
    z, _ = rmsn.qk_norm_rope_fwd(q.to(DEV), k.to(DEV), *rest, pos.expand(3, 10), EPS)
    ref, bound = R.fwd(q, wq, cos, sin, pos.cpu().expand(3, 10), EPS, False)
    R.assert_within(y, ref, bound, BF16)
    assert torch.equal(y, z)


def test_no_tokens():
    q, k, gq, gk, wq, wk, cos, sin, pos = (t.to(DEV) for t in make(None, 0, 4, 2, 64, 64, BF16, F32, "dense"))
    y, _ = rmsn.qk_norm_rope_fwd(q, k, wq, wk, cos, sin, pos)
    assert y.shape == (0, 4, 64)
    dwq, dwk = torch.ones(64, device=DEV), torch.ones(64, device=DEV)
    rmsn.qk_norm_rope_bwd(gq, gk, q, k, wq, wk, cos, sin, pos, dwq=dwq, dwk=dwk)
    assert not dwq.any() and not dwk.any()


def test_refusals_with_device_tensors():
    q, k, gq, gk, wq, wk, cos, sin, pos = (t.to(DEV) for t in make(None, 4, 4, 2, 64, 64, BF16, F32, "dense"))
    f = rmsn.qk_norm_rope_fwd
    with pytest.raises(TypeError):
        f(q, k.float(), wq, wk, cos, sin, pos)
    with pytest.raises(TypeError):
        f(q.half(), k.half(), wq, wk, cos, sin, pos)
    with pytest.raises(TypeError):
        f(q, k, wq, wk.bfloat16(), cos, sin, pos)
    with pytest.raises(TypeError):
        f(q, k, wq, wk, cos.double(), sin.double(), pos)
    with pytest.raises(TypeError):
        f(q, k, wq, wk, cos, sin, pos.int())
    with pytest.raises(ValueError):
        f(q, k[:3], wq, wk, cos, sin, pos)
    with pytest.raises(ValueError):
        f(q, k, wq, wk, cos, sin, pos[:3])
    with pytest.raises(ValueError):
        f(q, k, wq[:32], wk, cos, sin, pos)
    with pytest.raises(ValueError):
        f(q.transpose(1, 2), k.transpose(1, 2), wq, wk, cos, sin, pos)
    with pytest.raises(ValueError):
        f(q, k, wq.cpu(), wk, cos, sin, pos)
    with pytest.raises(rmsn.RmsnError) as e:
        f(q, k, wq, wk, cos, sin, pos, q_out=q[:1].expand(4, 4, 64))  # an output on top of itself
    assert e.value.status == 1
    with pytest.raises(rmsn.RmsnError) as e:
        buf = torch.zeros(4 * 4 * 64 + 1, dtype=BF16, device=DEV)
        f(buf[1:].view(4, 4, 64), k, wq, wk, cos, sin, pos)
    assert e.value.status == 3
    with pytest.raises(rmsn.RmsnError) as e:
        rmsn.qk_norm_rope_bwd(gq, gk, q, k, wq, wk, cos, sin, pos, workspace=torch.zeros(64, device=DEV))
    assert e.value.status == 4


def test_expanded_inputs():
    """Inputs may share memory: one k head read as four."""
    q, k, _, _, wq, wk, cos, sin, pos = make(None, 9, 4, 1, 64, 64, BF16, F32, "dense", seed=8)
    y = rmsn.qk_norm_rope_fwd(q.to(DEV), k.to(DEV).expand(9, 4, 64), *(t.to(DEV) for t in (wq, wk, cos, sin, pos)))[1]
    ref, bound = R.fwd(k.expand(9, 4, 64), wk, cos, sin, pos, EPS, False)
    R.assert_within(y, ref, bound, BF16)


def test_graph_replay_and_other_stream():
    """Captured forward and backward on a side stream, two graphs over one set of leaves, fresh inputs
    between replays: the bits of eager calls."""
    q, k, gq, gk, wq, wk, cos, sin, pos = (t.to(DEV) for t in make(None, 300, 8, 2, 128, 128, BF16, F32, "dense", seed=9))

    def run():
        y = rmsn.qk_norm_rope_fwd(q, k, wq, wk, cos, sin, pos, EPS)
        return [*y, *rmsn.qk_norm_rope_bwd(gq, gk, q, k, wq, wk, cos, sin, pos, EPS)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
        graphs = []
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                outs = run()
            graphs.append((g, outs))
    torch.cuda.current_stream().wait_stream(side)
    for rep in range(3):
        gen_ = torch.Generator(device=DEV).manual_seed(rep)
        for t in (q, k, gq, gk):
            t.copy_(torch.randn(t.shape, generator=gen_, device=DEV))
        eager = run()
        for g, outs in graphs:
            g.replay()
            torch.cuda.synchronize()
            for a, b in zip(eager, outs):
                assert torch.equal(a, b)
    assert rmsn.rmsn_device_status() == 0


def test_beyond_32_bit_offsets():
    """A token stride that takes the last rows past 2^31 elements (4 GiB in bf16)."""
    T, step = 5, 1 << 29
    buf = torch.empty((T - 1) * step + 6 * 64 + 64, dtype=BF16, device=DEV)
    x = buf.as_strided((T, 6, 64), (step, 64, 1))
    q, k, _, _, wq, wk, cos, sin, pos = make(None, T, 4, 2, 64, 64, BF16, F32, "dense", seed=10)
    x.copy_(torch.cat([q, k], 1).to(DEV))
    yq, yk = rmsn.qk_norm_rope_fwd(x[:, :4], x[:, 4:], *(t.to(DEV) for t in (wq, wk, cos, sin, pos)), EPS,
                                   q_out=x[:, :4], k_out=x[:, 4:])
    R.assert_within(yq, *R.fwd(q, wq, cos, sin, pos, EPS, False), BF16)
    R.assert_within(yk, *R.fwd(k, wk, cos, sin, pos, EPS, False), BF16)
