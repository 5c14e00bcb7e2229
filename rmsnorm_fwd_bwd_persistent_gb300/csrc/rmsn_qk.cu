// rmsn_qk.cu -- RMS norm of every query and key head with the position rotation in the same
// pass: forward, and the backward with the weights' gradients.
//
// Forward, per row (one head of one token, D elements):
//   r = 1/sqrt(mean(x^2) + eps),  n = (x r) w,  y = R n      (FP32, one rounding to x's type)
// with R the rotation of the pairs below rd by the token's angles.  Backward, with h = R^T gy:
//   g = h w,  dx = r (g - x r^2 mean(g x)),  dw = sum over tokens and heads of h x r
// The backward takes r from x again: sum(x^2) joins the reduction of sum(g x) that it needs
// anyway, which is cheaper than an [tokens, heads] array written and read back.
//
// Both are bound by HBM: every row is read and written once, and the arithmetic is far below
// the issue limit.  A token's angles and the weights stay in registers while a warp goes over
// the token's heads.
#include <type_traits>

#include "rmsn_internal.h"
#include "rmsn_pipe.cuh"
#include "rmsn_qk.cuh"

namespace rmsn {

namespace {

constexpr int kWarps = 4;  // warps per CTA (they are independent)

struct FwdArgs {
    Heads x[2], y[2];
    const void* w[2];
    Span span[2];
    Rope rope;
    unsigned* err;
    int tokens, T, D, w_bf16;
    float eps;
};

// One unit of work per warp: tpw tokens and the chunks [part * per_part, ...) of their heads.
// blockIdx.y picks q or k and the part, blockIdx.x and the warp the tokens.
template <typename T, int LPR, bool NB>
__global__ void __launch_bounds__(kWarps * 32) qk_fwd_kernel(const FwdArgs a) {
    constexpr int RPW = 32 / LPR;
    constexpr int U = sizeof(T) == 2 ? 4 : 2;  // chunks in flight: 4 KiB of rows per warp
    const int side = blockIdx.y < a.span[0].parts ? 0 : 1;
    const Span sp = a.span[side];
    const int part = blockIdx.y - (side ? a.span[0].parts : 0);
    const int lane = threadIdx.x & 31, l = lane % LPR, rr = lane / LPR;
    const int hsub = rr & ((1 << sp.log_hpw) - 1), tsub = rr >> sp.log_hpw;
    const int tpw = RPW >> sp.log_hpw;
    const int64_t first = ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * tpw;
    if (first >= a.tokens) return;
    const Token tk = find_token((int)min(first + tsub, (int64_t)a.tokens), a.tokens, a.T, a.rope, a.err,
                                side == 0 && part == 0 && l == 0 && hsub == 0);
    const bool lane_ok = tk.ok && 16 * l < a.D;

    RowLane<NB> rl;
    rl.init(l, a.rope.rd);
    const T* x = a.x[side].row<T>(tk.b, tk.t);
    T* y = a.y[side].row<T>(tk.b, tk.t);
    const int64_t sxh = a.x[side].sh, syh = a.y[side].sh;
    const int c1 = min(sp.chunks, (part + 1) * sp.per_part);

    Angles ang;
    float w0[8], w1[8];
    bool have = false;
    for (int c = part * sp.per_part; c < c1; c += U) {
        Raw8<T> r0[U], r1[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int h = ((c + i) << sp.log_hpw) + hsub;
            r0[i].clear();
            r1[i].clear();
            if (lane_ok && c + i < c1 && h < sp.heads) {
                r0[i].load(x + h * sxh + rl.off0);
                r1[i].load(x + h * sxh + rl.off1);
            }
        }
        if (!have) {  // after the first rows are on their way
            have = true;
            ang.identity();
            if (lane_ok) {
                if (rl.turns) {
                    const int64_t at = tk.pos * (a.rope.rd / 2) + 8 * l;
                    ang.load(a.rope.cos + at, a.rope.sin + at);
                }
                load_w8(a.w[side], a.w_bf16, rl.off0, w0);
                load_w8(a.w[side], a.w_bf16, rl.off1, w1);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) w0[i] = w1[i] = 0.f;
            }
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int h = ((c + i) << sp.log_hpw) + hsub;
            if (c + i >= c1) break;  // the same for the whole warp
            float u[8], v[8];
            r0[i].get(u);
            r1[i].get(v);
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(u[e], u[e], ss);
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(v[e], v[e], ss);
            const float r = row_rstd(row_sum<LPR>(ss), (float)a.D, a.eps);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                u[e] = u[e] * r * w0[e];
                v[e] = v[e] * r * w1[e];
            }
            rotate<NB, false>(u, v, ang);
            r0[i].set(u);
            r1[i].set(v);
            if (lane_ok && h < sp.heads) {
                r0[i].store(y + h * syh + rl.off0);
                r1[i].store(y + h * syh + rl.off1);
            }
        }
    }
}

struct BwdArgs {
    Heads x[2], g[2], dx[2];
    const void* w[2];
    Span span[2];
    int grid[2];  // CTAs of q and of k
    Rope rope;
    float* ws;    // [CTA][hi, lo][D]
    unsigned* err;
    int tokens, T, D, w_bf16;
    float eps;
};

// Persistent: the first grid[0] CTAs take q's units, the others k's; a unit is tpw tokens and
// one part of their heads.  Every lane keeps the (high, low) TwoSum pair of its 16 columns of
// dw over all its rows; the pairs of the CTA's lanes are merged in a fixed order and written
// to the workspace, whose CTA partials qk_dw_reduce_kernel adds in a fixed order.
template <typename T, int LPR, bool NB>
__global__ void __launch_bounds__(kWarps * 32) qk_bwd_kernel(const BwdArgs a) {
    constexpr int RPW = 32 / LPR;
    const int side = (int)blockIdx.x < a.grid[0] ? 0 : 1;
    const int cta = blockIdx.x - (side ? a.grid[0] : 0);
    const Span sp = a.span[side];
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31, l = lane % LPR, rr = lane / LPR;
    const int hsub = rr & ((1 << sp.log_hpw) - 1), tsub = rr >> sp.log_hpw;
    const int tpw = RPW >> sp.log_hpw;
    const int64_t groups = ((int64_t)a.tokens + tpw - 1) / tpw;
    const int64_t units = groups * sp.parts;
    const bool dims_ok = 16 * l < a.D;

    RowLane<NB> rl;
    rl.init(l, a.rope.rd);
    float w0[8], w1[8];
    f2 hi[8], lo[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        w0[i] = w1[i] = 0.f;
        hi[i] = lo[i] = 0ull;
    }
    if (dims_ok) {
        load_w8(a.w[side], a.w_bf16, rl.off0, w0);
        load_w8(a.w[side], a.w_bf16, rl.off1, w1);
    }
    const int64_t sxh = a.x[side].sh, sgh = a.g[side].sh, sdh = a.dx[side].sh;
    const float inv_d = __frcp_rn((float)a.D);

    for (int64_t unit = (int64_t)cta * kWarps + warp; unit < units;
         unit += (int64_t)a.grid[side] * kWarps) {
        const int64_t grp = sp.parts == 1 ? unit : unit / sp.parts;
        const int part = (int)(unit - grp * sp.parts);
        const Token tk = find_token((int)min(grp * tpw + tsub, (int64_t)a.tokens), a.tokens, a.T,
                                    a.rope, a.err, side == 0 && part == 0 && l == 0 && hsub == 0);
        const bool ok = tk.ok && dims_ok;
        const T* x = a.x[side].row<T>(tk.b, tk.t);
        const T* g = a.g[side].row<T>(tk.b, tk.t);
        T* dx = a.dx[side].row<T>(tk.b, tk.t);
        const int c0 = part * sp.per_part, c1 = min(sp.chunks, c0 + sp.per_part);

        auto fetch = [&](int c, Raw8<T>& x0, Raw8<T>& x1, Raw8<T>& g0, Raw8<T>& g1) {
            const int h = (c << sp.log_hpw) + hsub;
            if (ok && h < sp.heads) {
                x0.load(x + h * sxh + rl.off0);
                x1.load(x + h * sxh + rl.off1);
                g0.load(g + h * sgh + rl.off0);
                g1.load(g + h * sgh + rl.off1);
            } else {
                x0.clear();
                x1.clear();
                g0.clear();
                g1.clear();
            }
        };
        Raw8<T> x0, x1, g0, g1;
        fetch(c0, x0, x1, g0, g1);
        Angles ang;
        ang.identity();
        if (ok && rl.turns) {
            const int64_t at = tk.pos * (a.rope.rd / 2) + 8 * l;
            ang.load(a.rope.cos + at, a.rope.sin + at);
        }
        for (int c = c0; c < c1; ++c) {
            Raw8<T> nx0, nx1, ng0, ng1;
            if (c + 1 < c1) fetch(c + 1, nx0, nx1, ng0, ng1);
            const int h = (c << sp.log_hpw) + hsub;
            float xu[8], xv[8], hu[8], hv[8];
            x0.get(xu);
            x1.get(xv);
            g0.get(hu);
            g1.get(hv);
            rotate<NB, true>(hu, hv, ang);
            float ss = 0.f, dot = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                ss = fmaf(xu[e], xu[e], ss);
                dot = fmaf(hu[e] * w0[e], xu[e], dot);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                ss = fmaf(xv[e], xv[e], ss);
                dot = fmaf(hv[e] * w1[e], xv[e], dot);
            }
            ss = row_sum<LPR>(ss);
            dot = row_sum<LPR>(dot);
            const float r = row_rstd(ss, (float)a.D, a.eps);
            const float k = r * (r * (dot * inv_d));  // r^2 mean(g x)
            const bool store = ok && h < sp.heads;
            if (store) {
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    comp_add2(hi[e / 2], lo[e / 2],
                              f2_make(hu[e] * (xu[e] * r), hu[e + 1] * (xu[e + 1] * r)));
                    comp_add2(hi[4 + e / 2], lo[4 + e / 2],
                              f2_make(hv[e] * (xv[e] * r), hv[e + 1] * (xv[e + 1] * r)));
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    xu[e] = r * fmaf(-xu[e], k, hu[e] * w0[e]);
                    xv[e] = r * fmaf(-xv[e], k, hv[e] * w1[e]);
                }
                x0.set(xu);
                x1.set(xv);
                x0.store(dx + h * sdh + rl.off0);
                x1.store(dx + h * sdh + rl.off1);
            }
            x0 = nx0;
            x1 = nx1;
            g0 = ng0;
            g1 = ng1;
        }
    }

    // merge the warp's rows (lanes of equal l), then the warps in order
    __shared__ float sm[kWarps][2][256];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float h0 = f2_lo(hi[i]), h1 = f2_hi(hi[i]), e0 = f2_lo(lo[i]), e1 = f2_hi(lo[i]);
#pragma unroll
        for (int o = LPR; o < 32; o <<= 1) {
            comp_merge(h0, e0, __shfl_xor_sync(0xffffffffu, h0, o),
                       __shfl_xor_sync(0xffffffffu, e0, o));
            comp_merge(h1, e1, __shfl_xor_sync(0xffffffffu, h1, o),
                       __shfl_xor_sync(0xffffffffu, e1, o));
        }
        if (rr == 0 && dims_ok) {
            const int col = (i < 4 ? rl.off0 : rl.off1 - 8) + 2 * i;
            sm[warp][0][col] = h0;
            sm[warp][0][col + 1] = h1;
            sm[warp][1][col] = e0;
            sm[warp][1][col + 1] = e1;
        }
    }
    __syncthreads();
    for (int col = threadIdx.x; col < a.D; col += kWarps * 32) {
        float h = sm[0][0][col], e = sm[0][1][col];
#pragma unroll
        for (int i = 1; i < kWarps; ++i) comp_merge(h, e, sm[i][0][col], sm[i][1][col]);
        float* out = a.ws + (int64_t)blockIdx.x * 2 * a.D + col;
        out[0] = h;
        out[a.D] = e;
    }
}

// dwq and dwk from the CTA partials: one CTA per 32 columns of one of them; warp s of 8 adds
// the partials s, s + 8, ... in order, the eight sums are merged in order, and high + low is
// rounded once.
__global__ void __launch_bounds__(256) qk_dw_reduce_kernel(const float* __restrict__ ws,
                                                           float* dwq, float* dwk, int D, int gq,
                                                           int gk) {
    __shared__ float sh[8][32], sl[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;
    const int n = blockIdx.y ? gk : gq;
    const float* p = ws + (blockIdx.y ? (int64_t)gq * 2 * D : 0);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float h = 0.f, e = 0.f;
    if (col < D) {
        for (int i = warp; i < n; i += 64) {
            float vh[8], vl[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int k = i + 8 * u;
                vh[u] = k < n ? __ldcg(p + (int64_t)k * 2 * D + col) : 0.f;
                vl[u] = k < n ? __ldcg(p + (int64_t)k * 2 * D + D + col) : 0.f;
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) comp_merge(h, e, vh[u], vl[u]);
        }
    }
    sh[warp][lane] = h;
    sl[warp][lane] = e;
    __syncthreads();
    if (warp == 0 && col < D) {
#pragma unroll
        for (int i = 1; i < 8; ++i) comp_merge(h, e, sh[i][lane], sl[i][lane]);
        (blockIdx.y ? dwk : dwq)[col] = __fadd_rn(h, e);
    }
}

template <typename T, int LPR, bool NB>
cudaError_t run_fwd(const QkCall& c, cudaStream_t s) {
    constexpr int RPW = 32 / LPR;
    FwdArgs a{};
    const int heads[2] = {c.heads[0], c.heads[1]};
    const int per = pick_per_part(heads, 2, c.tokens, RPW, c.sms);
    int64_t gx = 1;
    for (int i = 0; i < 2; ++i) {
        a.x[i] = c.x[i];
        a.y[i] = c.y[i];
        a.w[i] = c.w[i];
        a.span[i] = make_span(heads[i], RPW, per);
        const int64_t g = (groups_of(c.tokens, a.span[i], RPW) + kWarps - 1) / kWarps;
        gx = g > gx ? g : gx;
    }
    a.rope = c.rope;
    a.err = c.err;
    a.tokens = (int)c.tokens;
    a.T = (int)c.T;
    a.D = c.D;
    a.w_bf16 = c.w_dt;
    a.eps = c.eps;
    qk_fwd_kernel<T, LPR, NB>
        <<<dim3((unsigned)gx, a.span[0].parts + a.span[1].parts), kWarps * 32, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T, int LPR, bool NB>
cudaError_t run_bwd(const QkCall& c, cudaStream_t s) {
    constexpr int RPW = 32 / LPR;
    BwdArgs a{};
    const int heads[2] = {c.heads[0], c.heads[1]};
    const int per = pick_per_part(heads, 2, c.tokens, RPW, c.sms);
    int64_t units[2], rows[2];
    for (int i = 0; i < 2; ++i) {
        a.x[i] = c.x[i];
        a.g[i] = c.g[i];
        a.dx[i] = c.y[i];
        a.w[i] = c.w[i];
        a.span[i] = make_span(heads[i], RPW, per);
        units[i] = groups_of(c.tokens, a.span[i], RPW) * a.span[i].parts;
        rows[i] = (int64_t)heads[i];
    }
    // the CTAs of both sides together are kQkBwdCtasPerSm per SM at most, shared out by rows
    const int64_t all = (int64_t)c.sms * kQkBwdCtasPerSm;
    int64_t gk = all * rows[1] / (rows[0] + rows[1]);
    gk = gk < 1 ? 1 : gk;
    int64_t g[2] = {all - gk, gk};
    for (int i = 0; i < 2; ++i) {
        const int64_t need = (units[i] + kWarps - 1) / kWarps;
        a.grid[i] = (int)(need < g[i] ? need : g[i]);
    }
    a.rope = c.rope;
    a.ws = c.ws;
    a.err = c.err;
    a.tokens = (int)c.tokens;
    a.T = (int)c.T;
    a.D = c.D;
    a.w_bf16 = c.w_dt;
    a.eps = c.eps;
    qk_bwd_kernel<T, LPR, NB><<<a.grid[0] + a.grid[1], kWarps * 32, 0, s>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;

    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((c.D + 31) / 32), 2);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, qk_dw_reduce_kernel, (const float*)c.ws, c.dw[0], c.dw[1], c.D,
                              a.grid[0], a.grid[1]);
}

template <typename T, bool NB>
cudaError_t by_lanes(const QkCall& c, cudaStream_t s) {
    const bool bwd = c.ws != nullptr;
    switch (lanes_per_row(c.D)) {
        case 1: return bwd ? run_bwd<T, 1, NB>(c, s) : run_fwd<T, 1, NB>(c, s);
        case 2: return bwd ? run_bwd<T, 2, NB>(c, s) : run_fwd<T, 2, NB>(c, s);
        case 4: return bwd ? run_bwd<T, 4, NB>(c, s) : run_fwd<T, 4, NB>(c, s);
        case 8: return bwd ? run_bwd<T, 8, NB>(c, s) : run_fwd<T, 8, NB>(c, s);
        case 16: return bwd ? run_bwd<T, 16, NB>(c, s) : run_fwd<T, 16, NB>(c, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_qk(const QkCall& c, cudaStream_t s) {
    if (c.x_dt == 1)
        return c.neighbours ? by_lanes<__nv_bfloat16, true>(c, s)
                            : by_lanes<__nv_bfloat16, false>(c, s);
    return c.neighbours ? by_lanes<float, true>(c, s) : by_lanes<float, false>(c, s);
}

}  // namespace rmsn
