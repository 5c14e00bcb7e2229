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
// Both are bound by HBM: every row is read and written once, and the arithmetic takes 56 to 59% of
// the issue slots.  A token's angles and the weights stay in registers while a warp goes over the
// token's heads.  Forward, measured on GB300 with 32 + 8 heads of 128 in bf16: T = 8192 30.5 us,
// T = 32768 113 us (89% of the copy rate).  A persistent grid that streams its rows through shared
// memory, as the backward does, was slower (33 us): the forward's four loads in flight per lane
// cost no more registers than it has.
#include <type_traits>

#include "rmsn_internal.h"
#include "rmsn_pipe.cuh"
#include "rmsn_qk.cuh"

namespace rmsn {

namespace {

constexpr int kWarps = 4;  // warps per CTA (they are independent)
constexpr int kBlock = 8;  // dw terms added in FP32 before a compensated addition, at most

struct FwdArgs {
    Heads x[2], y[2];
    const void* w[2];
    Span span[2];
    Rope rope;
    unsigned* err;
    int tokens, T, D, w_bf16;
    bool wide;  // rows of the outputs start on 32 bytes
    float eps;
};

// One unit of work per warp: tpw tokens and the chunks [part * per_part, ...) of their heads.
// blockIdx.y picks q or k and the part, blockIdx.x and the warp the tokens.
// U chunks are in flight: up to 4 KiB of rows per warp as far as a unit has them; units of one or
// two chunks (few heads) take fewer registers and more CTAs instead (T = 8192 with 4 + 4 heads of
// 128 12.7 -> 9.9 us, with 1 + 1 4.7 -> 3.7).
template <typename T, int LPR, bool NB, int U>
__global__ void __launch_bounds__(kWarps * 32, U == 1 ? 7 : U == 2 && sizeof(T) == 2 ? 6 : 5)
    qk_fwd_kernel(const FwdArgs a) {
    constexpr int RPW = 32 / LPR;
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

    const float inv_d = __frcp_rn((float)a.D);
    Angles ang;
    f2 w0[4], w1[4];
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
            if (lane_ok && rl.turns) {
                const int64_t at = tk.pos * (a.rope.rd / 2) + 8 * l;
                ang.load(a.rope.cos + at, a.rope.sin + at);
            }
            load_weights(a.w[side], a.w_bf16, rl.off0, rl.off1, lane_ok, w0, w1);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int h = ((c + i) << sp.log_hpw) + hsub;
            if (c + i >= c1) break;  // the same for the whole warp
            f2 u[4], v[4];
            r0[i].pairs(u);
            r1[i].pairs(v);
            norm_rotate<NB, LPR>(u, v, w0, w1, ang, inv_d, a.eps);
            if (lane_ok && h < sp.heads) {
                T* to = y + h * syh;
                store_row<T, NB>(to + rl.off0, to + rl.off1, u, v, a.wide);
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
    bool wide;  // rows of the outputs start on 32 bytes
    float eps;
};

// Shared memory of the backward: the rings of rows of x and g, as they lie in memory (a row of
// LPR lanes has LPR * 16 elements' room), and every lane's (high, low) sums.
template <typename T>
struct BwdSmem {
    static constexpr int S = sizeof(T) == 2 ? 4 : 3;  // 8 and 12 KiB per warp
    union {
        T ring[kWarps][S][2][512];
        float merge[8][2][64];  // of heads of at most 64
    };
    ulonglong2 sums[2][4][kWarps * 32];  // high, low: four pairs of f2 per lane
};

// Persistent: the first grid[0] CTAs take q's units, the others k's; a unit is tpw tokens and
// one part of their heads (up to 8 chunks).  Rows stream through a ring in shared memory that
// belongs to the warp (asynchronous copies, no CTA barriers), so the bytes in flight do not cost
// registers.  The lanes of a row copy it piece by piece in the order of memory, whatever dims they
// work on: with each lane copying its own dims, 16-byte pieces 32 bytes apart (FP32; neighbouring
// pairs) held the copies to 2.8 TB/s at any depth of the ring.  A lane adds the dw terms of up to
// kBlock chunks in FP32 and such sums to a (high, low) pair with TwoSum; the pairs of the CTA's
// lanes are merged in a fixed order and written to the workspace, whose CTA partials
// qk_dw_reduce_kernel adds in a fixed order.  Two-element FP32 instructions halve the arithmetic.
//
// Measured on GB300 with the reduce, 32 + 8 heads of 128: bf16, T = 8192 43.8 us, 86% of the copy
// rate, T = 32768 165 us, 91% (373 us with register loads, scalar arithmetic and TwoSum per term);
// FP32, T = 8192 83 us, 90% (121 us before the copies went in memory order).  The launches, the
// first copies and the merges cost 6 us: with 4 + 4 heads of 128, T = 8192, 44%.  Merging the lanes
// by shuffles instead of from shared memory took 1 to 2 us more.  Deeper rings are
// slower, for DRAM's sake: bf16, T = 32768 with 4, 5, 6 and 7 stages 160, 169, 173 and 176 us.
template <typename T, int LPR, bool NB>
__global__ void __launch_bounds__(kWarps * 32, 3)
    qk_bwd_kernel(const BwdArgs a) {
    using Sm = BwdSmem<T>;
    constexpr int RPW = 32 / LPR, S = Sm::S, E = 16 / sizeof(T);
    // A unit's angles are loaded while the unit before it is worked on, its position one more
    // ahead; the FP32 kernel has no registers left for that.
    constexpr bool AHEAD = sizeof(T) == 2;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    Sm& sm = *reinterpret_cast<Sm*>(smem_raw);
    asm volatile("griddepcontrol.launch_dependents;");  // the reduce waits for this grid's end
    const int side = (int)blockIdx.x < a.grid[0] ? 0 : 1;
    const int cta = blockIdx.x - (side ? a.grid[0] : 0);
    const Span sp = a.span[side];
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31, l = lane % LPR, rr = lane / LPR;
    const int hsub = rr & ((1 << sp.log_hpw) - 1), tsub = rr >> sp.log_hpw;
    const int tpw = RPW >> sp.log_hpw;
    const int64_t units = ((int64_t)a.tokens + tpw - 1) / tpw * sp.parts;
    const int64_t stride = (int64_t)a.grid[side] * kWarps;
    const bool dims_ok = 16 * l < a.D;

    RowLane<NB> rl;
    rl.init(l, a.rope.rd);
    f2 w0[4], w1[4], acc[8];
    load_weights(a.w[side], a.w_bf16, rl.off0, rl.off1, dims_ok, w0, w1);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        sm.sums[0][i][threadIdx.x] = sm.sums[1][i][threadIdx.x] = make_ulonglong2(0ull, 0ull);
    if (!dims_ok)  // lanes past the row's end add zeros to its sums
        for (int i = 0; i < 2 * S; ++i)
            for (int e = 0; e < 16; ++e) sm.ring[warp][i / 2][i % 2][rr * LPR * 16 + 16 * l + e] = T(0.f);
    const int hpw = 1 << sp.log_hpw;
    const int64_t step_x = hpw * a.x[side].sh, step_g = hpw * a.g[side].sh;
    const int64_t step_d = hpw * a.dx[side].sh;
    const float inv_d = __frcp_rn((float)a.D);

    // A place in the warp's line of chunks: the unit, the next head of this row and the end of
    // the unit's part of them, and the row's token.
    struct At {
        int64_t unit;
        int c, c1, tok;
    };
    auto enter = [&](At& at) {
        const int64_t grp = sp.parts == 1 ? at.unit
                            : (at.unit >> 32) ? at.unit / sp.parts
                                              : (int64_t)((uint32_t)at.unit / (uint32_t)sp.parts);
        const int part = (int)(at.unit - grp * sp.parts);
        at.c = part * sp.per_part;
        at.c1 = min(sp.chunks, at.c + sp.per_part);
        at.tok = (int)min(grp * tpw + tsub, (int64_t)a.tokens);
    };
    // The copying side runs S - 1 chunks ahead; px and pg: this lane's first piece of its row.
    const uint32_t ring = smem_addr(&sm.ring[warp][0][0][rr * LPR * 16 + E * l]);
    const int pieces = a.D / E;
    const T *px = nullptr, *pg = nullptr;
    At in{(int64_t)cta * kWarps + warp, 0, 0, 0};
    auto rows_in = [&]() {
        if (in.unit >= units) return;
        enter(in);
        const int t = in.tok < a.tokens ? in.tok : 0;
        const int b = a.tokens == a.T ? 0 : t / a.T;
        const int h = (in.c << sp.log_hpw) + hsub;
        px = a.x[side].row<T>(b, t - b * a.T) + h * a.x[side].sh + E * l;
        pg = a.g[side].row<T>(b, t - b * a.T) + h * a.g[side].sh + E * l;
    };
    auto fetch = [&](int stage) {  // the next chunk of rows, if there is one
        if (in.unit < units) {
            if (in.tok < a.tokens && (in.c << sp.log_hpw) + hsub < sp.heads) {
                const uint32_t dst = ring + (uint32_t)stage * (1024 * sizeof(T));
#pragma unroll
                for (int i = 0; i < (int)sizeof(T); ++i)
                    if (l + i * LPR < pieces) {
                        copy16(dst + i * LPR * 16, px + i * LPR * E);
                        copy16(dst + 512 * sizeof(T) + i * LPR * 16, pg + i * LPR * E);
                    }
            }
            px += step_x;
            pg += step_g;
            if (++in.c == in.c1) {
                in.unit += stride;
                rows_in();
            }
        }
        copy_commit();
    };
    rows_in();
#pragma unroll
    for (int i = 0; i < S - 1; ++i) fetch(i);

#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0ull;
    auto flush = [&]() {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            ulonglong2 hi = sm.sums[0][i][threadIdx.x], lo = sm.sums[1][i][threadIdx.x];
            f2 h0 = hi.x, l0 = lo.x, h1 = hi.y, l1 = lo.y;
            comp_add2(h0, l0, acc[2 * i]);
            comp_add2(h1, l1, acc[2 * i + 1]);
            sm.sums[0][i][threadIdx.x] = make_ulonglong2(h0, h1);
            sm.sums[1][i][threadIdx.x] = make_ulonglong2(l0, l1);
            acc[2 * i] = acc[2 * i + 1] = 0ull;
        }
    };
    auto position = [&](const At& at) -> int64_t {
        const int t = at.tok < a.tokens ? at.tok : 0, b = a.tokens == a.T ? 0 : t / a.T;
        return at.unit < units ? __ldg(a.rope.pos + b * a.rope.pos_sb + (t - b * a.T) * a.rope.pos_st) : 0;
    };
    auto turn = [&](Angles& ang, int64_t pos) {
        ang.identity();
        if (rl.turns && pos >= 0 && pos < a.rope.rows) {
            const int64_t p = pos * (a.rope.rd / 2) + 8 * l;
            ang.load(a.rope.cos + p, a.rope.sin + p);
        }
    };
    int stage = 0, added = 0;
    At at{(int64_t)cta * kWarps + warp, 0, 0, 0}, nx{at.unit + stride, 0, 0, 0};
    enter(at);
    int64_t pos = 0, pos_nx = 0;
    Angles ang, ang_nx;
    if (AHEAD) {
        enter(nx);
        pos = position(at);
        pos_nx = position(nx);
        turn(ang_nx, pos);
    }
    while (at.unit < units) {
        At n2{nx.unit + stride, 0, 0, 0};
        if (!AHEAD) pos = position(at);
        const bool there = pos >= 0 && pos < a.rope.rows;
        const bool ok = at.tok < a.tokens && there && dims_ok;
        if (!there && at.tok < a.tokens && side == 0 && at.c == 0 && l == 0 && hsub == 0)
            atomicOr(a.err, ERR_INDEX);
        if (AHEAD) {
            ang = ang_nx;
            turn(ang_nx, pos_nx);
            pos = pos_nx;
            enter(n2);
            pos_nx = position(n2);
        } else {
            turn(ang, pos);
        }
        const int tok = at.tok < a.tokens ? at.tok : 0, bt = a.tokens == a.T ? 0 : tok / a.T;
        int h = (at.c << sp.log_hpw) + hsub;
        T* d0 = a.dx[side].row<T>(bt, tok - bt * a.T) + h * a.dx[side].sh;
        T* d1 = d0 + rl.off1;
        d0 += rl.off0;
        if (added + at.c1 - at.c > kBlock) {
            flush();
            added = 0;
        }
        added += at.c1 - at.c;
        for (int c = at.c; c < at.c1; ++c) {
            copy_wait<S - 2>();
            __syncwarp();  // the other lanes' pieces, and their reads of the stage before
            const T* row = &sm.ring[warp][stage][0][rr * LPR * 16];
            f2 x0[4], x1[4], h0[4], h1[4];
            pairs8(row + rl.off0, x0);
            pairs8(row + rl.off1, x1);
            pairs8(row + 512 + rl.off0, h0);
            pairs8(row + 512 + rl.off1, h1);
            // the stage read one chunk ago is free
            fetch(stage == 0 ? S - 1 : stage - 1);
            stage = stage + 1 == S ? 0 : stage + 1;

            rotate2<NB, true>(h0, h1, ang);
            f2 ss2 = 0ull, dot2 = 0ull;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                ss2 = fma2(x0[i], x0[i], ss2);
                dot2 = fma2(mul2(h0[i], w0[i]), x0[i], dot2);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                ss2 = fma2(x1[i], x1[i], ss2);
                dot2 = fma2(mul2(h1[i], w1[i]), x1[i], dot2);
            }
            const float ss = row_sum<LPR>(f2_lo(ss2) + f2_hi(ss2));
            const float dot = row_sum<LPR>(f2_lo(dot2) + f2_hi(dot2));
            const float r = row_rstd(ss, inv_d, a.eps);
            // dx = (h r) w - x r k,  k = r^2 mean(g x);  dw += (h r) x
            const f2 r2 = f2_splat(r), nk = f2_splat(-(r * (r * (r * (dot * inv_d)))));
            if (ok && h < sp.heads) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const f2 hr = mul2(h0[i], r2);
                    acc[i] = fma2(hr, x0[i], acc[i]);
                    x0[i] = fma2(x0[i], nk, mul2(hr, w0[i]));
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const f2 hr = mul2(h1[i], r2);
                    acc[4 + i] = fma2(hr, x1[i], acc[4 + i]);
                    x1[i] = fma2(x1[i], nk, mul2(hr, w1[i]));
                }
                store_row<T, NB>(d0, d1, x0, x1, a.wide);
            }
            h += hpw;
            d0 += step_d;
            d1 += step_d;
        }
        at = nx;
        if (AHEAD)
            nx = n2;
        else
            nx.unit += stride, enter(at);
    }
    flush();
    copy_wait<0>();
    __syncthreads();

    // Every column's sums of the CTA's 128 / LPR rows: G threads per column merge 16 rows (or 8)
    // each in order, and their results are merged in order.
    constexpr int G = LPR < 8 ? 8 / LPR : 1, ROWS = kWarps * 32 / LPR / G;
    float* out = a.ws + (int64_t)blockIdx.x * 2 * a.D;
    const float* sums = reinterpret_cast<const float*>(sm.sums);
    for (int x = threadIdx.x; x < 16 * LPR * G; x += kWarps * 32) {
        const int cl = x % LPR, e = x / LPR % 16, part = x / (16 * LPR);
        if (16 * cl >= a.D) continue;
        const float* p = sums + ((e / 4) * kWarps * 32 + part * ROWS * LPR + cl) * 4 + e % 4;
        constexpr int LOW = 4 * kWarps * 32 * 4;  // from a high to its low
        float h = p[0], low = p[LOW];
#pragma unroll 4
        for (int r = 1; r < ROWS; ++r) comp_merge(h, low, p[r * LPR * 4], p[r * LPR * 4 + LOW]);
        RowLane<NB> at;
        at.init(cl, a.rope.rd);
        const int col = e < 8 ? at.off0 + e : at.off1 + e - 8;
        if (G == 1) {
            out[col] = h;
            out[a.D + col] = low;
        } else {
            sm.merge[part][0][col] = h;
            sm.merge[part][1][col] = low;
        }
    }
    if (G == 1) return;
    __syncthreads();
    for (int col = threadIdx.x; col < a.D; col += kWarps * 32) {
        float h = sm.merge[0][0][col], low = sm.merge[0][1][col];
#pragma unroll
        for (int i = 1; i < G; ++i) comp_merge(h, low, sm.merge[i][0][col], sm.merge[i][1][col]);
        out[col] = h;
        out[a.D + col] = low;
    }
}

// dwq and dwk from the CTA partials: one CTA per 32 columns of one of them; warp w of 32 adds
// the partials w, w + 32, ... in order, the 32 sums are merged by a fixed tree, and high + low is
// rounded once.
constexpr int kReduceWarps = 32;

__global__ void __launch_bounds__(kReduceWarps * 32)
    qk_dw_reduce_kernel(const float* __restrict__ ws, float* dwq, float* dwk, int D, int gq, int gk) {
    __shared__ float sh[kReduceWarps][33], sl[kReduceWarps][33];
    constexpr int U = 15;  // all of a warp's partials are in flight at once
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;
    const int n = blockIdx.y ? gk : gq;
    const float* p = ws + (blockIdx.y ? (int64_t)gq * 2 * D : 0);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float h = 0.f, e = 0.f;
    if (col < D) {
        const uint32_t step = 2 * kReduceWarps * D;
        p += col;
        for (int i = warp; i < n; i += U * kReduceWarps) {
            float vh[U], vl[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t at = (uint32_t)i * 2 * D + u * step;
                vh[u] = vl[u] = 0.f;
                if (i + kReduceWarps * u < n) {
                    vh[u] = __ldcg(p + at);
                    vl[u] = __ldcg(p + at + D);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) comp_merge(h, e, vh[u], vl[u]);
        }
    }
    sh[warp][lane] = h;
    sl[warp][lane] = e;
    __syncthreads();
    // a column's 32 sums go to one warp and are merged pairwise
    h = sh[lane][warp];
    e = sl[lane][warp];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float ho = __shfl_down_sync(0xffffffffu, h, o);
        const float eo = __shfl_down_sync(0xffffffffu, e, o);
        comp_merge(h, e, ho, eo);
    }
    const int out = blockIdx.x * 32 + warp;
    if (lane == 0 && out < D) (blockIdx.y ? dwk : dwq)[out] = __fadd_rn(h, e);
}

// Whether every row of both outputs starts on 32 bytes.
bool rows_on_32_bytes(const Heads (&y)[2], int dt) {
    const uintptr_t e = dt == 1 ? 2 : 4;
    for (const Heads& h : y)
        if ((reinterpret_cast<uintptr_t>(h.p) | (uintptr_t)h.sb * e | (uintptr_t)h.st * e |
             (uintptr_t)h.sh * e) % 32 != 0)
            return false;
    return true;
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
    a.wide = rows_on_32_bytes(c.y, c.x_dt);
    a.eps = c.eps;
    const dim3 grid((unsigned)gx, a.span[0].parts + a.span[1].parts);
    constexpr int U = sizeof(T) == 2 ? 4 : 2;
    const int most = a.span[0].per_part > a.span[1].per_part ? a.span[0].per_part : a.span[1].per_part;
    if (most == 1)
        qk_fwd_kernel<T, LPR, NB, 1><<<grid, kWarps * 32, 0, s>>>(a);
    else if (U > 2 && most == 2)
        qk_fwd_kernel<T, LPR, NB, 2><<<grid, kWarps * 32, 0, s>>>(a);
    else
        qk_fwd_kernel<T, LPR, NB, U><<<grid, kWarps * 32, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T, int LPR, bool NB>
cudaError_t run_bwd(const QkCall& c, cudaStream_t s) {
    constexpr int RPW = 32 / LPR;
    BwdArgs a{};
    const int heads[2] = {c.heads[0], c.heads[1]};
    const int per = pick_per_part(heads, 2, c.tokens, RPW, c.sms);
    int64_t units[2], work[2];
    for (int i = 0; i < 2; ++i) {
        a.x[i] = c.x[i];
        a.g[i] = c.g[i];
        a.dx[i] = c.y[i];
        a.w[i] = c.w[i];
        a.span[i] = make_span(heads[i], RPW, per);
        units[i] = groups_of(c.tokens, a.span[i], RPW) * a.span[i].parts;
        work[i] = units[i] * (2 * a.span[i].per_part + (sizeof(T) == 2 ? 2 : 3));
    }
    // The CTAs of both sides together are those that are resident at once, shared out by the
    // work: a unit's chunks, and about one chunk's time for entering it (pointers, sums; in FP32,
    // where the angles are waited for, one and a half).  Measured with 32 + 8 heads of 128 (bf16), T = 4096 / 8192 / 32768: with half a chunk's time 28.1 / 47.1
    // / 172 us, with one 27.4 / 45.5 / 167, with one and a half 29.1 / 46.7 / 164; shared out by rows
    // it was a fifth slower, waiting for k's units of two chunks.
    Launch L{};
    L.sms = c.sms;
    L.grid = (int64_t)c.sms * kQkBwdCtasPerSm;
    L.smem = sizeof(BwdSmem<T>);
    int64_t all = 0;
    auto kernel = qk_bwd_kernel<T, LPR, NB>;
    cudaError_t e = fit_grid((const void*)kernel, L, kWarps * 32, &all);
    if (e != cudaSuccess) return e;
    int64_t gk = (int64_t)((double)all * work[1] / ((double)work[0] + work[1]) + 0.5);
    gk = gk < 1 ? 1 : gk > all - 1 ? all - 1 : gk;
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
    a.wide = rows_on_32_bytes(c.y, c.x_dt);
    a.eps = c.eps;
    kernel<<<a.grid[0] + a.grid[1], kWarps * 32, sizeof(BwdSmem<T>), s>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;

    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((c.D + 31) / 32), 2);
    cfg.blockDim = dim3(kReduceWarps * 32);
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
