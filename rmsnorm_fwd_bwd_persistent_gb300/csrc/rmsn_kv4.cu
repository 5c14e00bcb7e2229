// rmsn_kv4.cu -- storing to and reading from the 4-bit cache (layout: rmsn_kv4_layout.h).
//
// kv4_append_kernel is the serving form of the norm + rotation: q is normed, rotated and
// written out, k is normed, rotated, rounded to bf16 and quantised into the cache, v is
// quantised as it is.  Per group of 32 dims of the bf16 values x:
//   z = min x,  s = bf16(max x / 15 - min x / 15),  code = clamp(rint((x - z) / s), 0, 15)
// (IEEE FP32 operations; s = 0: code 0; a group with a NaN or an infinity gets s = z = NaN, so
// it reads back as NaN).  The codes are a function of the bf16 values alone.
// kv4_read_kernel is the inverse: code * s + z, rounded once to bf16.
#include "rmsn_internal.h"
#include "rmsn_kv4.cuh"
#include "rmsn_pipe.cuh"

namespace rmsn {

namespace {

using bf16 = __nv_bfloat16;
constexpr int kWarps = 4;

__device__ __forceinline__ uint32_t bf16_bits(float v) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// Quantises the 16 neighbouring dims of this lane (two lanes hold a group): two words of eight
// codes, and the group's scale (low half) and minimum (high half) as bf16.
__device__ __forceinline__ void quantise16(const Raw8<bf16>& a, const Raw8<bf16>& b,
                                           uint32_t (&word)[2], uint32_t& scale_min) {
    float x[2][8];
    a.get(x[0]);
    b.get(x[1]);
    float mn = x[0][0], mx = x[0][0], odd = 0.f;
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            mn = fminf(mn, x[e][i]);
            mx = fmaxf(mx, x[e][i]);
            odd = fmaf(x[e][i], 0.f, odd);  // NaN if any element is not finite
        }
    mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    odd += __shfl_xor_sync(0xffffffffu, odd, 1);
    const bool bad = odd != odd;
    const uint32_t sb = bf16_bits(__fsub_rn(__fdiv_rn(mx, 15.f), __fdiv_rn(mn, 15.f)));
    const float s = __uint_as_float(sb << 16);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        word[e] = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float c = rintf(__fdiv_rn(__fsub_rn(x[e][i], mn), s));
            const uint32_t code = s > 0.f ? (uint32_t)fminf(fmaxf(c, 0.f), 15.f) : 0u;
            word[e] |= code << (4 * i);
        }
        if (bad) word[e] = 0u;
    }
    scale_min = bad ? 0x7fc07fc0u : sb | (bf16_bits(mn) << 16);
}

struct AppendArgs {
    Heads x[3], y;  // q, k, v in; q out
    const void* w[2];
    Span span[3];
    Rope rope;
    uint8_t* cache;
    const int64_t* slots;
    int64_t pages;
    unsigned* err;
    int tokens, blocks_per_page, kv_heads, w_bf16;
    float eps;
};

template <int LPR, bool NB>
__global__ void __launch_bounds__(kWarps * 32) kv4_append_kernel(const AppendArgs a) {
    constexpr int RPW = 32 / LPR, D = 16 * LPR, U = 2;
    __shared__ __align__(16) bf16 turn[kWarps][RPW * D];
    int part = blockIdx.y, side = 0;
    while (side < 2 && part >= a.span[side].parts) part -= a.span[side++].parts;
    const Span sp = a.span[side];
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31, l = lane % LPR, rr = lane / LPR;
    const int hsub = rr & ((1 << sp.log_hpw) - 1), tsub = rr >> sp.log_hpw;
    const int tpw = RPW >> sp.log_hpw;
    const int64_t first = ((int64_t)blockIdx.x * kWarps + warp) * tpw;
    if (first >= a.tokens) return;
    const bool report = side == 0 && part == 0 && l == 0 && hsub == 0;
    Token tk = find_token((int)min(first + tsub, (int64_t)a.tokens), a.tokens, a.tokens, a.rope,
                          a.err, false);
    int64_t slot = -1;
    if (first + tsub < a.tokens) {
        slot = __ldg(a.slots + tk.t);
        const bool in = slot < a.pages * a.blocks_per_page * kKv4Block;
        if (slot >= 0 && report && (!in || !tk.ok)) atomicOr(a.err, ERR_INDEX);
        tk.ok = tk.ok && slot >= 0 && in;
    }
    const bool ok = tk.ok;

    RowLane<NB> rl;
    rl.init(l, side == 2 ? 0 : a.rope.rd);
    const bf16* x = a.x[side].row<bf16>(0, tk.t);
    bf16* y = a.y.row<bf16>(0, tk.t);
    const int64_t sxh = a.x[side].sh, syh = a.y.sh;
    const int c1 = min(sp.chunks, (part + 1) * sp.per_part);
    uint8_t* rec0 = a.cache;
    if (ok && side > 0)
        rec0 += kv4_record(slot, a.pages, a.blocks_per_page, a.kv_heads, 0) * kv4_record_bytes(D);
    const int64_t head_bytes = (int64_t)a.blocks_per_page * kv4_record_bytes(D);
    const int r = (int)(slot & (kKv4Block - 1));

    Angles ang;
    float w0[8], w1[8];
    bool have = false;
    for (int c = part * sp.per_part; c < c1; c += U) {
        Raw8<bf16> r0[U], r1[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int h = ((c + i) << sp.log_hpw) + hsub;
            r0[i].clear();
            r1[i].clear();
            if (ok && c + i < c1 && h < sp.heads) {
                r0[i].load(x + h * sxh + rl.off0);
                r1[i].load(x + h * sxh + rl.off1);
            }
        }
        if (!have && side < 2) {  // after the first rows are on their way
            have = true;
            ang.identity();
            if (ok && rl.turns) {
                const int64_t at = tk.pos * (a.rope.rd / 2) + 8 * l;
                ang.load(a.rope.cos + at, a.rope.sin + at);
            }
            load_w8(a.w[side], a.w_bf16, rl.off0, w0);
            load_w8(a.w[side], a.w_bf16, rl.off1, w1);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (c + i >= c1) break;  // the same for the whole warp
            const int h = ((c + i) << sp.log_hpw) + hsub;
            const bool row_ok = ok && h < sp.heads;
            if (side < 2) {
                float u[8], v[8];
                r0[i].get(u);
                r1[i].get(v);
                float ss = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = fmaf(u[e], u[e], ss);
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = fmaf(v[e], v[e], ss);
                const float rs = row_rstd(row_sum<LPR>(ss), (float)D, a.eps);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    u[e] = u[e] * rs * w0[e];
                    v[e] = v[e] * rs * w1[e];
                }
                rotate<NB, false>(u, v, ang);
                r0[i].set(u);
                r1[i].set(v);
                if (side == 0) {
                    if (row_ok) {
                        r0[i].store(y + h * syh + rl.off0);
                        r1[i].store(y + h * syh + rl.off1);
                    }
                    continue;
                }
                if (!NB) {  // to neighbouring dims: lane l takes dims [16l, 16l + 16)
                    bf16* row = turn[warp] + rr * D;
                    r0[i].store(row + rl.off0);
                    r1[i].store(row + rl.off1);
                    __syncwarp();
                    r0[i].a = *reinterpret_cast<const uint4*>(row + 16 * l);
                    r1[i].a = *reinterpret_cast<const uint4*>(row + 16 * l + 8);
                    __syncwarp();
                }
            }
            uint32_t word[2], sm;
            quantise16(r0[i], r1[i], word, sm);
            if (!row_ok) continue;
            uint8_t* rec = rec0 + h * head_bytes;
            const int j = l >> 1;
            if (side == 1) {
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    *reinterpret_cast<uint32_t*>(rec + kv4_k_word(D, r, 2 * l + e)) = word[e];
                if ((l & 1) == 0)
                    *reinterpret_cast<uint32_t*>(rec + kv4_k_scale(D, r, j)) = sm;
            } else {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int wd = 2 * l + e;
                    *reinterpret_cast<uint32_t*>(rec + kv4_v_unit(D, r, wd / (D / 64)) +
                                                 4 * (wd % (D / 64))) = word[e];
                }
                if ((l & 1) == 0) {
                    uint16_t* p = reinterpret_cast<uint16_t*>(rec + kv4_v_scale(D, r, j));
                    p[0] = (uint16_t)(sm & 0xffffu);
                    p[2] = (uint16_t)(sm >> 16);
                }
            }
        }
    }
}

// Eight codes, scale and minimum -> eight values.
__device__ __forceinline__ void values8(uint32_t word, float s, float z, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = fmaf((float)((word >> (4 * i)) & 15u), s, z);
}

struct ReadArgs {
    const uint8_t* cache;
    const int64_t* slots;
    Heads k, v;
    Span span;
    int64_t pages;
    unsigned* err;
    int tokens, blocks_per_page;
};

template <int LPR>
__global__ void __launch_bounds__(kWarps * 32) kv4_read_kernel(const ReadArgs a) {
    constexpr int RPW = 32 / LPR, D = 16 * LPR, U = 4;
    const Span sp = a.span;
    const int part = blockIdx.y;
    const int lane = threadIdx.x & 31, l = lane % LPR, rr = lane / LPR;
    const int hsub = rr & ((1 << sp.log_hpw) - 1), tsub = rr >> sp.log_hpw;
    const int tpw = RPW >> sp.log_hpw;
    const int64_t tok = ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * tpw + tsub;
    if (tok >= a.tokens) return;
    const int64_t slot = __ldg(a.slots + tok);
    if (slot < 0) return;
    if (slot >= a.pages * a.blocks_per_page * kKv4Block) {
        if (part == 0 && l == 0 && hsub == 0) atomicOr(a.err, ERR_INDEX);
        return;
    }
    const uint8_t* rec0 =
        a.cache + kv4_record(slot, a.pages, a.blocks_per_page, sp.heads, 0) * kv4_record_bytes(D);
    const int64_t head_bytes = (int64_t)a.blocks_per_page * kv4_record_bytes(D);
    const int r = (int)(slot & (kKv4Block - 1));
    const int j = l >> 1;
    bf16* ko = a.k.row<bf16>(0, (int)tok) + 16 * l;
    bf16* vo = a.v.row<bf16>(0, (int)tok) + 16 * l;
    const int c1 = min(sp.chunks, (part + 1) * sp.per_part);
    for (int c = part * sp.per_part; c < c1; c += U) {
        uint32_t kw[U][2], vw[U][2], ks[U], vs[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int h = ((c + i) << sp.log_hpw) + hsub;
            if (c + i >= c1 || h >= sp.heads) continue;
            const uint8_t* rec = rec0 + h * head_bytes;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int wd = 2 * l + e;
                kw[i][e] = *reinterpret_cast<const uint32_t*>(rec + kv4_k_word(D, r, wd));
                vw[i][e] = *reinterpret_cast<const uint32_t*>(
                    rec + kv4_v_unit(D, r, wd / (D / 64)) + 4 * (wd % (D / 64)));
            }
            ks[i] = *reinterpret_cast<const uint32_t*>(rec + kv4_k_scale(D, r, j));
            const uint16_t* p = reinterpret_cast<const uint16_t*>(rec + kv4_v_scale(D, r, j));
            vs[i] = (uint32_t)p[0] | ((uint32_t)p[2] << 16);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int h = ((c + i) << sp.log_hpw) + hsub;
            if (c + i >= c1 || h >= sp.heads) continue;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float f[8];
                Raw8<bf16> o;
                values8(kw[i][e], bf16_lo(ks[i]), bf16_hi(ks[i]), f);
                o.set(f);
                o.store(ko + h * a.k.sh + 8 * e);
                values8(vw[i][e], bf16_lo(vs[i]), bf16_hi(vs[i]), f);
                o.set(f);
                o.store(vo + h * a.v.sh + 8 * e);
            }
        }
    }
}

template <int LPR, bool NB>
cudaError_t run_append(const Kv4Append& c, cudaStream_t s) {
    constexpr int RPW = 32 / LPR;
    AppendArgs a{};
    const int heads[3] = {c.heads, c.kv_heads, c.kv_heads};
    const int per = pick_per_part(heads, 3, c.tokens, RPW, c.sms);
    int64_t gx = 1;
    int gy = 0;
    for (int i = 0; i < 3; ++i) {
        a.x[i] = c.x[i];
        a.span[i] = make_span(heads[i], RPW, per);
        const int64_t g = (groups_of(c.tokens, a.span[i], RPW) + kWarps - 1) / kWarps;
        gx = g > gx ? g : gx;
        gy += a.span[i].parts;
    }
    a.y = c.y;
    a.w[0] = c.w[0];
    a.w[1] = c.w[1];
    a.rope = c.rope;
    a.cache = c.cache;
    a.slots = c.slots;
    a.pages = c.pages;
    a.err = c.err;
    a.tokens = (int)c.tokens;
    a.blocks_per_page = c.blocks_per_page;
    a.kv_heads = c.kv_heads;
    a.w_bf16 = c.w_dt;
    a.eps = c.eps;
    kv4_append_kernel<LPR, NB><<<dim3((unsigned)gx, gy), kWarps * 32, 0, s>>>(a);
    return cudaGetLastError();
}

template <int LPR>
cudaError_t run_read(const Kv4Read& c, cudaStream_t s) {
    constexpr int RPW = 32 / LPR;
    ReadArgs a{};
    const int per = pick_per_part(&c.kv_heads, 1, c.tokens, RPW, c.sms);
    a.cache = c.cache;
    a.slots = c.slots;
    a.k = c.k;
    a.v = c.v;
    a.span = make_span(c.kv_heads, RPW, per);
    a.pages = c.pages;
    a.err = c.err;
    a.tokens = (int)c.tokens;
    a.blocks_per_page = c.blocks_per_page;
    const int64_t gx = (groups_of(c.tokens, a.span, RPW) + kWarps - 1) / kWarps;
    kv4_read_kernel<LPR><<<dim3((unsigned)gx, a.span.parts), kWarps * 32, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4Append& c, cudaStream_t s) {
    switch (c.D) {
        case 64: return c.neighbours ? run_append<4, true>(c, s) : run_append<4, false>(c, s);
        case 128: return c.neighbours ? run_append<8, true>(c, s) : run_append<8, false>(c, s);
        case 256: return c.neighbours ? run_append<16, true>(c, s) : run_append<16, false>(c, s);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_kv4_read(const Kv4Read& c, cudaStream_t s) {
    switch (c.D) {
        case 64: return run_read<4>(c, s);
        case 128: return run_read<8>(c, s);
        case 256: return run_read<16>(c, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace rmsn
