// rmsn_kv4.cu -- storing to and reading from the 4-bit cache (layout: rmsn_kv4_layout.h).
//
// kv4_append_kernel is the serving form of the norm + rotation: q is normed, rotated and
// written out, k is normed, rotated, rounded to bf16 and quantised into the cache, v is
// quantised as it is.  Per group of 32 dims of the bf16 values x:
//   z = min x,  s = bf16(max x / 15 - min x / 15),  code = clamp(rint((x - z) / s), 0, 15)
// (IEEE FP32 operations; s = 0: code 0; a group with a NaN or an infinity gets s = z = NaN, so
// it reads back as NaN).  The codes are a function of the bf16 values alone.
// kv4_read_kernel is the inverse: code * s + z, rounded once to bf16.
#include <algorithm>

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

__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
    asm("min.NaN.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
    return a;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
    return a;
}

// Quantises the 16 neighbouring dims of this lane (two lanes hold a group): two words of eight
// codes, and the group's scale (low half) and minimum (high half) as bf16.
//
// The quotient t/s (t = x - z) is formed as q = t y, y = 1/s rounded, and one step
// q + y (t - q s), whose remainder is exact (Markstein).  That is within 2^-22 of half a step of
// t/s, and since s has 8 bits and t 24, t/s is never closer than 2^-9 of a step to the middle
// between two FP32 numbers: so it is the rounded quotient that a division gives, at a fifth of the
// instructions.  Scales outside [2^-60, 2^60], where a product could leave the range, divide.
__device__ __forceinline__ void quantise16(const Raw8<bf16>& a, const Raw8<bf16>& b,
                                           uint32_t (&word)[2], uint32_t& scale_min) {
    uint32_t lo = min2(min2(min2(a.a.x, a.a.y), min2(a.a.z, a.a.w)),
                       min2(min2(b.a.x, b.a.y), min2(b.a.z, b.a.w)));
    uint32_t up = max2(max2(max2(a.a.x, a.a.y), max2(a.a.z, a.a.w)),
                       max2(max2(b.a.x, b.a.y), max2(b.a.z, b.a.w)));
    lo = min2(lo, __shfl_xor_sync(0xffffffffu, lo, 1));
    up = max2(up, __shfl_xor_sync(0xffffffffu, up, 1));
    lo = min2(lo, __byte_perm(lo, lo, 0x1032));
    up = max2(up, __byte_perm(up, up, 0x1032));
    const float mn = bf16_lo(lo), mx = bf16_lo(up);
    const uint32_t sb = bf16_bits(__fsub_rn(__fdiv_rn(mx, 15.f), __fdiv_rn(mn, 15.f)));
    const float s = __uint_as_float(sb << 16);
    const bool bad = !(fabsf(mn) <= 3.402823466e38f && fabsf(mx) <= 3.402823466e38f);
    f2 x[2][4];
    Pairs<bf16>::get(a.a, x[0]);
    Pairs<bf16>::get(b.a, x[1]);
    if (s >= 8.67361738e-19f && s <= 1.152921505e18f) {
        const float y = __frcp_rn(s);
        const f2 y2 = f2_splat(y), n2 = f2_splat(-s), m2 = f2_splat(mn);
        const f2 magic = f2_splat(12582912.f);  // 1.5 2^23: the sum's low bits are the integer
        constexpr uint32_t kMagic = 0x4B400000u * 0x11111111u;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            uint32_t wd = 0u - kMagic;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f2 t = sub2(x[e][i], m2);
                const f2 q = mul2(t, y2);
                const f2 c = add2(fma2(fma2(q, n2, t), y2, q), magic);
                wd += (__float_as_uint(f2_lo(c)) << (8 * i)) + (__float_as_uint(f2_hi(c)) << (8 * i + 4));
            }
            word[e] = wd;
        }
        scale_min = sb | (lo << 16);
        return;
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        word[e] = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float v = i & 1 ? f2_hi(x[e][i / 2]) : f2_lo(x[e][i / 2]);
            const float c = rintf(__fdiv_rn(__fsub_rn(v, mn), s));
            if (s > 0.f && !bad) word[e] |= (uint32_t)fminf(fmaxf(c, 0.f), 15.f) << (4 * i);
        }
    }
    scale_min = bad ? 0x7fc07fc0u : sb | (lo << 16);
}

// Stores the codes of dims [16l, 16l + 16) of token r, and from every second lane its group's
// scale and minimum, to a record.
template <int D>
__device__ __forceinline__ void put16(uint8_t* rec, int r, int l, bool k, const uint32_t (&word)[2],
                                      uint32_t scale_min) {
    const int j = l >> 1;
    if (k) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
            *reinterpret_cast<uint32_t*>(rec + kv4_k_word(D, r, 2 * l + e)) = word[e];
        if ((l & 1) == 0) *reinterpret_cast<uint32_t*>(rec + kv4_k_scale(D, r, j)) = scale_min;
    } else {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int wd = 2 * l + e;
            *reinterpret_cast<uint32_t*>(rec + kv4_v_unit(D, r, wd / (D / 64)) + 4 * (wd % (D / 64))) =
                word[e];
        }
        if ((l & 1) == 0) {
            uint16_t* p = reinterpret_cast<uint16_t*>(rec + kv4_v_scale(D, r, j));
            p[0] = (uint16_t)(scale_min & 0xffffu);
            p[2] = (uint16_t)(scale_min >> 16);
        }
    }
}

struct AppendArgs {
    Heads x[3], y;  // q, k, v in; q out
    const void* w[2];
    Span span[3];
    int grid[3];  // CTAs of q, k and v (streaming kernel)
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
    constexpr int RPW = 32 / LPR, D = 16 * LPR, U = 4;
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
        rec0 += kv4_record_of(slot, a.blocks_per_page, a.kv_heads) * kv4_record_bytes(D);
    const int64_t head_bytes = (int64_t)a.blocks_per_page * kv4_record_bytes(D);
    const int r = (int)(slot & (kKv4Block - 1));

    Angles ang;
    f2 w0[4], w1[4];
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
            load_weights(a.w[side], a.w_bf16, rl.off0, rl.off1, true, w0, w1);
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (c + i >= c1) break;  // the same for the whole warp
            const int h = ((c + i) << sp.log_hpw) + hsub;
            const bool row_ok = ok && h < sp.heads;
            if (side < 2) {
                f2 u[4], v[4];
                r0[i].pairs(u);
                r1[i].pairs(v);
                norm_rotate<NB, LPR>(u, v, w0, w1, ang, 1.f / D, a.eps);
                r0[i].a = Pairs<bf16>::put(u);
                r1[i].a = Pairs<bf16>::put(v);
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
            put16<D>(rec0 + h * head_bytes, r, l, side == 1, word, sm);
        }
    }
}

// A warp's place in its line of units: the unit, the chunks [c, c1) of its part of the heads, and
// the token of this lane's row (tokens where there is none).
struct UnitAt {
    int64_t unit;
    int c, c1, tok;

    __device__ __forceinline__ void enter(const Span& sp, int tpw, int tsub, int tokens) {
        const int64_t grp = sp.parts == 1 ? unit
                            : (unit >> 32) ? unit / sp.parts
                                           : (int64_t)((uint32_t)unit / (uint32_t)sp.parts);
        const int part = (int)(unit - grp * sp.parts);
        c = part * sp.per_part;
        c1 = min(sp.chunks, c + sp.per_part);
        tok = (int)min(grp * tpw + tsub, (int64_t)tokens);
    }
};

// A tensor's rows streamed through a ring in shared memory that belongs to the warp: S stages of
// one chunk, copied asynchronously S - 1 chunks ahead (across units too), so the bytes in flight
// cost neither registers nor CTA barriers.  The lanes of a row copy it piece by piece in the order
// of memory.  Rows that do not exist are not copied; what their places hold is not used.
template <int S, int LPR>
struct RowStream {
    using Ring = bf16[S][512];  // of one warp: its rows one after the other

    const bf16* p;  // this lane's first piece of its row
    int64_t step, stride, units;
    UnitAt in;
    uint32_t ring;
    int hsub, tsub, tpw;

    __device__ __forceinline__ void rows(const Heads& x, const Span& sp, int tokens) {
        if (in.unit >= units) return;
        in.enter(sp, tpw, tsub, tokens);
        p = x.row<bf16>(0, in.tok < tokens ? in.tok : 0) + ((in.c << sp.log_hpw) + hsub) * x.sh +
            8 * (threadIdx.x % LPR);
    }

    // Copies the next chunk, if there is one, to a stage.
    __device__ __forceinline__ void fetch(int stage, const Heads& x, const Span& sp, int tokens) {
        if (in.unit < units) {
            if (in.tok < tokens && (in.c << sp.log_hpw) + hsub < sp.heads) {
                copy16(ring + (uint32_t)stage * 1024, p);
                copy16(ring + (uint32_t)stage * 1024 + 16 * LPR, p + 8 * LPR);
            }
            p += step;
            if (++in.c == in.c1) {
                in.unit += stride;
                rows(x, sp, tokens);
            }
        }
        copy_commit();
    }
};

constexpr int kAppendStages = 4;  // 4 KiB per warp
constexpr int kStreamFrom = 4;    // units per warp from which the streaming kernel is taken

struct AppendSmem {
    bf16 ring[kWarps][kAppendStages][512];
    bf16 turn[kWarps][512];  // rows of k on their way to neighbouring dims
};

// The same for many tokens: persistent, with CTAs for q, for k and for v, each warp streaming the
// rows of its units.  Measured with 32 + 8 + 8 heads of 128: at 16384 tokens (with the read that
// follows) 111.5 us with the kernel above, 93 so; at 64 tokens, where there is nothing to run
// ahead of, 7.6 and 8.5.  With the read that is 57% of the
// copy rate at 4096 tokens, 72% at 16384; 56% of the issue slots are in use.
template <int LPR, bool NB>
__global__ void __launch_bounds__(kWarps * 32) kv4_append_stream_kernel(const AppendArgs a) {
    constexpr int RPW = 32 / LPR, D = 16 * LPR, S = kAppendStages;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    auto& sm = *reinterpret_cast<AppendSmem*>(smem_raw);
    int side = 0, cta = blockIdx.x;
    while (side < 2 && cta >= a.grid[side]) cta -= a.grid[side++];
    const Span sp = a.span[side];
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31, l = lane % LPR, rr = lane / LPR;
    const int hsub = rr & ((1 << sp.log_hpw) - 1), tsub = rr >> sp.log_hpw;
    const int tpw = RPW >> sp.log_hpw;
    const int64_t units = ((int64_t)a.tokens + tpw - 1) / tpw * sp.parts;
    const int64_t first = (int64_t)cta * kWarps + warp, stride = (int64_t)a.grid[side] * kWarps;
    RowLane<NB> rl;
    rl.init(l, side == 2 ? 0 : a.rope.rd);
    const Heads& x = a.x[side];
    RowStream<S, LPR> rows;
    rows.ring = smem_addr(&sm.ring[warp][0][rr * D + 8 * l]);
    rows.stride = stride;
    rows.units = units;
    rows.hsub = hsub;
    rows.tsub = tsub;
    rows.tpw = tpw;
    rows.step = (int64_t)(1 << sp.log_hpw) * x.sh;
    rows.in.unit = first;
    rows.rows(x, sp, a.tokens);
#pragma unroll
    for (int i = 0; i < S - 1; ++i) rows.fetch(i, x, sp, a.tokens);
    f2 w0[4], w1[4];
    load_weights(a.w[side & 1], a.w_bf16, rl.off0, rl.off1, side < 2, w0, w1);
    const int hpw = 1 << sp.log_hpw;
    const int64_t head_bytes = (int64_t)a.blocks_per_page * kv4_record_bytes(D);
    int stage = 0;
    for (UnitAt at{first, 0, 0, 0}; at.unit < units; at.unit += stride) {
        at.enter(sp, tpw, tsub, a.tokens);
        const Token tk = find_token(at.tok, a.tokens, a.tokens, a.rope, a.err, false);
        bool ok = false;
        int r = 0;  // the token's place in its record
        bf16* y = a.y.row<bf16>(0, tk.t);
        uint8_t* rec = a.cache;
        if (at.tok < a.tokens) {
            const int64_t slot = __ldg(a.slots + tk.t);
            const bool in = slot < a.pages * a.blocks_per_page * kKv4Block;
            ok = tk.ok && slot >= 0 && in;
            if (slot >= 0 && (!in || !tk.ok) && side == 0 && at.c == 0 && l == 0 && hsub == 0)
                atomicOr(a.err, ERR_INDEX);
            if (ok && side > 0) {
                rec += kv4_record_of(slot, a.blocks_per_page, a.kv_heads) * kv4_record_bytes(D);
                r = (int)(slot & (kKv4Block - 1));
            }
        }
        Angles ang;
        ang.identity();
        if (ok && rl.turns) {
            const int64_t p = tk.pos * (a.rope.rd / 2) + 8 * l;
            ang.load(a.rope.cos + p, a.rope.sin + p);
        }
        int h = (at.c << sp.log_hpw) + hsub;
        y += h * a.y.sh;
        rec += h * head_bytes;
        for (int c = at.c; c < at.c1; ++c) {
            copy_wait<S - 2>();
            __syncwarp();  // the other lanes' pieces, and their reads of the stage before
            const bf16* row = &sm.ring[warp][stage][rr * D];
            Raw8<bf16> r0{*reinterpret_cast<const uint4*>(row + rl.off0)};
            Raw8<bf16> r1{*reinterpret_cast<const uint4*>(row + rl.off1)};
            // the stage read one chunk ago is free
            rows.fetch(stage == 0 ? S - 1 : stage - 1, x, sp, a.tokens);
            stage = stage + 1 == S ? 0 : stage + 1;
            const bool row_ok = ok && h < sp.heads;
            if (side < 2) {
                f2 u[4], v[4];
                Pairs<bf16>::get(r0.a, u);
                Pairs<bf16>::get(r1.a, v);
                norm_rotate<NB, LPR>(u, v, w0, w1, ang, 1.f / D, a.eps);
                r0.a = Pairs<bf16>::put(u);
                r1.a = Pairs<bf16>::put(v);
            }
            if (side == 0) {
                if (row_ok) {
                    r0.store(y + rl.off0);
                    r1.store(y + rl.off1);
                }
            } else {
                if (!NB && side == 1) {  // to neighbouring dims: lane l takes dims [16l, 16l + 16)
                    bf16* row = sm.turn[warp] + rr * D;
                    r0.store(row + rl.off0);
                    r1.store(row + rl.off1);
                    __syncwarp();
                    r0.a = *reinterpret_cast<const uint4*>(row + 16 * l);
                    r1.a = *reinterpret_cast<const uint4*>(row + 16 * l + 8);
                    __syncwarp();
                }
                uint32_t word[2], sz;
                quantise16(r0, r1, word, sz);
                if (row_ok) put16<D>(rec, r, l, side == 1, word, sz);
            }
            h += hpw;
            y += hpw * a.y.sh;
            rec += hpw * head_bytes;
        }
    }
    copy_wait<0>();
}

// Eight codes -> eight bf16 values c s + z, one rounding each (s and z twice in their words).
// 128 + c is a bf16 with the code in its low bits, so c comes out exactly; the FMA rounds.
__device__ __forceinline__ uint4 values8(uint32_t word, uint32_t s2, uint32_t z2) {
    uint32_t v[4];  // dims (i, i + 4)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = ((word >> (4 * i)) & 0x000f000fu) | 0x43004300u;
        asm("sub.rn.bf16x2 %0, %0, %1;" : "+r"(v[i]) : "r"(0x43004300u));
        asm("fma.rn.bf16x2 %0, %0, %1, %2;" : "+r"(v[i]) : "r"(s2), "r"(z2));
    }
    return make_uint4(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410),
                      __byte_perm(v[0], v[1], 0x7632), __byte_perm(v[2], v[3], 0x7632));
}

struct ReadArgs {
    const uint8_t* cache;
    const int64_t* slots;
    Heads k, v;
    Span span;
    int64_t pages;
    unsigned* err;
    int tokens, blocks_per_page;
    bool wide;  // 32-byte stores: every row of k and v starts on 32 bytes
};

// Lanes per row D/64: a lane takes 64 dims of K and 64 of V, which are 32 bytes of codes each (K:
// the 16 dims 16 h .. of four groups, two words each; V: neighbours), so it loads six 16-byte
// pieces and writes eight of 32 bytes, whole sectors.  Measured at 32768 tokens of 8 heads of 128
// (floor 26 us): 29.7 us, 92% of the copy rate at 65536; 42 us with 16 dims per lane, ten loads of 2
// to 4 bytes and four times the lanes' instructions.
template <int D>
__global__ void __launch_bounds__(kWarps * 32) kv4_read_kernel(const ReadArgs a) {
    constexpr int LN = D / 64, RPW = 32 / LN;
    const Span sp = a.span;
    const int part = blockIdx.y;
    const int lane = threadIdx.x & 31, q = lane % LN, rr = lane / LN;
    const int hsub = rr & ((1 << sp.log_hpw) - 1), tsub = rr >> sp.log_hpw;
    const int tpw = RPW >> sp.log_hpw;
    const int64_t tok = ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * tpw + tsub;
    if (tok >= a.tokens) return;
    const int64_t slot = __ldg(a.slots + tok);
    if (slot < 0) return;
    if (slot >= a.pages * a.blocks_per_page * kKv4Block) {
        if (part == 0 && q == 0 && hsub == 0) atomicOr(a.err, ERR_INDEX);
        return;
    }
    const int r = (int)(slot & (kKv4Block - 1));
    const int h16 = q & 1, quad = q >> 1;  // K: dims 16 h16 .. of groups 4 quad ..  (D = 64: both h16)
    const int64_t head_bytes = (int64_t)a.blocks_per_page * kv4_record_bytes(D);
    int h = (part * sp.per_part << sp.log_hpw) + hsub;
    const uint8_t* rec = a.cache + kv4_record_of(slot, a.blocks_per_page, sp.heads) * kv4_record_bytes(D) +
                         h * head_bytes;
    bf16* ko = a.k.row<bf16>(0, (int)tok) + h * a.k.sh;
    bf16* vo = a.v.row<bf16>(0, (int)tok) + h * a.v.sh + 64 * q;
    const int h1 = min(sp.heads, (part + 1) * sp.per_part << sp.log_hpw), hpw = 1 << sp.log_hpw;
    // byte offsets of the lane's pieces in a record
    const int k0 = D == 64 ? kv4_k_word(D, r, 0) : kv4_k_word(D, r, 2 * h16 + 16 * quad);
    const int k1 = D == 64 ? k0 + 16 : kv4_k_word(D, r, 2 * h16 + 1 + 16 * quad);
    const int ks = kv4_k_scale(D, r, 4 * quad);
    const int v0 = kv4_v_unit(D, r, 8 / LN * q), vs = kv4_v_scale(D, r & ~1, 2 * q);
    const uint32_t odd = r & 1 ? 0x3232 : 0x1010;  // this token's half of a pair of scales
    for (; h < h1; h += hpw) {
        uint32_t kw[8], vw[8], sk[4], sv[4];
        auto load4 = [&](int at, uint32_t* w) {
            const uint4 x = __ldg(reinterpret_cast<const uint4*>(rec + at));
            w[0] = x.x;
            w[1] = x.y;
            w[2] = x.z;
            w[3] = x.w;
        };
        load4(k0, kw);
        load4(k1, kw + 4);
        if (D == 64) {
            const uint2 x = __ldg(reinterpret_cast<const uint2*>(rec + ks));
            sk[0] = x.x;
            sk[1] = x.y;
        } else {
            load4(ks, sk);
        }
        load4(v0, vw);
        load4(v0 + 16, vw + 4);
        load4(vs, sv);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // D = 64: words (t, j) at 2 t + j; else t = 2 h16 in kw[0 .. 3], 2 h16 + 1 in kw[4 .. 7]
            const int j = D == 64 ? i / 2 : i, half = D == 64 ? i % 2 : h16;
            const uint32_t wa = D == 64 ? kw[4 * (i % 2) + j] : kw[i];
            const uint32_t wb = D == 64 ? kw[4 * (i % 2) + 2 + j] : kw[4 + i];
            const uint32_t s2 = __byte_perm(sk[j], 0, 0x1010), z2 = __byte_perm(sk[j], 0, 0x3232);
            store32(ko + 32 * (4 * quad + j) + 16 * half, values8(wa, s2, z2), values8(wb, s2, z2), a.wide);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t s2 = __byte_perm(sv[2 * (i / 2)], 0, odd);
            const uint32_t z2 = __byte_perm(sv[2 * (i / 2) + 1], 0, odd);
            store32(vo + 16 * i, values8(vw[2 * i], s2, z2), values8(vw[2 * i + 1], s2, z2), a.wide);
        }
        rec += hpw * head_bytes;
        ko += hpw * a.k.sh;
        vo += hpw * a.v.sh;
    }
}

// Shares the append's CTAs out to q, k and v by their work: a unit's chunks (norm and rotation; both
// and the quantiser; the quantiser alone), and one and a half chunks' time for entering it.
void share_ctas(int64_t all, const Span (&sp)[3], const int64_t (&units)[3], int (&grid)[3]) {
    const double factor[3] = {1, 1.8, 1.2};
    double work[3], sum = 0;
    for (int i = 0; i < 3; ++i) {
        work[i] = (double)units[i] * (sp[i].per_part * factor[i] + 1.5);
        sum += work[i];
    }
    for (int i = 0; i < 3; ++i) {
        const int64_t g = std::max<int64_t>(1, (int64_t)((double)all * work[i] / sum + 0.5));
        grid[i] = (int)std::min(g, (units[i] + kWarps - 1) / kWarps);
    }
}

template <int LPR, bool NB>
cudaError_t run_append(const Kv4Append& c, cudaStream_t s) {
    constexpr int RPW = 32 / LPR;
    AppendArgs a{};
    const int heads[3] = {c.heads, c.kv_heads, c.kv_heads};
    const int per = pick_per_part(heads, 3, c.tokens, RPW, c.sms);
    int64_t units[3], gx = 1, sum = 0;
    int gy = 0;
    for (int i = 0; i < 3; ++i) {
        a.x[i] = c.x[i];
        a.span[i] = make_span(heads[i], RPW, per);
        const int64_t g = groups_of(c.tokens, a.span[i], RPW);
        units[i] = g * a.span[i].parts;
        sum += units[i];
        gx = std::max(gx, (g + kWarps - 1) / kWarps);
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
    if (sum < (int64_t)c.sms * 16 * kStreamFrom) {  // 16 warps run on an SM at once
        kv4_append_kernel<LPR, NB><<<dim3((unsigned)gx, gy), kWarps * 32, 0, s>>>(a);
        return cudaGetLastError();
    }
    Launch L{};
    L.sms = c.sms;
    L.grid = (int64_t)c.sms * 16;
    L.smem = sizeof(AppendSmem);
    int64_t all = 0;
    auto kernel = kv4_append_stream_kernel<LPR, NB>;
    cudaError_t e = fit_grid((const void*)kernel, L, kWarps * 32, &all);
    if (e != cudaSuccess) return e;
    share_ctas(all, a.span, units, a.grid);
    kernel<<<a.grid[0] + a.grid[1] + a.grid[2], kWarps * 32, (size_t)L.smem, s>>>(a);
    return cudaGetLastError();
}

template <int D>
cudaError_t run_read(const Kv4Read& c, cudaStream_t s) {
    constexpr int RPW = 32 * 64 / D;
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
    a.wide = true;
    for (const Heads* x : {&c.k, &c.v})
        if ((reinterpret_cast<uintptr_t>(x->p) | (uintptr_t)x->st * 2 | (uintptr_t)x->sh * 2) % 32 != 0)
            a.wide = false;
    const int64_t gx = (groups_of(c.tokens, a.span, RPW) + kWarps - 1) / kWarps;
    kv4_read_kernel<D><<<dim3((unsigned)gx, a.span.parts), kWarps * 32, 0, s>>>(a);
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
        case 64: return run_read<64>(c, s);
        case 128: return run_read<128>(c, s);
        case 256: return run_read<256>(c, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace rmsn
