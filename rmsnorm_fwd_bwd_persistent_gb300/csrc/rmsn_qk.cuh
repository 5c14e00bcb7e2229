// rmsn_qk.cuh -- the row geometry shared by the per-head norm + rotation kernels.
//
// A row is one head of one token: D elements, D a multiple of 16, at most 256.  LPR lanes
// (the power of two >= D/16) share a row, so a warp works on RPW = 32/LPR rows at a time;
// lane l of a row holds 16 elements as two vectors of 8, chosen so that both members of every
// rotated pair are in the same lane and no exchange between lanes is needed:
//   half pairs (i, i + rd/2):  lanes l < rd/16 hold dims [8l, 8l+8) and rd/2 + [8l, 8l+8)
//   neighbours (2i, 2i+1):     dims [16l, 16l+16)
//   the part that is not rotated (dims >= rd): dims [16l, 16l+16), with cos = 1, sin = 0
// In both styles lane l needs the angles [8l, 8l+8) of its token's table row.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "rmsn_device.cuh"

namespace rmsn {

constexpr unsigned ERR_INDEX = 8u;  // a position, slot or page outside its table

// Eight elements as they are in memory.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) {
        a = __ldg(reinterpret_cast<const uint4*>(p));
    }
    __device__ __forceinline__ void clear() { a = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void get(float (&f)[8]) const { Elem<__nv_bfloat16>::unpack(a, f); }
    __device__ __forceinline__ void pairs(f2 (&f)[4]) const { Pairs<__nv_bfloat16>::get(a, f); }
    __device__ __forceinline__ void store(__nv_bfloat16* p) const {
        *reinterpret_cast<uint4*>(p) = a;
    }
};
template <>
struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = __ldg(reinterpret_cast<const float4*>(p));
        b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
    __device__ __forceinline__ void pairs(f2 (&f)[4]) const {
        f[0] = f2_make(a.x, a.y);
        f[1] = f2_make(a.z, a.w);
        f[2] = f2_make(b.x, b.y);
        f[3] = f2_make(b.z, b.w);
    }
};

// A lane's place in its row, and the angles and weights that go with it.
template <bool NEIGHBOURS>
struct RowLane {
    int off0, off1;  // first dims of its two vectors
    bool turns;      // holds rotated dims

    __device__ __forceinline__ void init(int l, int rd) {
        turns = 16 * l < rd;
        if (!NEIGHBOURS && turns) {
            off0 = 8 * l;
            off1 = rd / 2 + 8 * l;
        } else {
            off0 = 16 * l;
            off1 = 16 * l + 8;
        }
    }
};

// Angles of one token: cos and sin of the lane's eight pairs.
struct Angles {
    float c[8], s[8];
    __device__ __forceinline__ void identity() {
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = 1.f, s[i] = 0.f;
    }
    __device__ __forceinline__ void load(const float* cosp, const float* sinp) {
        const float4* p = reinterpret_cast<const float4*>(cosp);
        const float4* q = reinterpret_cast<const float4*>(sinp);
        const float4 c0 = __ldg(p), c1 = __ldg(p + 1), s0 = __ldg(q), s1 = __ldg(q + 1);
        c[0] = c0.x; c[1] = c0.y; c[2] = c0.z; c[3] = c0.w;
        c[4] = c1.x; c[5] = c1.y; c[6] = c1.z; c[7] = c1.w;
        s[0] = s0.x; s[1] = s0.y; s[2] = s0.z; s[3] = s0.w;
        s[4] = s1.x; s[5] = s1.y; s[6] = s1.z; s[7] = s1.w;
    }
};

// Rotates the lane's 16 elements (u: first vector, v: second) by its angles, in place;
// TRANSPOSE rotates back (the gradient's direction).
template <bool NEIGHBOURS, bool TRANSPOSE>
__device__ __forceinline__ void rotate(float (&u)[8], float (&v)[8], const Angles& t) {
    auto turn = [](float& a, float& b, float c, float s) {
        const float x = a, y = b;
        if (TRANSPOSE) {
            a = fmaf(y, s, __fmul_rn(x, c));
            b = __fsub_rn(__fmul_rn(y, c), __fmul_rn(x, s));
        } else {
            a = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
            b = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
        }
    };
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (NEIGHBOURS) {
            if (i < 4)
                turn(u[2 * i], u[2 * i + 1], t.c[i], t.s[i]);
            else
                turn(v[2 * i - 8], v[2 * i - 7], t.c[i], t.s[i]);
        } else {
            turn(u[i], v[i], t.c[i], t.s[i]);
        }
    }
}

// Eight weights as FP32.
__device__ __forceinline__ void load_w8(const void* w, int bf16, int off, float (&f)[8]) {
    if (bf16) {
        Raw8<__nv_bfloat16> r;
        r.load(static_cast<const __nv_bfloat16*>(w) + off);
        r.get(f);
    } else {
        Raw8<float> r;
        r.load(static_cast<const float*>(w) + off);
        r.get(f);
    }
}

// Sum over the LPR lanes of a row (every lane gets the same bits).
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// 1/sqrt(ss/D + eps) for inv_d = 1/D: the hardware's approximation (2^-22.9 relative) and one
// Newton step r + r/2 (1 - m r^2), which leaves about one rounding; the IEEE divide, square root
// and reciprocal are four times the instructions.  A sum of squares beyond FP32 gives 0, as in
// the row kernels.
__device__ __forceinline__ float row_rstd(float ss, float inv_d, float eps) {
    const float m = fmaf(ss, inv_d, eps);
    float r;
    asm("rsqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(m));
    r = fmaf(0.5f * r, fmaf(-(m * r), r, 1.f), r);
    return m > 3.402823466e38f ? 0.f : r;
}

// The same with the rounding of an IEEE square root and an IEEE reciprocal, as the row kernels'
// forward has it: the root and its reciprocal refined together (Goldschmidt's iteration from the
// hardware's approximation), then each by one step from its exact FMA remainder, which rounds
// correctly (Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990).  Ten FMAs and no branches; the intrinsics cost the forward 6%.
__device__ __forceinline__ float row_rstd_exact(float ss, float inv_d, float eps) {
    const float m = __fadd_rn(__fmul_rn(ss, inv_d), eps);
    float r;
    asm("rsqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(m));
    float g = __fmul_rn(m, r), h = 0.5f * r;
    const float e = fmaf(-g, h, 0.5f);
    g = fmaf(g, e, g);
    h = fmaf(h, e, h);
    g = fmaf(fmaf(-g, g, m), h, g);  // the root
    r = h + h;
    r = fmaf(fmaf(-g, r, 1.f), r, r);  // 1 / g
    return m > 3.402823466e38f ? 0.f : r;
}

// One operand of the kernels: the rows of q, k or v in memory.  Strides in elements.
struct Heads {
    void* p;
    int64_t sb, st, sh;
    template <typename T>
    __device__ __forceinline__ T* row(int b, int t) const {
        T* r = static_cast<T*>(p) + t * st;
        return b ? r + b * sb : r;
    }
};

// How a warp's rows lie over tokens and heads: hpw heads (a power of two) of tpw tokens at a
// time, `chunks` such steps for all heads of the tokens, split into `parts` units of work.
struct Span {
    int heads, log_hpw, chunks, per_part, parts;
};

struct Rope {
    const float* cos;
    const float* sin;
    const int64_t* pos;
    int64_t pos_sb, pos_st, rows;
    int rd;
};

// The token of one row of a warp: index, position, and whether its row is worked on.
struct Token {
    int b, t;
    bool ok;
    int64_t pos;
};

__device__ __forceinline__ Token find_token(int tok, int tokens, int T, const Rope& rope,
                                            unsigned* err, bool report) {
    Token k;
    k.ok = tok < tokens;
    const int c = k.ok ? tok : 0;
    k.b = tokens == T ? 0 : c / T;
    k.t = c - k.b * T;
    k.pos = __ldg(rope.pos + k.b * rope.pos_sb + k.t * rope.pos_st);
    if (k.ok && (k.pos < 0 || k.pos >= rope.rows)) {
        if (report) atomicOr(err, ERR_INDEX);
        k.ok = false;
    }
    return k;
}

// Lanes per row for a head of D elements.
inline int lanes_per_row(int D) {
    int n = 1;
    while (16 * n < D) n *= 2;
    return n;
}

// The rows of one side over a warp: as many heads of a token as fit (a power of two), the
// rest of the warp's rows on the next tokens.
inline Span make_span(int heads, int rpw, int per_part) {
    Span s{};
    s.heads = heads;
    while ((2 << s.log_hpw) <= rpw && (1 << s.log_hpw) < heads) ++s.log_hpw;
    s.chunks = (heads + (1 << s.log_hpw) - 1) >> s.log_hpw;
    s.per_part = per_part < s.chunks ? per_part : s.chunks;
    s.parts = (s.chunks + s.per_part - 1) / s.per_part;
    return s;
}

inline int64_t groups_of(int64_t tokens, const Span& s, int rpw) {
    const int tpw = rpw >> s.log_hpw;
    return (tokens + tpw - 1) / tpw;
}

// Chunks per unit of work: the most (8 at first) that still leave about two warps for each
// of an SM's four schedulers.
inline int pick_per_part(const int* heads, int sides, int64_t tokens, int rpw, int sms) {
    int per = 8;
    for (; per > 1; per /= 2) {
        int64_t units = 0;
        for (int i = 0; i < sides; ++i) {
            const Span s = make_span(heads[i], rpw, per);
            units += groups_of(tokens, s, rpw) * s.parts;
        }
        if (units >= (int64_t)sms * 8) break;
    }
    return per;
}

// 16 bytes from global to this lane's own place in shared memory.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Eight elements in shared memory as FP32 pairs.
__device__ __forceinline__ void pairs8(const __nv_bfloat16* p, f2 (&f)[4]) {
    Pairs<__nv_bfloat16>::get(*reinterpret_cast<const uint4*>(p), f);
}
__device__ __forceinline__ void pairs8(const float* p, f2 (&f)[4]) {
    const ulonglong2 a = reinterpret_cast<const ulonglong2*>(p)[0];
    const ulonglong2 b = reinterpret_cast<const ulonglong2*>(p)[1];
    f[0] = a.x;
    f[1] = a.y;
    f[2] = b.x;
    f[3] = b.y;
}

// 32 bytes to memory: at once, or in halves where they start on 16 bytes only.
__device__ __forceinline__ void store32(void* p, const uint4& a, const uint4& b, bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x),
                     "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                     : "memory");
    } else {
        reinterpret_cast<uint4*>(p)[0] = a;
        reinterpret_cast<uint4*>(p)[1] = b;
    }
}

// A lane's two vectors to memory.  Vectors that lie together (neighbouring pairs) and FP32
// vectors are 32 bytes of one lane, stored at once so that whole sectors are written.
template <typename T, bool NEIGHBOURS>
__device__ __forceinline__ void store_row(T* p0, T* p1, const f2 (&u)[4], const f2 (&v)[4], bool wide) {
    if constexpr (sizeof(T) == 2) {
        const uint4 a = Pairs<__nv_bfloat16>::put(u), b = Pairs<__nv_bfloat16>::put(v);
        if (NEIGHBOURS) {
            store32(p0, a, b, wide);
        } else {
            *reinterpret_cast<uint4*>(p0) = a;
            *reinterpret_cast<uint4*>(p1) = b;
        }
    } else {
        auto half = [](f2 x, f2 y) {
            return make_uint4((uint32_t)x, (uint32_t)(x >> 32), (uint32_t)y, (uint32_t)(y >> 32));
        };
        store32(p0, half(u[0], u[1]), half(u[2], u[3]), wide);
        store32(p1, half(v[0], v[1]), half(v[2], v[3]), wide);
    }
}

// rotate() on pairs.  The gradient's direction of half pairs, where a lane's vectors are the
// partners, goes two at a time; the rest one at a time, which keeps the forward's products rounded
// before their sum (the two-element multiply and add are free to be joined) at no cost in time.
template <bool NEIGHBOURS, bool TRANSPOSE>
__device__ __forceinline__ void rotate2(f2 (&u)[4], f2 (&v)[4], const Angles& t) {
    if constexpr (NEIGHBOURS || !TRANSPOSE) {
        float a[8], b[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[2 * i] = f2_lo(u[i]);
            a[2 * i + 1] = f2_hi(u[i]);
            b[2 * i] = f2_lo(v[i]);
            b[2 * i + 1] = f2_hi(v[i]);
        }
        rotate<NEIGHBOURS, TRANSPOSE>(a, b, t);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            u[i] = f2_make(a[2 * i], a[2 * i + 1]);
            v[i] = f2_make(b[2 * i], b[2 * i + 1]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f2 c = f2_make(t.c[2 * i], t.c[2 * i + 1]);
            const f2 s = f2_make(t.s[2 * i], t.s[2 * i + 1]);
            const f2 x = u[i], y = v[i];
            u[i] = fma2(y, s, mul2(x, c));
            v[i] = sub2(mul2(y, c), mul2(x, s));
        }
    }
}

// (x r) w, rotated: the forward of one row's lane.  All forward kernels share it, so that a row
// gets the same bits whichever of them it goes through.
template <bool NEIGHBOURS, int LPR>
__device__ __forceinline__ void norm_rotate(f2 (&u)[4], f2 (&v)[4], const f2 (&w0)[4], const f2 (&w1)[4],
                                            const Angles& ang, float inv_d, float eps) {
    f2 ss2 = 0ull;
#pragma unroll
    for (int i = 0; i < 4; ++i) ss2 = fma2(u[i], u[i], ss2);
#pragma unroll
    for (int i = 0; i < 4; ++i) ss2 = fma2(v[i], v[i], ss2);
    const float r = row_rstd_exact(row_sum<LPR>(f2_lo(ss2) + f2_hi(ss2)), inv_d, eps);
    const f2 r2 = f2_splat(r);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        u[i] = mul2(mul2(u[i], r2), w0[i]);
        v[i] = mul2(mul2(v[i], r2), w1[i]);
    }
    rotate2<NEIGHBOURS, false>(u, v, ang);
}

// The weights beside a lane's two vectors (zero where it has none).
__device__ __forceinline__ void load_weights(const void* w, int bf16, int off0, int off1, bool ok,
                                             f2 (&w0)[4], f2 (&w1)[4]) {
    float f0[8], f1[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f0[i] = f1[i] = 0.f;
    if (ok) {
        load_w8(w, bf16, off0, f0);
        load_w8(w, bf16, off1, f1);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w0[i] = f2_make(f0[2 * i], f0[2 * i + 1]);
        w1[i] = f2_make(f1[2 * i], f1[2 * i + 1]);
    }
}

// A checked call of the norm + rotation (x -> y, or with ws the backward: g, x -> y = dx).
struct QkCall {
    Heads x[2], y[2], g[2];
    const void* w[2];
    float* dw[2];
    int heads[2];
    Rope rope;
    float* ws;
    unsigned* err;
    int64_t tokens, T;
    int D, x_dt, w_dt, sms;
    bool neighbours;
    float eps;
};
constexpr int kQkBwdCtasPerSm = 4;  // the backward's persistent CTAs (its workspace's size)

cudaError_t launch_qk(const QkCall& c, cudaStream_t s);

}  // namespace rmsn
