// rmsn_kv4_attn.cu -- attention of a few query tokens per sequence over the 4-bit paged cache.
//
//   o = softmax(scale q K^T) V,  lse = log sum exp;  K = c s + z per group of 32 dims
//
// What bounds it: the cache is read once (1.25 D bytes per token and head), and every code
// has to reach a matrix instruction as a 16-bit number; with one query token per sequence the
// second takes more issue slots than the first takes memory time, so the work per code is what
// the layout and the arithmetic below keep small.
//
// Mathematics.  The scores are formed transposed, S^T = K q^T, with 16 tokens as the M rows and
// 8 (query token, head) columns of one kv head as N, so no row of the matrix instruction is
// padding when a kv head serves 8 query heads.  A matrix step of 16 dims stays inside one group
// of 32, so the scale and minimum come after the product, in FP32:
//   q . k = sum_j ( s_j (c . q)_j + z_j (sum of q)_j )
// and the codes themselves are the operand: a nibble masked out of its word is the binary16
// subnormal c 2^-24 (or, four bits up, c 2^-20: those dims of q are divided by 16), so one AND
// makes two operands; q is scaled by a power of two to use binary16's range, which is exact for
// its bf16 values down to 2^-17 of the row's largest.  The softmax runs over one pass with a running
// maximum per column that moves only when a score exceeds it by 2^8 (the probabilities of up
// to 256 are harmless in bf16 and FP32), so most blocks need one vote instead of a reduction.
// O^T = V^T P^T takes the probabilities transposed by movmatrix, rounded to bf16, and V as
// bf16 values c s + z (c exact by 128 + c - 128 in bf16, one FMA rounding).  Sums, maxima and
// outputs are FP32.
//
// Work split.  Blocks of 16 tokens of all (sequence, kv head) items form one line of units that
// is cut into equal shares, one per CTA, so ragged batches and single long sequences load all
// SMs alike; a CTA's four warps take the blocks of an item in turn, each streaming its own
// blocks through a ring in shared memory (bulk copies of a whole record), and merge at the
// item's end.  An item that lies in several CTAs leaves partial sums in the workspace, which
// kv4_combine_kernel adds in CTA order: results do not depend on timing.
#include <cfloat>

#include "rmsn_internal.h"
#include "rmsn_kv4.cuh"
#include "rmsn_pipe.cuh"

namespace rmsn {

namespace {

using bf16 = __nv_bfloat16;
constexpr int kWarps = 4;
constexpr int kCtasPerSm = 4;      // at most (sizes the workspace)
constexpr int kMinShare = 8;       // least blocks per CTA: two for each warp

__host__ __device__ constexpr int stages_of(int D) { return D == 64 ? 4 : 3; }

struct Args {
    const bf16* q;
    int64_t q_st, q_sh, out_st, out_sh;
    bf16* out;
    float* lse;
    const uint8_t* cache;
    const int* table;
    int64_t table_stride;
    const int* kv_lens;
    const int* cu_q;
    int64_t* prefix;  // [seqs + 1] first unit of every sequence
    float* part;      // [CTA][2][columns][D]
    float2* part_ml;  // [CTA][2][columns] (maximum, sum)
    unsigned* err;
    uint64_t limit_ns;
    int64_t pages;
    int tokens, seqs, heads, kv_heads, group, table_width, nb;
    float scale_log2;
};

// One sequence's share of the problem.
struct Seq {
    int q0, n, len, blocks, qblocks;
};

template <int QC>
__device__ __forceinline__ Seq seq_of(const Args& a, int b, bool report) {
    Seq s;
    if (a.cu_q) {
        s.q0 = min(max(__ldg(a.cu_q + b), 0), a.tokens);
        s.n = max(min(__ldg(a.cu_q + b + 1), a.tokens) - s.q0, 0);
    } else {
        s.q0 = b;
        s.n = 1;
    }
    const int len = __ldg(a.kv_lens + b);
    const int most = a.table_width * a.nb * kKv4Block;
    if (len > most && report) atomicOr(a.err, ERR_INDEX);
    s.len = min(max(len, 0), most);
    s.blocks = (s.len + kKv4Block - 1) / kKv4Block;
    s.qblocks = (s.n * a.group + QC - 1) / QC;
    return s;
}

__device__ __forceinline__ int64_t share_of(int64_t units, int ctas) {
    const int64_t per = (units + ctas - 1) / ctas;
    return per < kMinShare ? kMinShare : per;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
    return d;
}

// Two codes (bits 0-3 and 16-19 of x, others masked) times s plus z, as bf16x2.
__device__ __forceinline__ uint32_t value2(uint32_t x, uint32_t s2, uint32_t z2) {
    uint32_t v = (x & 0x000f000fu) | 0x43004300u;  // 128 + c in bf16
    asm("sub.rn.bf16x2 %0, %0, %1;" : "+r"(v) : "r"(0x43004300u));
    asm("fma.rn.bf16x2 %0, %0, %1, %2;" : "+r"(v) : "r"(s2), "r"(z2));
    return v;
}

// N 32-bit words from shared memory in the widest loads.
template <int N>
__device__ __forceinline__ void lds_words(const uint8_t* p, uint32_t (&w)[N]) {
    if constexpr (N == 1) {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (N == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        w[0] = v.x;
        w[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const uint4 v = *reinterpret_cast<const uint4*>(p + 4 * i);
            w[i] = v.x;
            w[i + 1] = v.y;
            w[i + 2] = v.z;
            w[i + 3] = v.w;
        }
    }
}


template <int D, int NT>
struct Smem {
    static constexpr int S = stages_of(D);
    static constexpr int QC = 8 * NT;
    static constexpr int OS = D + 4;  // padded row of the merge buffer
    uint8_t ring[kWarps][S][20 * D];
    float o[kWarps][QC][OS];
    float m[kWarps][QC], l[kWarps][QC];
    uint64_t full[kWarps][S];
    int64_t sum[kWarps], found;
    int found_seq;
};

// The columns' state of one warp over one item.
template <int D, int NT>
struct Warp {
    static constexpr int NG = D / 32;  // groups, and K words per lane and token
    static constexpr int VW = D / 64;  // V words per lane and token
    static constexpr int MT = D / 16;  // M tiles of O^T
    uint32_t qf[NT][NG][4];            // q as binary16 pairs, column g
    float qz[NT][NG][2];               // (sum of q)_j, columns 2t and 2t + 1, log2 units
    float f[NT][2];                    // factor of the code products, log2 units
    int lim[NT][2];                    // tokens that the column sees
    float o[NT][MT][4];
    float m[NT][2], l[NT][2];

    // Loads the item's query rows and resets the sums.
    __device__ __forceinline__ void begin(const Args& a, const Seq& s, int qb, int h, int lane) {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int col = (qb * NT + nt) * 8 + g;
            float x[NG][8];
            float amax = 0.f;
            const bool ok = col < s.n * a.group;
            const int i = ok ? col / a.group : 0;
            const bf16* row = a.q + (int64_t)(s.q0 + i) * a.q_st +
                              (int64_t)(h * a.group + (ok ? col - i * a.group : 0)) * a.q_sh;
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                Raw8<bf16> r;
                r.clear();
                if (ok) r.load(row + 32 * j + 8 * t);
                r.get(x[j]);
#pragma unroll
                for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(x[j][e]));
            }
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            int ex = 0;  // the row's largest becomes 2^14 .. 2^15
            if (amax > 0.f && amax <= FLT_MAX) {
                frexpf(amax, &ex);
                ex -= 15;
            }
            float z[NG];
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                z[j] = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) z[j] += x[j][e];
                z[j] += __shfl_xor_sync(0xffffffffu, z[j], 1);
                z[j] += __shfl_xor_sync(0xffffffffu, z[j], 2);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int sh = e & 1 ? -ex - 4 : -ex;
                    const __half2 p = __floats2half2_rn(ldexpf(x[j][e], sh), ldexpf(x[j][e + 4], sh));
                    qf[nt][j][e] = *reinterpret_cast<const uint32_t*>(&p);
                }
            }
            const float fac = ldexpf(a.scale_log2, ex + 24);
#pragma unroll
            for (int c = 0; c < 2; ++c) {  // from the lanes of column 2t + c
                const int src = 8 * t + 4 * c;
                f[nt][c] = __shfl_sync(0xffffffffu, fac, src);
#pragma unroll
                for (int j = 0; j < NG; ++j)
                    qz[nt][j][c] = __shfl_sync(0xffffffffu, z[j], src) * a.scale_log2;
                const int cc = (qb * NT + nt) * 8 + 2 * t + c;
                lim[nt][c] = cc < s.n * a.group ? s.len - s.n + 1 + cc / a.group : 0;
                m[nt][c] = -FLT_MAX;
                l[nt][c] = 0.f;
            }
#pragma unroll
            for (int i2 = 0; i2 < MT; ++i2)
#pragma unroll
                for (int c = 0; c < 4; ++c) o[nt][i2][c] = 0.f;
        }
    }

    // Adds the 16 tokens of one record; `full`: every column sees all of them.
    __device__ __forceinline__ void block(const uint8_t* rec, int tok0, int len, bool full,
                                          int lane) {
        const int g = lane >> 2, t = lane & 3;
        float sc[NT][4], zs[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) sc[nt][c] = zs[nt][c] = 0.f;
        {
            uint32_t k0[NG], k1[NG], s0[NG], s1[NG];
            if constexpr (D == 256) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    uint32_t w[4];
                    lds_words(rec + kv4_k_word(D, g, t + 16 * u), w);
#pragma unroll
                    for (int i = 0; i < 4; ++i) k0[(4 * u + i) % NG] = w[i];
                    lds_words(rec + kv4_k_word(D, g + 8, t + 16 * u), w);
#pragma unroll
                    for (int i = 0; i < 4; ++i) k1[(4 * u + i) % NG] = w[i];
                }
            } else {
                lds_words(rec + kv4_k_word(D, g, t), k0);
                lds_words(rec + kv4_k_word(D, g + 8, t), k1);
            }
            lds_words(rec + kv4_k_scale(D, g, 0), s0);
            lds_words(rec + kv4_k_scale(D, g + 8, 0), s1);
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                const uint32_t h0 = k0[j] >> 8, h1 = k1[j] >> 8;
                const uint32_t lo = 0x000f000fu, up = 0x00f000f0u;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float d[4] = {0.f, 0.f, 0.f, 0.f};
                    mma_f16(d, k0[j] & lo, k1[j] & lo, k0[j] & up, k1[j] & up, qf[nt][j][0],
                            qf[nt][j][1]);
                    mma_f16(d, h0 & lo, h1 & lo, h0 & up, h1 & up, qf[nt][j][2], qf[nt][j][3]);
                    sc[nt][0] = fmaf(bf16_lo(s0[j]), d[0], sc[nt][0]);
                    sc[nt][1] = fmaf(bf16_lo(s0[j]), d[1], sc[nt][1]);
                    sc[nt][2] = fmaf(bf16_lo(s1[j]), d[2], sc[nt][2]);
                    sc[nt][3] = fmaf(bf16_lo(s1[j]), d[3], sc[nt][3]);
                    zs[nt][0] = fmaf(bf16_hi(s0[j]), qz[nt][j][0], zs[nt][0]);
                    zs[nt][1] = fmaf(bf16_hi(s0[j]), qz[nt][j][1], zs[nt][1]);
                    zs[nt][2] = fmaf(bf16_hi(s1[j]), qz[nt][j][0], zs[nt][2]);
                    zs[nt][3] = fmaf(bf16_hi(s1[j]), qz[nt][j][1], zs[nt][3]);
                }
            }
        }
        bool up = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                float v = fmaf(sc[nt][c], f[nt][c & 1], zs[nt][c]);
                if (!full && tok0 + g + 8 * (c >> 1) >= lim[nt][c & 1])
                    v = -__int_as_float(0x7f800000);
                sc[nt][c] = v;
                up |= v > m[nt][c & 1] + 8.f;
            }
        if (__any_sync(0xffffffffu, up)) {  // move the maxima, rescale the sums
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float v = fmaxf(sc[nt][c], sc[nt][c + 2]);
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                    v = fmaxf(v, m[nt][c]);
                    const float r = ex2(m[nt][c] - v);
                    m[nt][c] = v;
                    l[nt][c] *= r;
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        o[nt][i][c] *= r;
                        o[nt][i][c + 2] *= r;
                    }
                }
        }
        uint32_t b0[NT], b1[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float p[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) p[c] = ex2(sc[nt][c] - m[nt][c & 1]);
            l[nt][0] += p[0] + p[2];
            l[nt][1] += p[1] + p[3];
            b0[nt] = transpose8x8(pack_bf16x2(p[0], p[1]));
            b1[nt] = transpose8x8(pack_bf16x2(p[2], p[3]));
        }
        // V of tokens 2t, 2t+1 (a) and 2t+8, 2t+9 (b), dims [g D/8, (g+1) D/8)
        constexpr int J = 256 / D;  // lanes g per group
        uint2 sa = *reinterpret_cast<const uint2*>(rec + kv4_v_scale(D, 2 * t, g / J));
        uint2 sb = *reinterpret_cast<const uint2*>(rec + kv4_v_scale(D, 2 * t + 8, g / J));
        bool odd = false;
        if (!full) {
            // tokens behind the last are not read; what a token that only some columns see
            // holds must not reach the others if it is not finite
            auto keep = [&](uint2& v, int r) {
                const uint32_t k = (tok0 + r < len ? 0xffffu : 0u) |
                                   (tok0 + r + 1 < len ? 0xffff0000u : 0u);
                v.x &= k;
                v.y &= k;
                uint32_t drop = 0u;
                if (((v.x & 0x7f80u) == 0x7f80u) || ((v.y & 0x7f80u) == 0x7f80u)) drop |= 0xffffu;
                if (((v.x & 0x7f800000u) == 0x7f800000u) || ((v.y & 0x7f800000u) == 0x7f800000u))
                    drop |= 0xffff0000u;
                odd |= drop != 0u;
                v.x &= ~drop;
                v.y &= ~drop;
            };
            keep(sa, 2 * t);
            keep(sb, 2 * t + 8);
        }
        uint32_t w0[VW], w1[VW], w8[VW], w9[VW];
        lds_words(rec + kv4_v_unit(D, 2 * t, g), w0);
        lds_words(rec + kv4_v_unit(D, 2 * t + 1, g), w1);
        lds_words(rec + kv4_v_unit(D, 2 * t + 8, g), w8);
        lds_words(rec + kv4_v_unit(D, 2 * t + 9, g), w9);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int w = i / 4, half = i / 2 % 2;
            const uint32_t pa = __byte_perm(w0[w], w1[w], half ? 0x7632 : 0x5410);
            const uint32_t pb = __byte_perm(w8[w], w9[w], half ? 0x7632 : 0x5410);
            const int sh = 8 * (i & 1);
            const uint32_t a0 = value2(pa >> sh, sa.x, sa.y);
            const uint32_t a1 = value2(pa >> (sh + 4), sa.x, sa.y);
            const uint32_t a2 = value2(pb >> sh, sb.x, sb.y);
            const uint32_t a3 = value2(pb >> (sh + 4), sb.x, sb.y);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_bf16(o[nt][i], a0, a1, a2, a3, b0[nt], b1[nt]);
        }
        if (__any_sync(0xffffffffu, odd)) not_finite(rec, tok0, len, g);
    }

    // The columns that see a token whose V is not finite become NaN in that group's dims.
    __device__ __forceinline__ void not_finite(const uint8_t* rec, int tok0, int len, int g) {
        for (int r = 0; r < kKv4Block && tok0 + r < len; ++r) {
            const uint16_t* p =
                reinterpret_cast<const uint16_t*>(rec + kv4_v_scale(D, r, g / (256 / D)));
            if ((p[0] & 0x7f80) != 0x7f80 && (p[2] & 0x7f80) != 0x7f80) continue;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    if (tok0 + r < lim[nt][c])
#pragma unroll
                        for (int i = 0; i < MT; ++i) {
                            o[nt][i][c] = __int_as_float(0x7fffffff);
                            o[nt][i][c + 2] = __int_as_float(0x7fffffff);
                        }
        }
    }
};

template <int D, int NT>
__global__ void __launch_bounds__(kWarps * 32) kv4_attention_kernel(const Args a) {
    using Sm = Smem<D, NT>;
    constexpr int S = Sm::S, QC = Sm::QC;
    constexpr uint32_t kRec = 20 * D;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    Sm& sm = *reinterpret_cast<Sm*>(smem_raw);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int ctas = gridDim.x;

    if (threadIdx.x == 0) {
        for (int w = 0; w < kWarps; ++w)
            for (int s = 0; s < S; ++s) mbar_init(&sm.full[w][s], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }

    // All units, then the sequence that holds this CTA's first one.
    auto units_of = [&](int b, bool report) -> int64_t {
        if (b >= a.seqs) return 0;
        const Seq s = seq_of<QC>(a, b, report);
        return (int64_t)s.blocks * s.qblocks * a.kv_heads;
    };
    int64_t sum = 0;
    for (int b = threadIdx.x; b < a.seqs; b += kWarps * 32) sum += units_of(b, blockIdx.x == 0);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) sm.sum[warp] = sum;
    __syncthreads();
    const int64_t total = sm.sum[0] + sm.sum[1] + sm.sum[2] + sm.sum[3];
    const int64_t per = share_of(total, ctas);
    const int64_t begin = blockIdx.x * per, end = min(begin + per, total);
    int64_t before = 0;
    for (int b0 = 0; b0 < a.seqs; b0 += kWarps * 32) {
        const int b = b0 + threadIdx.x;
        const int64_t mine = units_of(b, false);
        int64_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        __syncthreads();
        if (lane == 31) sm.sum[warp] = incl;
        __syncthreads();
        int64_t excl = before + incl - mine;
        for (int w = 0; w < warp; ++w) excl += sm.sum[w];
        if (blockIdx.x == 0 && b < a.seqs) a.prefix[b] = excl;
        if (begin >= excl && begin < excl + mine) {
            sm.found_seq = b;
            sm.found = excl;
        }
        before += sm.sum[0] + sm.sum[1] + sm.sum[2] + sm.sum[3];
        if (blockIdx.x != 0 && before > begin) break;  // the same for the whole CTA
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) a.prefix[a.seqs] = total;
    __syncthreads();
    if (begin >= end) return;

    int b = sm.found_seq;
    int64_t seq_first = sm.found;
    Seq s = seq_of<QC>(a, b, false);
    uint32_t phase = 0u, pending = 0u;  // per stage: parity waited for next, copy in flight
    bool dead = false;
    Warp<D, NT> st;

    for (int64_t u = begin; u < end;) {
        while (u >= seq_first + (int64_t)s.blocks * s.qblocks * a.kv_heads) {
            seq_first += (int64_t)s.blocks * s.qblocks * a.kv_heads;
            s = seq_of<QC>(a, ++b, false);  // u < total, so a sequence with work follows
        }
        const int item = (int)((u - seq_first) / s.blocks);
        const int64_t item_first = seq_first + (int64_t)item * s.blocks;
        const int k0 = (int)(u - item_first);
        const int k1 = (int)min((int64_t)s.blocks, end - item_first);
        const int qb = item / a.kv_heads, h = item - qb * a.kv_heads;
        // every column sees the tokens before this
        const int safe = s.len - s.n + 1 + qb * QC / a.group;

        // record of this warp's x-th block (lane by lane); -1: page outside the cache
        auto record = [&](int x) -> int {
            const int kb = k0 + warp + x * kWarps;
            if (kb >= k1) return -1;
            const int p = kb / a.nb;
            const int page = __ldg(a.table + b * a.table_stride + p);
            if (page < 0 || page >= a.pages) {
                atomicOr(a.err, ERR_INDEX);
                return -1;
            }
            return (page * a.kv_heads + h) * a.nb + (kb - p * a.nb);
        };
        auto issue = [&](int stage, int rec) {
            if (rec < 0) return;
            pending |= 1u << stage;
            if (lane == 0) {
                mbar_arrive_expect_tx(&sm.full[warp][stage], kRec);
                bulk_load(sm.ring[warp][stage], a.cache + (int64_t)rec * kRec, kRec,
                          &sm.full[warp][stage]);
            }
        };
        const int n = dead ? 0 : max(0, (k1 - k0 - warp + kWarps - 1) / kWarps);
        int now = record(lane), next = record(32 + lane);
        for (int i = 0; i < S && i < n; ++i) issue(i, __shfl_sync(0xffffffffu, now, i));
        st.begin(a, s, qb, h, lane);
        int stage = 0;
        for (int i = 0; i < n; ++i) {
            const int rec = __shfl_sync(0xffffffffu, now, i & 31);
            if (rec >= 0) {
                const bool landed = mbar_wait(&sm.full[warp][stage], (phase >> stage) & 1u,
                                              a.limit_ns);
                if (!__all_sync(0xffffffffu, landed)) {
                    if (lane == 0) atomicOr(a.err, ERR_WAIT_FULL);
                    dead = true;
                    break;
                }
                phase ^= 1u << stage;
                pending &= ~(1u << stage);
                const int tok0 = (k0 + warp + i * kWarps) * kKv4Block;
                st.block(sm.ring[warp][stage], tok0, s.len, tok0 + kKv4Block <= safe, lane);
                __syncwarp();
            }
            const int ahead = i + S;
            const int rn = __shfl_sync(0xffffffffu, (ahead >> 5) == (i >> 5) ? now : next,
                                       ahead & 31);
            if (ahead < n) issue(stage, rn);
            if ((i & 31) == 31) {
                now = next;
                next = record(i + 33 + lane);
            }
            stage = stage + 1 == S ? 0 : stage + 1;
        }

        // merge the warps
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float l = st.l[nt][c];
                l += __shfl_xor_sync(0xffffffffu, l, 4);
                l += __shfl_xor_sync(0xffffffffu, l, 8);
                l += __shfl_xor_sync(0xffffffffu, l, 16);
                const int col = nt * 8 + 2 * t + c;
                if (g == 0) {
                    sm.m[warp][col] = st.m[nt][c];
                    sm.l[warp][col] = l;
                }
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
                    *reinterpret_cast<float2*>(&sm.o[warp][col][g * (D / 8) + 2 * i]) =
                        make_float2(st.o[nt][i][c], st.o[nt][i][c + 2]);
            }
        }
        __syncthreads();
        const bool whole = k0 == 0 && k1 == s.blocks;
        const int slot = item_first <= begin ? 0 : 1;
        for (int x = threadIdx.x; x < QC * D / 4; x += kWarps * 32) {
            const int col = x / (D / 4), d = x % (D / 4) * 4;
            const int idx = qb * QC + col;
            if (idx >= s.n * a.group) continue;
            float m = sm.m[0][col];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) m = fmaxf(m, sm.m[w][col]);
            float l = 0.f;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float e = ex2(sm.m[w][col] - m);
                const float4 o = *reinterpret_cast<const float4*>(&sm.o[w][col][d]);
                l = fmaf(e, sm.l[w][col], l);
                v.x = fmaf(e, o.x, v.x);
                v.y = fmaf(e, o.y, v.y);
                v.z = fmaf(e, o.z, v.z);
                v.w = fmaf(e, o.w, v.w);
            }
            if (whole) {
                const float inv = l == 0.f ? 0.f : __frcp_rn(l);
                const int i = idx / a.group, hq = h * a.group + idx - i * a.group;
                const uint2 r = make_uint2(pack_bf16x2(v.x * inv, v.y * inv),
                                           pack_bf16x2(v.z * inv, v.w * inv));
                *reinterpret_cast<uint2*>(a.out + (int64_t)(s.q0 + i) * a.out_st +
                                          (int64_t)hq * a.out_sh + d) = r;
                if (d == 0 && a.lse)
                    a.lse[(int64_t)(s.q0 + i) * a.heads + hq] =
                        l == 0.f ? -__int_as_float(0x7f800000)
                                 : (m + log2f(l)) * 0.693147180559945309f;
            } else {
                const int64_t at = ((int64_t)blockIdx.x * 2 + slot) * QC + col;
                *reinterpret_cast<float4*>(a.part + at * D + d) = v;
                if (d == 0) a.part_ml[at] = make_float2(m, l);
            }
        }
        __syncthreads();
        u = item_first + k1;
    }
    // after a wait that ran out: the copies still in flight must land before the CTA ends
    for (int i = 0; i < S; ++i)
        if ((pending >> i) & 1u)
            if (!mbar_wait(&sm.full[warp][i], (phase >> i) & 1u, a.limit_ns) && lane == 0)
                atomicOr(a.err, ERR_WAIT_DRAIN);
}

// Rows (query token blockIdx.x, head blockIdx.y) whose item lies in several CTAs, or has no
// tokens at all.  D/4 lanes hold the row; the 512/D groups of lanes take the CTAs' partial sums
// in turn and are merged in order.
template <int D, int NT>
__global__ void __launch_bounds__(128) kv4_combine_kernel(const Args a, int ctas) {
    constexpr int QC = 8 * NT, LN = D / 4, GR = 128 / LN;
    __shared__ float4 so[GR][LN];
    __shared__ float smx[GR], sl[GR];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int row = blockIdx.x, hq = blockIdx.y, h = hq / a.group;
    int b = row;
    if (a.cu_q) {  // the last sequence that starts at or before the row
        int lo = 0, hi = a.seqs;
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (__ldg(a.cu_q + mid) <= row) lo = mid;
            else hi = mid;
        }
        b = lo;
    }
    if (b >= a.seqs) return;
    const Seq s = seq_of<QC>(a, b, false);
    if (row < s.q0 || row >= s.q0 + s.n) return;
    const int idx = (row - s.q0) * a.group + hq - h * a.group;
    const int qb = idx / QC, col = idx - qb * QC;
    const int ln = threadIdx.x % LN, gr = threadIdx.x / LN;
    bf16* out = a.out + (int64_t)row * a.out_st + (int64_t)hq * a.out_sh + 4 * ln;
    if (s.blocks == 0) {
        if (gr == 0) *reinterpret_cast<uint2*>(out) = make_uint2(0u, 0u);
        if (threadIdx.x == 0 && a.lse)
            a.lse[(int64_t)row * a.heads + hq] = -__int_as_float(0x7f800000);
        return;
    }
    const int64_t per = share_of(a.prefix[a.seqs], ctas);
    const int64_t u0 = a.prefix[b] + ((int64_t)qb * a.kv_heads + h) * s.blocks;
    const int c0 = (int)(u0 / per), c1 = (int)((u0 + s.blocks - 1) / per);
    if (c0 == c1) return;
    float m = -FLT_MAX, l = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = c0 + gr; c <= c1; c += GR) {
        const int slot = u0 <= c * per ? 0 : 1;
        const int64_t at = ((int64_t)c * 2 + slot) * QC + col;
        const float2 ml = __ldcg(a.part_ml + at);
        const float4 o = __ldcg(reinterpret_cast<const float4*>(a.part + at * D) + ln);
        const float mn = fmaxf(m, ml.x);
        const float e0 = ex2(m - mn), e1 = ex2(ml.x - mn);
        m = mn;
        l = fmaf(e1, ml.y, e0 * l);
        v.x = fmaf(e1, o.x, e0 * v.x);
        v.y = fmaf(e1, o.y, e0 * v.y);
        v.z = fmaf(e1, o.z, e0 * v.z);
        v.w = fmaf(e1, o.w, e0 * v.w);
    }
    so[gr][ln] = v;
    if (ln == 0) {
        smx[gr] = m;
        sl[gr] = l;
    }
    __syncthreads();
    if (gr != 0) return;
#pragma unroll
    for (int k = 1; k < GR; ++k) m = fmaxf(m, smx[k]);
    l = 0.f;
    v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < GR; ++k) {
        const float e = ex2(smx[k] - m);
        const float4 o = so[k][ln];
        l = fmaf(e, sl[k], l);
        v.x = fmaf(e, o.x, v.x);
        v.y = fmaf(e, o.y, v.y);
        v.z = fmaf(e, o.z, v.z);
        v.w = fmaf(e, o.w, v.w);
    }
    const float inv = l == 0.f ? 0.f : __frcp_rn(l);
    *reinterpret_cast<uint2*>(out) =
        make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
    if (ln == 0 && a.lse)
        a.lse[(int64_t)row * a.heads + hq] = l == 0.f ? -__int_as_float(0x7f800000)
                                                       : (m + log2f(l)) * 0.693147180559945309f;
}

int64_t prefix_bytes(int seqs) { return ((int64_t)(seqs + 1) * 8 + 255) / 256 * 256; }

// Columns (a multiple of 8) of one item for heads of D: what the registers hold.
int most_tiles(int D) { return D == 64 ? 4 : D == 128 ? 2 : 1; }

template <int D, int NT>
cudaError_t run(const Kv4Attention& c, cudaStream_t s) {
    Args a{};
    a.q = static_cast<const bf16*>(c.q);
    a.q_st = c.q_st;
    a.q_sh = c.q_sh;
    a.out_st = c.out_st;
    a.out_sh = c.out_sh;
    a.out = static_cast<bf16*>(c.out);
    a.lse = c.lse;
    a.cache = c.cache;
    a.table = c.page_table;
    a.table_stride = c.table_stride;
    a.kv_lens = c.kv_lens;
    a.cu_q = c.cu_q;
    a.err = c.err;
    a.limit_ns = c.limit_ns;
    a.pages = c.pages;
    a.tokens = c.tokens;
    a.seqs = c.seqs;
    a.heads = c.heads;
    a.kv_heads = c.kv_heads;
    a.group = c.heads / c.kv_heads;
    a.table_width = c.table_width;
    a.nb = c.blocks_per_page;
    a.scale_log2 = c.scale * 1.44269504088896340736f;

    Launch L{};
    L.sms = c.sms;
    L.grid = (int64_t)c.sms * kCtasPerSm;
    L.smem = sizeof(Smem<D, NT>);
    int64_t grid = 0;
    auto k = kv4_attention_kernel<D, NT>;
    cudaError_t e = fit_grid((const void*)k, L, kWarps * 32, &grid);
    if (e != cudaSuccess) return e;
    uint8_t* ws = static_cast<uint8_t*>(c.ws);
    a.prefix = reinterpret_cast<int64_t*>(ws);
    a.part = reinterpret_cast<float*>(ws + prefix_bytes(c.seqs));
    a.part_ml = reinterpret_cast<float2*>(a.part + grid * 2 * 8 * NT * D);
    k<<<(unsigned)grid, kWarps * 32, (size_t)L.smem, s>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;

    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)c.tokens, (unsigned)c.heads);
    cfg.blockDim = dim3(128);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv4_combine_kernel<D, NT>, (const Args)a, (int)grid);
}

}  // namespace

int64_t kv4_attention_workspace(int seqs, int D, int sms) {
    const int64_t cols = 8 * most_tiles(D);
    return prefix_bytes(seqs) + (int64_t)sms * kCtasPerSm * 2 * cols * (D + 2) * 4;
}

cudaError_t launch_kv4_attention(const Kv4Attention& c, cudaStream_t s) {
    // the fewest column tiles that hold the queries of one item
    const int64_t cols = (int64_t)c.max_q * (c.heads / c.kv_heads);
    switch (c.D) {
        case 64:
            return cols <= 8 ? run<64, 1>(c, s) : cols <= 16 ? run<64, 2>(c, s) : run<64, 4>(c, s);
        case 128: return cols <= 8 ? run<128, 1>(c, s) : run<128, 2>(c, s);
        case 256: return run<256, 1>(c, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace rmsn
