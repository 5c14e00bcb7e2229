// rmsn_kv4_attn.cu -- attention of a few query tokens per sequence over the 4-bit paged cache.
//
//   o = softmax(scale q K^T) V,  lse = log sum exp;  K = c s + z per group of 32 dims
//
// What bounds it: the cache is read once (1.25 D bytes per token and head), and every code
// has to reach a matrix instruction as a 16-bit number.  The logic pipe that takes codes out of
// their words issues every other cycle, so the work per code is what the layout and the
// arithmetic below keep small.
//
// Scores.  They are formed transposed, S^T = K q^T, with 16 tokens as the M rows and 8 (query
// token, head) columns of one kv head as N, so no row of the matrix instruction is padding when
// a kv head serves 8 query heads.  A matrix step of 16 dims stays inside one group of 32, so the
// scale comes after the product, in FP32, and the minima are a product of their own:
//   q . k = sum_j s_j (c . q)_j + sum_j z_j (sum of q)_j
// The codes themselves are the operand: a nibble masked out of its word is the binary16
// subnormal c 2^-24 (or, four bits up, c 2^-20: those dims of q are divided by 16), so one AND
// makes two operands.  q is scaled by a power of two to use binary16's range, which is exact for
// its bf16 values down to 2^-17 of the row's largest.  The sums of q enter as three bf16 terms
// (24 bits) against the bf16 minima as they lie in the cache.
//
// Softmax.  One pass with a running reference per column, which moves only when a score exceeds
// it by 2^8, so most blocks need one vote instead of a reduction.
//
// Values.  O^T = V^T P^T takes the probabilities (binary16, at most 2^8) transposed by
// movmatrix, and V as binary16 values c s + z by one FMA on the masked codes.  binary16 keeps 11
// bits where bf16 keeps 8 (with bf16 the result was 2.8e-3 off instead of 1.7e-3, of which 1.7e-3
// is the output's own rounding); its range is given by a running power of two per group, 2^k,
// that rises when a scale or minimum needs it.  Sums, references and outputs are FP32.
//
// Work split.  Units of 32 tokens of all (sequence, kv head) items form one line, each item
// with kItemCost places before its units for what entering and merging it costs; the line is cut
// into equal shares, one per CTA, so ragged batches and single long sequences load all SMs
// alike.  (Without those places CTAs that got many short items were late: 64 sequences of up to
// 500 tokens took 35 us, 16 of up to 2000, the same tokens, 16.)  A CTA's four warps take the
// units of an item in turn, each streaming its own through a ring in shared memory (bulk copies of
// whole records), and merge at the item's end, while the next item's first units are copied.  An
// item that lies in several CTAs leaves partial sums in the workspace, which kv4_combine_kernel
// adds in CTA order: results do not depend on timing.
// Where no sequence is longer than 512 tokens no item is split, and the combine has nothing to do;
// it is not launched where the page table holds no more than that.  Split and whole: one sequence
// of 16 tokens 8.7 and 6.0 us, 64 of up to 100 11.6 and 8.6, 300 of up to 500 60 and 51, but 64 of
// up to 1000 23.0 and 23.3, of up to 2000 29.9 and 37.4.  Where such items are many, each is one
// warp's.
//
// Measured on GB300, 32 + 8 heads of 128, replayed from a graph: one sequence of 131072 tokens
// 40.7 us (floor 24.7), 64 sequences of 500 to 16000 122 us (floor 100); longer caches add 93% of
// the copy rate.  What is left of a call is 8 to 11 us for its launches, the first copies, the merges
// and the combine; while it streams, 57% of the issue slots and 53% of the logic pipe are in use
// and the matrix pipe is at 23%.  Tried and not kept: units split finer at the ends of shares, one
// CTA per SM (drafts 22 -> 37 us), a dependent launch announced before the end (no change).
#include <algorithm>
#include <cfloat>

#include "rmsn_internal.h"
#include "rmsn_kv4.cuh"
#include "rmsn_pipe.cuh"

namespace rmsn {

namespace {

using bf16 = __nv_bfloat16;
constexpr int kWarps = 4;
constexpr int kUnit = 2 * kKv4Block;  // tokens per unit of work
constexpr int kMinShare = kWarps;  // least share of a CTA: a unit for each warp
constexpr int kItemCost = 8;  // what entering and merging an item costs, in units
constexpr int kWholeUnits = 16;  // no item is split where no sequence is longer
constexpr int kSoloUnits = 4;    // short enough for a warp to each item as soon as every CTA has one

// CTAs per SM that the registers are divided among, and ring stages of one unit per warp (two are
// 160 KiB in flight per SM at D = 128 and 256 with four CTAs).
__host__ __device__ constexpr int ctas_of(int D, int NT) {
    return D == 256 || NT >= 3 ? 2 : NT == 2 ? 3 : 4;
}
__host__ __device__ constexpr int stages_of(int D, int NT) {
    return D == 64 ? 4 : D == 128 && NT >= 3 ? 3 : 2;
}
// Whether a lane's fragments of q lie in shared memory (each lane's own place, behind its warp's
// ring) instead of registers.
__host__ __device__ constexpr bool q_in_smem(int D, int NT) { return NT * D > 256; }

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
    int64_t* prefix;  // [seqs + 1] first place of every sequence
    float* part;      // [CTA][2][columns][D]
    float2* part_ml;  // [CTA][2][columns] (maximum, sum)
    unsigned* err;
    uint64_t limit_ns;
    int64_t pages;
    int tokens, seqs, heads, kv_heads, group, table_width, nb;
    uint64_t group_inv;  // 2^64 / group, rounded up
    float scale_log2;
    // n / group, 0 <= n < 2^31 (exact: the inverse is off by less than group / 2^64)
    __device__ __forceinline__ int over_group(int n) const {
        return group == 1 ? n : (int)__umul64hi((uint64_t)n, group_inv);
    }
};

// One sequence's share of the problem.
struct Seq {
    int q0, n, len, units, qblocks;
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
    s.units = (s.len + kUnit - 1) / kUnit;
    s.qblocks = (s.n * a.group + QC - 1) / QC;
    return s;
}

// Places of one sequence's items on the line, and places per CTA.  Where no item is split
// (`whole`), each has one place, those without tokens too.
__device__ __forceinline__ int64_t places_of(const Seq& s, int kv_heads, bool whole) {
    const int64_t items = (int64_t)s.qblocks * kv_heads;
    return whole ? items : s.units ? (s.units + kItemCost) * items : 0;
}
__device__ __forceinline__ int64_t share_of(int64_t places, int ctas, int least) {
    const int64_t up = places + ctas - 1;
    const int64_t per = up >> 32 ? up / ctas : (int64_t)((uint32_t)up / (uint32_t)ctas);
    return per < least ? least : per;
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

// a b + c in binary16, two at a time.
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t pack_f16x2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// 2^e for e in [-126, 127], limited to that range
__device__ __forceinline__ float pow2(int e) {
    return __int_as_float((min(max(e, -126), 127) + 127) << 23);
}
// exponent e of a finite v > 0 with v < 2^e; -126 for 0 and for what is not finite
__device__ __forceinline__ int exponent(float v) {
    const int e = (__float_as_int(v) >> 23) & 255;
    return e == 255 ? -126 : e - 126;
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


// A CTA's piece of an item: units [k0, k1) of a (query block, kv head) of a sequence.
struct Piece {
    Seq s;
    int b, qb, h, k0, k1;
    int64_t seq_first, u;  // first place of the sequence; first place behind the item
};

// Shared memory of a CTA.  A warp's sums at the end of an item take the place of the last stages
// of its own ring, which is empty then, and of its q; the first P stages are already filled for the
// next item meanwhile.  Dims are in the order of the fragments (dim_of), which keeps the stores free
// of bank conflicts.
template <int D, int NT>
struct Smem {
    static constexpr int S = stages_of(D, NT);
    static constexpr int QC = 8 * NT;
    static constexpr int OS = D + 4;           // padded row of the sums
    static constexpr int kStage = 2 * 20 * D;  // bytes
    static constexpr int kQ = q_in_smem(D, NT) ? NT * (D / 32) * 512 : 0;
    static constexpr int kRoom = S * kStage + kQ;  // of a warp: its ring and its fragments of q
    static constexpr int P = (kRoom - QC * OS * 4) / kStage;
    static_assert(kRoom >= QC * OS * 4, "the sums fit");
    uint8_t room[kWarps][kRoom];
    float m[kWarps][QC], l[kWarps][QC];
    uint64_t full[kWarps][S];
    Piece piece[kWarps];
    __device__ __forceinline__ float* sums(int w, int col) {
        return reinterpret_cast<float*>(room[w] + P * kStage) + col * OS;
    }
};

// First of the two dims in the n-th pair of a row of sums: pairs run over g, then over the
// dims of a lane.
template <int D>
__device__ __forceinline__ int dim_of(int n) {
    return (n & 7) * (D / 8) + 2 * (n >> 3);
}

// Writes the n-th four of a row's sums divided by l, and at n = 0 the log of the sum.
template <int D>
__device__ __forceinline__ void put_row(bf16* out, float* lse, int n, float4 v, float m, float l) {
    const float inv = l == 0.f ? 0.f : __frcp_rn(l);
    *reinterpret_cast<uint32_t*>(out + dim_of<D>(2 * n)) = pack_bf16x2(v.x * inv, v.y * inv);
    *reinterpret_cast<uint32_t*>(out + dim_of<D>(2 * n + 1)) = pack_bf16x2(v.z * inv, v.w * inv);
    if (n == 0 && lse)
        *lse = l == 0.f ? -__int_as_float(0x7f800000) : (m + log2f(l)) * 0.693147180559945309f;
}

// The columns' state of one warp over one item.
template <int D, int NT>
struct Warp {
    static constexpr int NG = D / 32;   // groups, and K words per lane and token
    static constexpr int VW = D / 64;   // V words per lane and token
    static constexpr int MT = D / 16;   // M tiles of O^T
    static constexpr int NZ = D == 256 ? 2 : 1;  // matrix steps of the minima
    static constexpr bool QS = q_in_smem(D, NT);
    uint32_t qf[QS ? 1 : NT][NG][4];    // q as binary16 pairs, column g
    uint4* qs;                          // the same in shared memory
    uint32_t qz[NT][NZ][2];             // sums of q per group, three bf16 terms, column g
    float f[NT][2];                     // factor of the code products, log2 units
    int col0, cols, seen0;              // the item's first column, all columns, tokens column 0 sees
    float o[NT][MT][4];                 // times 2^k
    float m[NT][2], l[NT][2];
    int k;                              // of the lane's group of V dims
    uint32_t bound_s, bound_z;          // 2^(k - 9) and 2^(k + 14) less one step, bf16 twice
    bool first;                         // no unit seen yet

    // Loads the item's query rows and resets the sums.
    __device__ __forceinline__ void begin(const Args& a, const Seq& s, int qb, int h, int lane) {
        const int g = lane >> 2, t = lane & 3;
        first = true;
        set_k(-100);  // V below about 2^-100 counts as 0
        col0 = qb * NT * 8;
        cols = s.n * a.group;
        seen0 = s.len - s.n + 1;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int col = (qb * NT + nt) * 8 + g;
            float x[NG][8];
            float amax = 0.f;
            const bool ok = col < s.n * a.group;
            const int i = ok ? a.over_group(col) : 0;
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
            // the row's largest becomes 2^14 .. 2^15 (unless it is below 2^-85)
            const int ex = amax > 0.f && amax <= FLT_MAX ? max(exponent(amax) - 15, -100) : 0;
            const float p0 = pow2(-ex), p1 = pow2(-ex - 4);
            float z[NG];
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                z[j] = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) z[j] += x[j][e];
                z[j] += __shfl_xor_sync(0xffffffffu, z[j], 1);
                z[j] += __shfl_xor_sync(0xffffffffu, z[j], 2);
                z[j] *= a.scale_log2;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float p = e & 1 ? p1 : p0;
                    qf[QS ? 0 : nt][j][e] = pack_f16x2(x[j][e] * p, x[j][e + 4] * p);
                }
                if (QS) qs[(nt * NG + j) * 32] = make_uint4(qf[0][j][0], qf[0][j][1], qf[0][j][2], qf[0][j][3]);
            }
            // the lane's two groups of the minima's product, each sum as three bf16 terms
            float u0 = z[0], u1 = z[1];
#pragma unroll
            for (int j = 2; j < NG; j += 2) {
                const bool mine = j == ((NG - 1) & (2 * t));
                u0 = mine ? z[j] : u0;
                u1 = mine ? z[j + 1] : u1;
            }
            uint32_t term[3];
#pragma unroll
            for (int e = 0; e < 3; ++e) {
                term[e] = pack_bf16x2(u0, u1);
                u0 -= bf16_lo(term[e]);
                u1 -= bf16_hi(term[e]);
            }
            if constexpr (D == 64) {  // steps: terms 0, 1, 2, none by t
                qz[nt][0][0] = t == 0 ? term[0] : t == 1 ? term[1] : t == 2 ? term[2] : 0u;
                qz[nt][0][1] = 0u;
            } else if constexpr (D == 128) {  // term 0 | 1 by t / 2, then 2 | none
                qz[nt][0][0] = t < 2 ? term[0] : term[1];
                qz[nt][0][1] = t < 2 ? term[2] : 0u;
            } else {
                qz[nt][0][0] = term[0];
                qz[nt][0][1] = term[1];
                qz[nt][NZ - 1][0] = term[2];
                qz[nt][NZ - 1][1] = 0u;
            }
            const float fac = a.scale_log2 * 16777216.f * pow2(ex);  // 2^(ex + 24) may leave FP32
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                f[nt][c] = __shfl_sync(0xffffffffu, fac, 8 * t + 4 * c);  // of column 2t + c
                m[nt][c] = l[nt][c] = 0.f;
            }
#pragma unroll
            for (int i2 = 0; i2 < MT; ++i2)
#pragma unroll
                for (int c = 0; c < 4; ++c) o[nt][i2][c] = 0.f;
        }
    }

    __device__ __forceinline__ void set_k(int kn) {
        k = kn;
        bound_s = (uint32_t)(((k - 9 + 127) << 7) - 1) * 0x10001u;
        bound_z = (uint32_t)((min(k + 14 + 127, 255) << 7) - 1) * 0x10001u;
    }
    // Tokens that column 8 nt + c of the item sees.
    __device__ __forceinline__ int limit(const Args& a, int c) const {
        const int cc = col0 + c;
        return cc < cols ? seen0 + a.over_group(cc) : 0;
    }

    // Scores less the reference (log2 units) of the 16 tokens of one record.  FULL: every
    // column sees all of them.
    template <bool FULL>
    __device__ __forceinline__ void scores(const Args& a, const uint8_t* rec, int tok0, int lane,
                                           float (&sc)[NT][4]) {
        const int g = lane >> 2, t = lane & 3;
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
        // minima of groups 2t, 2t + 1 of the product's steps
        const int jz = D == 64 ? 0 : D == 128 ? 2 * (t & 1) : 2 * t;
        uint32_t z0[2], z1[2];
        lds_words(rec + kv4_k_scale(D, g, jz), z0);
        lds_words(rec + kv4_k_scale(D, g + 8, jz), z1);
        const uint32_t za = __byte_perm(z0[0], z0[1], 0x7632), zb = __byte_perm(z1[0], z1[1], 0x7632);
        float zs[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                sc[nt][c] = 0.f;
                zs[nt][c] = -m[nt][c & 1];
            }
            mma_bf16(zs[nt], za, zb, za, zb, qz[nt][0][0], qz[nt][0][1]);
            if constexpr (NZ == 2) mma_bf16(zs[nt], za, zb, za, zb, qz[nt][1][0], qz[nt][1][1]);
        }
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            const uint32_t h0 = k0[j] >> 8, h1 = k1[j] >> 8;
            const uint32_t lo = 0x000f000fu, up = 0x00f000f0u;
            const float f0 = bf16_lo(s0[j]), f1 = bf16_lo(s1[j]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float d[4] = {0.f, 0.f, 0.f, 0.f};
                const uint4 q = QS ? qs[(nt * NG + j) * 32]
                                   : make_uint4(qf[QS ? 0 : nt][j][0], qf[QS ? 0 : nt][j][1],
                                                qf[QS ? 0 : nt][j][2], qf[QS ? 0 : nt][j][3]);
                mma_f16(d, k0[j] & lo, k1[j] & lo, k0[j] & up, k1[j] & up, q.x, q.y);
                mma_f16(d, h0 & lo, h1 & lo, h0 & up, h1 & up, q.z, q.w);
                sc[nt][0] = fmaf(f0, d[0], sc[nt][0]);
                sc[nt][1] = fmaf(f0, d[1], sc[nt][1]);
                sc[nt][2] = fmaf(f1, d[2], sc[nt][2]);
                sc[nt][3] = fmaf(f1, d[3], sc[nt][3]);
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                sc[nt][c] = fmaf(sc[nt][c], f[nt][c & 1], zs[nt][c]);
                if (!FULL && tok0 + g + 8 * (c >> 1) >= limit(a, 8 * nt + 2 * t + (c & 1)))
                    sc[nt][c] = -__int_as_float(0x7f800000);
            }
    }

    // Scales (x) and minima (y) of V of tokens r, r + 1 in the lane's group.
    __device__ __forceinline__ uint2 scale_words(const uint8_t* rec, int r, int lane) {
        return *reinterpret_cast<const uint2*>(rec + kv4_v_scale(D, r, (lane >> 2) / (256 / D)));
    }
    // The largest of what has to fit: s 2^9 and |z| 2^-14, as FP32 (NaN left out).
    __device__ __forceinline__ float need(uint2 v) {
        return fmaxf(fmaxf(bf16_lo(v.x), bf16_hi(v.x)) * 512.f,
                     fmaxf(fabsf(bf16_lo(v.y)), fabsf(bf16_hi(v.y))) * 6.103515625e-5f);
    }
    // FULL false: tokens at `len` and behind are left out; so is what is not finite, since it
    // must not reach the columns that do not see its token.
    template <bool FULL>
    __device__ __forceinline__ void keep(uint2& v, int tok, int len, bool& odd) {
        if (FULL) return;
        const uint32_t in = (tok < len ? 0xffffu : 0u) | (tok + 1 < len ? 0xffff0000u : 0u);
        v.x &= in;
        v.y &= in;
        uint32_t drop = 0u;
        if ((v.x & 0x7f80u) == 0x7f80u || (v.y & 0x7f80u) == 0x7f80u) drop |= 0xffffu;
        if ((v.x & 0x7f800000u) == 0x7f800000u || (v.y & 0x7f800000u) == 0x7f800000u)
            drop |= 0xffff0000u;
        odd |= drop != 0u;
        v.x &= ~drop;
        v.y &= ~drop;
    }

    // o += V^T P^T for the 16 tokens of one record.
    template <bool FULL>
    __device__ __forceinline__ void values(const Args& a, const uint8_t* rec, int tok0, int len, int lane, uint2 va,
                                           uint2 vb, bool odd, const float (&sc)[NT][4]) {
        const int g = lane >> 2, t = lane & 3;
        uint32_t b0[NT], b1[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float p[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) p[c] = ex2(sc[nt][c]);
            l[nt][0] += p[0] + p[2];
            l[nt][1] += p[1] + p[3];
            b0[nt] = transpose8x8(pack_f16x2(p[0], p[1]));
            b1[nt] = transpose8x8(pack_f16x2(p[2], p[3]));
        }
        const float ps = pow2(24 - k), pz = pow2(-k);
        const uint32_t sa = pack_f16x2(bf16_lo(va.x) * ps, bf16_hi(va.x) * ps);
        const uint32_t sb = pack_f16x2(bf16_lo(vb.x) * ps, bf16_hi(vb.x) * ps);
        const uint32_t za = pack_f16x2(bf16_lo(va.y) * pz, bf16_hi(va.y) * pz);
        const uint32_t zb = pack_f16x2(bf16_lo(vb.y) * pz, bf16_hi(vb.y) * pz);
        const uint32_t sa4 = hmul2(sa, 0x2c002c00u), sb4 = hmul2(sb, 0x2c002c00u);  // 2^-4
        uint32_t w0[VW], w1[VW], w8[VW], w9[VW];
        lds_words(rec + kv4_v_unit(D, 2 * t, g), w0);
        lds_words(rec + kv4_v_unit(D, 2 * t + 1, g), w1);
        lds_words(rec + kv4_v_unit(D, 2 * t + 8, g), w8);
        lds_words(rec + kv4_v_unit(D, 2 * t + 9, g), w9);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int w = i / 4, half = i / 2 % 2;
            uint32_t pa = __byte_perm(w0[w], w1[w], half ? 0x7632 : 0x5410);
            uint32_t pb = __byte_perm(w8[w], w9[w], half ? 0x7632 : 0x5410);
            if (i & 1) {
                pa >>= 8;
                pb >>= 8;
            }
            const uint32_t a0 = hfma2(pa & 0x000f000fu, sa, za);
            const uint32_t a1 = hfma2(pa & 0x00f000f0u, sa4, za);
            const uint32_t a2 = hfma2(pb & 0x000f000fu, sb, zb);
            const uint32_t a3 = hfma2(pb & 0x00f000f0u, sb4, zb);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_f16(o[nt][i], a0, a1, a2, a3, b0[nt], b1[nt]);
        }
        if (!FULL && __any_sync(0xffffffffu, odd)) not_finite(a, rec, tok0, len, g, t);
    }

    // The columns that see a token whose V is not finite become NaN in that group's dims.
    __device__ __forceinline__ void not_finite(const Args& a, const uint8_t* rec, int tok0, int len, int g,
                                               int t) {
        for (int r = 0; r < kKv4Block && tok0 + r < len; ++r) {
            const uint16_t* p =
                reinterpret_cast<const uint16_t*>(rec + kv4_v_scale(D, r, g / (256 / D)));
            if ((p[0] & 0x7f80) != 0x7f80 && (p[2] & 0x7f80) != 0x7f80) continue;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    if (tok0 + r < limit(a, 8 * nt + 2 * t + c))
#pragma unroll
                        for (int i = 0; i < MT; ++i) {
                            o[nt][i][c] = __int_as_float(0x7fffffff);
                            o[nt][i][c + 2] = __int_as_float(0x7fffffff);
                        }
        }
    }

    // Adds the 32 tokens of one unit; `have`: bit i is set where record i is there.
    template <bool FULL>
    __device__ __forceinline__ void unit(const Args& a, const uint8_t* rec, int tok0, int len, int have,
                                         int lane) {
        const uint8_t* rec1 = rec + 20 * D;
        const int t = lane & 3;
        // a record that is not there: no token of it is seen
        const int t0 = FULL || (have & 1) ? tok0 : 0x40000000;
        const int t1 = FULL || (have & 2) ? tok0 + kKv4Block : 0x40000000;
        float sc0[NT][4], sc1[NT][4];
        scores<FULL>(a, rec, t0, lane, sc0);
        scores<FULL>(a, rec1, t1, lane, sc1);
        uint2 v[4] = {scale_words(rec, 2 * t, lane), scale_words(rec, 2 * t + 8, lane),
                      scale_words(rec1, 2 * t, lane), scale_words(rec1, 2 * t + 8, lane)};
        bool odd0 = false, odd1 = false;
        keep<FULL>(v[0], t0 + 2 * t, len, odd0);
        keep<FULL>(v[1], t0 + 2 * t + 8, len, odd0);
        keep<FULL>(v[2], t1 + 2 * t, len, odd1);
        keep<FULL>(v[3], t1 + 2 * t + 8, len, odd1);
        // s < 2^(k - 9) and |z| < 2^(k + 14), as bf16 numbers two at a time
        const uint32_t ms = max_u16x2(max_u16x2(v[0].x, v[1].x), max_u16x2(v[2].x, v[3].x));
        const uint32_t mz = max_u16x2(max_u16x2(v[0].y & 0x7fff7fffu, v[1].y & 0x7fff7fffu),
                                      max_u16x2(v[2].y & 0x7fff7fffu, v[3].y & 0x7fff7fffu));
        bool up = first || max_u16x2(ms, bound_s) != bound_s || max_u16x2(mz, bound_z) != bound_z;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c)
                up |= fmaxf(fmaxf(sc0[nt][c], sc0[nt][c + 2]), fmaxf(sc1[nt][c], sc1[nt][c + 2])) > 8.f;
        if (__any_sync(0xffffffffu, up)) raise(v, sc0, sc1);
        values<FULL>(a, rec, t0, len, lane, v[0], v[1], odd0, sc0);
        values<FULL>(a, rec1, t1, len, lane, v[2], v[3], odd1, sc1);
    }

    // Moves the references to the unit's largest scores where they are above them (at the first
    // unit in any case), and 2^k above what V needs; rescales the sums.
    __device__ __forceinline__ void raise(const uint2 (&v4)[4], float (&sc0)[NT][4],
                                          float (&sc1)[NT][4]) {
        const float nd = fmaxf(fmaxf(need(v4[0]), need(v4[1])), fmaxf(need(v4[2]), need(v4[3])));
        int kn = nd >= pow2(k) && k < 127 ? min(exponent(nd) + 1, 127) : k;
        if (kn < k) kn = k;  // what is not finite asks for nothing
#pragma unroll
        for (int o2 = 1; o2 < (D == 64 ? 16 : D == 128 ? 8 : 4); o2 <<= 1)
            kn = max(kn, __shfl_xor_sync(0xffffffffu, kn, o2));
        const float rk = pow2(k - kn);
        set_k(kn);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float v = fmaxf(fmaxf(sc0[nt][c], sc0[nt][c + 2]), fmaxf(sc1[nt][c], sc1[nt][c + 2]));
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                if (first ? v == -__int_as_float(0x7f800000) : !(v > 0.f)) v = 0.f;
                const float r = first ? 0.f : ex2(-v);
                m[nt][c] += v;
                l[nt][c] *= r;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    sc0[nt][c + 2 * i] -= v;
                    sc1[nt][c + 2 * i] -= v;
                }
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    o[nt][i][c] *= r * rk;
                    o[nt][i][c + 2] *= r * rk;
                }
            }
        first = false;
    }
};

// SOLO: every item is a warp's own (no sequence is longer than kWholeUnits).
template <int D, int NT, bool SOLO>
__global__ void __launch_bounds__(kWarps * 32, ctas_of(D, NT)) kv4_attention_kernel(const Args a) {
    using Sm = Smem<D, NT>;
    constexpr int S = Sm::S, QC = Sm::QC;
    constexpr uint32_t kRec = 20 * D;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    Sm& sm = *reinterpret_cast<Sm*>(smem_raw);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

    if (threadIdx.x == 0) {
        for (int w = 0; w < kWarps; ++w)
            for (int s = 0; s < S; ++s) mbar_init(&sm.full[w][s], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }

    __syncthreads();  // the barriers are there
    // The length of the line, then the sequence that holds this CTA's first place: every warp
    // for itself.
    const bool report = blockIdx.x == 0 && warp == 0;
    int64_t total = 0, items = 0;
    int longest = 0;
    for (int b = lane; b < a.seqs; b += 32) {
        const Seq s = seq_of<QC>(a, b, report);
        total += places_of(s, a.kv_heads, false);
        items += places_of(s, a.kv_heads, true);
        longest = max(longest, s.units);
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    const bool whole = SOLO || longest <= kWholeUnits;
    if (whole) total = items;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    const int first_warp = SOLO ? 0 : warp;
    constexpr int WARPS = SOLO ? 1 : kWarps;  // that share an item
    const int64_t per = share_of(total, gridDim.x * (kWarps / WARPS), whole ? 1 : kMinShare);
    const int64_t begin = (SOLO ? blockIdx.x * kWarps + warp : blockIdx.x) * per;
    const int64_t end = min(begin + per, total);
    if (begin >= end && blockIdx.x != 0) return;
    int b = 0;
    int64_t seq_first = 0;  // first place of sequence b
    int64_t before = 0;
    for (int b0 = 0; b0 < a.seqs; b0 += 32) {
        const int64_t mine =
            b0 + lane < a.seqs ? places_of(seq_of<QC>(a, b0 + lane, false), a.kv_heads, whole) : 0;
        int64_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        const int64_t excl = before + incl - mine;
        if (report && !whole && b0 + lane < a.seqs) a.prefix[b0 + lane] = excl;
        const unsigned hit = __ballot_sync(0xffffffffu, begin >= excl && begin < excl + mine);
        if (hit) {
            b = b0 + __ffs(hit) - 1;
            seq_first = __shfl_sync(0xffffffffu, excl, __ffs(hit) - 1);
            if (!report || whole) break;
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (report && lane == 0) a.prefix[a.seqs] = whole ? -1 : total;
    if (begin >= end) return;

    // Every warp's own copy of where it is, in shared memory: the registers are the sums'.
    Piece& it = sm.piece[warp];
    auto advance = [&](Piece p) -> bool {  // from p to the CTA's next piece, if there is one
        bool found = false;
        while (p.u < end && !found) {
            while (p.u >= p.seq_first + places_of(p.s, a.kv_heads, whole)) {
                p.seq_first += places_of(p.s, a.kv_heads, whole);
                p.s = seq_of<QC>(a, ++p.b, false);  // u < total, so a sequence with work follows
            }
            const int64_t in_seq = p.u - p.seq_first;
            const int len = whole ? 1 : p.s.units + kItemCost;
            const int item =
                in_seq >> 32 ? (int)(in_seq / len) : (int)((uint32_t)in_seq / (uint32_t)len);
            const int64_t first = p.seq_first + (int64_t)item * len + kItemCost;  // of its units
            p.k0 = whole ? 0 : (int)max(p.u - first, (int64_t)0);
            p.k1 = whole ? p.s.units : (int)min((int64_t)p.s.units, end - first);
            p.u = whole ? p.u + 1 : first + p.s.units;
            p.qb = item / a.kv_heads;
            p.h = item - p.qb * a.kv_heads;
            found = whole || p.k1 > p.k0;
        }
        __syncwarp();  // every lane has read it
        if (lane == 0) it = p;
        __syncwarp();
        return found;
    };
    uint32_t phase = 0u, have = 0u;  // per stage: parity waited for next; records in flight
    bool dead = false;
    // record x & 1 of this warp's unit x / 2; -1: behind the end, or page outside the cache
    auto record = [&](int x) -> int {
        const int ku = it.k0 + first_warp + (x >> 1) * WARPS, kb = 2 * ku + (x & 1);
        if (ku >= it.k1 || kb * kKv4Block >= it.s.len) return -1;
        const int p = kb / a.nb;
        const int page = __ldg(a.table + it.b * a.table_stride + p);
        if (page < 0 || page >= a.pages) {
            atomicOr(a.err, ERR_INDEX);
            return -1;
        }
        return (page * a.kv_heads + it.h) * a.nb + (kb - p * a.nb);
    };
    // copies unit x's records (rec of this lane's window) to a stage; which ones there are
    auto issue = [&](int stage, int window, int x) {
        const int r0 = __shfl_sync(0xffffffffu, window, 2 * x & 31);
        const int r1 = __shfl_sync(0xffffffffu, window, (2 * x + 1) & 31);
        const uint32_t got = (r0 >= 0 ? 1u : 0u) | (r1 >= 0 ? 2u : 0u);
        have = (have & ~(3u << (2 * stage))) | got << (2 * stage);
        if (lane == 0 && got) {
            uint64_t* bar = &sm.full[warp][stage];
            uint8_t* dst = sm.room[warp] + stage * Sm::kStage;
            mbar_arrive_expect_tx(bar, got == 3u ? 2 * kRec : kRec);
            if (got == 3u && r1 == r0 + 1) {
                bulk_load(dst, a.cache + (int64_t)r0 * kRec, 2 * kRec, bar);
            } else {
                if (r0 >= 0) bulk_load(dst, a.cache + (int64_t)r0 * kRec, kRec, bar);
                if (r1 >= 0) bulk_load(dst + kRec, a.cache + (int64_t)r1 * kRec, kRec, bar);
            }
        }
    };
    auto units_of = [&]() {
        return dead ? 0 : max(0, (it.k1 - it.k0 - first_warp + WARPS - 1) / WARPS);
    };

    auto together = [] {  // the warps that share an item
        if constexpr (SOLO) __syncwarp();
        else __syncthreads();
    };

    if (!advance(Piece{seq_of<QC>(a, b, false), b, 0, 0, 0, 0, seq_first, begin})) return;
    int now = record(lane), next = record(32 + lane), n = units_of();
#pragma unroll
    for (int i = 0; i < S; ++i)
        if (i < n) issue(i, now, i);
    Warp<D, NT> st;
    st.qs = reinterpret_cast<uint4*>(sm.room[warp] + S * Sm::kStage) + lane;
    for (;;) {
        const Seq s = it.s;
        const int len = s.len;
        // every column sees the tokens before this one
        const int safe = len - s.n + 1 + a.over_group(it.qb * QC);
        st.begin(a, s, it.qb, it.h, lane);
        int stage = 0, tok0 = (it.k0 + first_warp) * kUnit;
        for (int i = 0; i < n; ++i) {
            const int got = (have >> (2 * stage)) & 3u;
            if (got) {
                const bool landed = mbar_wait(&sm.full[warp][stage], (phase >> stage) & 1u,
                                              a.limit_ns);
                if (!__all_sync(0xffffffffu, landed)) {
                    if (lane == 0) atomicOr(a.err, ERR_WAIT_FULL);
                    dead = true;
                    break;
                }
                phase ^= 1u << stage;
                have &= ~(3u << (2 * stage));
                if (got == 3 && tok0 + kUnit <= safe)
                    st.template unit<true>(a, sm.room[warp] + stage * Sm::kStage, tok0, len, got, lane);
                else
                    st.template unit<false>(a, sm.room[warp] + stage * Sm::kStage, tok0, len, got, lane);
                __syncwarp();
            }
            const int ahead = i + S;
            if (ahead < n) issue(stage, (ahead >> 4) == (i >> 4) ? now : next, ahead);
            if ((i & 15) == 15) {
                now = next;
                next = record(2 * (i + 17) + lane);
            }
            stage = stage + 1 == S ? 0 : stage + 1;
            tok0 += WARPS * kUnit;
        }

        // merge the warps
        const int g = lane >> 2, t = lane & 3;
        const float pk = pow2(st.k);
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
                    sm.m[warp][col] = l == 0.f ? -FLT_MAX : st.m[nt][c];
                    sm.l[warp][col] = l;
                }
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
                    *reinterpret_cast<float2*>(sm.sums(warp, col) + 16 * i + 2 * g) =
                        make_float2(st.o[nt][i][c] * pk, st.o[nt][i][c + 2] * pk);
            }
        }
        const bool alone = it.k0 == 0 && it.k1 == it.s.units;
        const int slot = it.u - it.s.units < begin ? 0 : 1;
        const int col0 = it.qb * QC, cols = it.s.n * a.group, head0 = it.h * a.group, q0 = it.s.q0;

        // the next piece's first units are on their way while this one's warps merge
        const bool more = it.u < end && advance(it);
        if (more) {
            now = record(lane);
            next = record(32 + lane);
            n = units_of();
#pragma unroll
            for (int i = 0; i < Sm::P; ++i)
                if (i < n) issue(i, now, i);
        }
        together();
        for (int x = SOLO ? lane : threadIdx.x; x < QC * D / 4; x += WARPS * 32) {
            const int col = x / (D / 4), e4 = x % (D / 4);
            const int idx = col0 + col;
            if (idx >= cols) continue;
            const int w0 = SOLO ? warp : 0;
            float m = sm.m[w0][col];
#pragma unroll
            for (int w = 1; w < WARPS; ++w) m = fmaxf(m, sm.m[w][col]);
            float l = 0.f;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                const float e = ex2(sm.m[w0 + w][col] - m);
                const float4 o = *reinterpret_cast<const float4*>(sm.sums(w0 + w, col) + 4 * e4);
                l = fmaf(e, sm.l[w0 + w][col], l);
                v.x = fmaf(e, o.x, v.x);
                v.y = fmaf(e, o.y, v.y);
                v.z = fmaf(e, o.z, v.z);
                v.w = fmaf(e, o.w, v.w);
            }
            if (alone) {
                const int i = a.over_group(idx), hq = head0 + idx - i * a.group;
                const int64_t row = q0 + i;
                put_row<D>(a.out + row * a.out_st + hq * a.out_sh,
                           a.lse ? a.lse + row * a.heads + hq : nullptr, e4, v, m, l);
            } else {
                const int64_t at = ((int64_t)blockIdx.x * 2 + slot) * QC + col;
                *reinterpret_cast<float4*>(a.part + at * D + 4 * e4) = v;
                if (e4 == 0) a.part_ml[at] = make_float2(m, l);
            }
        }
        if (!more) break;
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the ring is next
        together();
#pragma unroll
        for (int i = Sm::P; i < S; ++i)
            if (i < n) issue(i, now, i);
    }
    // after a wait that ran out: the copies still in flight must land before the CTA ends
    for (int i = 0; i < S; ++i)
        if ((have >> (2 * i)) & 3u)
            if (!mbar_wait(&sm.full[warp][i], (phase >> i) & 1u, a.limit_ns) && lane == 0)
                atomicOr(a.err, ERR_WAIT_DRAIN);
}

// Rows (query token, head) whose item lies in several CTAs, or has no tokens at all.  D/4 lanes
// hold a row.  WIDE: a CTA per row, whose 4096/D groups of lanes take the partial sums in turn
// and are merged in order; otherwise each group has a row of its own (items that lie in a few
// CTAs only).
__host__ __device__ constexpr int combine_threads(bool wide) { return wide ? 1024 : 256; }

template <int D, int NT, bool WIDE>
__global__ void __launch_bounds__(combine_threads(WIDE)) kv4_combine_kernel(const Args a, int ctas) {
    constexpr int QC = 8 * NT, LN = D / 4, GR = combine_threads(WIDE) / LN, U = WIDE ? 2 : 4;
    constexpr int STEP = WIDE ? GR : 1;
    __shared__ float4 so[WIDE ? GR : 1][LN];
    __shared__ float smx[GR], sl[GR];
    const int ln = threadIdx.x % LN, gr = threadIdx.x / LN;
    const int64_t at_row = WIDE ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * GR + gr;
    const bool in = at_row < (int64_t)a.tokens * a.heads;
    const int row = in ? (int)at_row / a.heads : 0, hq = in ? (int)at_row - row * a.heads : 0;
    const int h = a.over_group(hq);
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
    const Seq s = seq_of<QC>(a, b, false);
    // every CTA waits here: what is launched next relies on this grid's end being the other's too
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!in || row < s.q0 || row >= s.q0 + s.n) return;
    const int idx = (row - s.q0) * a.group + hq - h * a.group;
    const int qb = idx / QC, col = idx - qb * QC;
    bf16* out = a.out + (int64_t)row * a.out_st + (int64_t)hq * a.out_sh;
    float* lse = a.lse ? a.lse + at_row : nullptr;
    if (s.units == 0) {
        if (!WIDE || gr == 0) {
            *reinterpret_cast<uint2*>(out + 4 * ln) = make_uint2(0u, 0u);
            if (ln == 0 && lse) *lse = -__int_as_float(0x7f800000);
        }
        return;
    }
    const int64_t places = a.prefix[a.seqs];
    if (places < 0) return;  // no item was split
    const int64_t per = share_of(places, ctas, kMinShare);
    const int64_t u0 = a.prefix[b] + ((int64_t)qb * a.kv_heads + h) * (s.units + kItemCost) + kItemCost;
    const int64_t u1 = u0 + s.units - 1;
    const bool big = ((u1 | per) >> 32) != 0;
    const int c0 = big ? (int)(u0 / per) : (int)((uint32_t)u0 / (uint32_t)per);
    const int c1 = big ? (int)(u1 / per) : (int)((uint32_t)u1 / (uint32_t)per);
    if (c0 == c1) return;
    float m = -FLT_MAX, l = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = c0 + (WIDE ? gr : 0); c <= c1; c += U * STEP) {
        float2 ml[U];
        float4 o[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int64_t cta = c + i * STEP;
            ml[i] = make_float2(-FLT_MAX, 0.f);
            o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (cta <= c1) {
                const int64_t at = (cta * 2 + (u0 < cta * per ? 0 : 1)) * QC + col;
                ml[i] = __ldcg(a.part_ml + at);
                o[i] = __ldcg(reinterpret_cast<const float4*>(a.part + at * D) + ln);
            }
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const float mn = fmaxf(m, ml[i].x);
            const float e0 = ex2(m - mn), e1 = ex2(ml[i].x - mn);
            m = mn;
            l = fmaf(e1, ml[i].y, e0 * l);
            v.x = fmaf(e1, o[i].x, e0 * v.x);
            v.y = fmaf(e1, o[i].y, e0 * v.y);
            v.z = fmaf(e1, o[i].z, e0 * v.z);
            v.w = fmaf(e1, o[i].w, e0 * v.w);
        }
    }
    if (WIDE) {
        so[gr][ln] = v;
        if (ln == 0) {
            smx[gr] = m;
            sl[gr] = l;
        }
        __syncthreads();
        if (gr != 0) return;
#pragma unroll 4
        for (int k = 1; k < GR; ++k) m = fmaxf(m, smx[k]);
        l = 0.f;
        v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int k = 0; k < GR; ++k) {
            const float e = ex2(smx[k] - m);
            const float4 o = so[k][ln];
            l = fmaf(e, sl[k], l);
            v.x = fmaf(e, o.x, v.x);
            v.y = fmaf(e, o.y, v.y);
            v.z = fmaf(e, o.z, v.z);
            v.w = fmaf(e, o.w, v.w);
        }
    }
    put_row<D>(out, lse, ln, v, m, l);
}

int64_t prefix_bytes(int seqs) { return ((int64_t)(seqs + 1) * 8 + 255) / 256 * 256; }

// The most tiles of 8 columns of one item for heads of D that registers hold without slowing down
// (D = 128, 32 columns in one item of four tiles and in two of two: 16 sequences of up to 8192 tokens
// 66 and 62 us, 64 of up to 1000 85 and 69; 24 columns in one of three and in two of two: 38
// sequences of 8329 tokens 137 and 210 us), and the most columns of all CTAs of an SM.
int most_tiles(int D) { return D == 64 ? 4 : D == 128 ? 3 : 2; }
int most_columns(int D) {
    int n = 0;
    for (int t = 1; t <= most_tiles(D); ++t) n = std::max(n, 8 * t * ctas_of(D, t));
    return n;
}

template <int D, int NT, bool SOLO>
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
    a.group_inv = a.group == 1 ? 0 : ~0ull / (uint64_t)a.group + 1;
    a.table_width = c.table_width;
    a.nb = c.blocks_per_page;
    a.scale_log2 = c.scale * 1.44269504088896340736f;

    Launch L{};
    L.sms = c.sms;
    L.grid = (int64_t)c.sms * ctas_of(D, NT);
    L.smem = sizeof(Smem<D, NT>);
    int64_t grid = 0;
    auto k = kv4_attention_kernel<D, NT, SOLO>;
    cudaError_t e = fit_grid((const void*)k, L, kWarps * 32, &grid);
    if (e != cudaSuccess) return e;
    uint8_t* ws = static_cast<uint8_t*>(c.ws);
    a.prefix = reinterpret_cast<int64_t*>(ws);
    a.part = reinterpret_cast<float*>(ws + prefix_bytes(c.seqs));
    a.part_ml = reinterpret_cast<float2*>(a.part + grid * 2 * 8 * NT * D);
    const int64_t rows = (int64_t)c.tokens * c.heads;
    const int64_t items = std::max((int64_t)c.seqs * c.kv_heads, rows / (8 * NT));
    k<<<(unsigned)grid, kWarps * 32, (size_t)L.smem, s>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if ((int64_t)c.table_width * c.blocks_per_page * kKv4Block <= kWholeUnits * kUnit) return e;

    // an item lies in about grid / items CTAs (all of the same length): from 8 on, a CTA per row
    const bool wide = grid >= 8 * items;
    const int per_cta = wide ? 1 : combine_threads(false) * 4 / D;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((rows + per_cta - 1) / per_cta));
    cfg.blockDim = dim3(combine_threads(wide));
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return wide ? cudaLaunchKernelEx(&cfg, kv4_combine_kernel<D, NT, true>, (const Args)a, (int)grid)
                : cudaLaunchKernelEx(&cfg, kv4_combine_kernel<D, NT, false>, (const Args)a, (int)grid);
}

}  // namespace

int64_t kv4_attention_workspace(int seqs, int D, int sms) {
    return prefix_bytes(seqs) + (int64_t)sms * 2 * most_columns(D) * (D + 2) * 4;
}

// Items of short sequences, more than there are CTAs: a warp to each.  It takes an item's units one
// after the other, but with no barriers and no merge (300 sequences of up to 16 / 100 / 200 tokens
// 24.2 / 31.1 / 36.0 us with a CTA to each, 12.8 / 17.6 / 23.7 so; with fewer items than CTAs it is
// slower: one sequence of 100 tokens 6.5 and 10.6).
template <int D, int NT>
cudaError_t short_or_long(const Kv4Attention& c, cudaStream_t s) {
    const int64_t ctas = (int64_t)c.sms * ctas_of(D, NT);
    const int64_t items = std::max((int64_t)c.seqs * c.kv_heads, (int64_t)c.tokens * c.heads / (8 * NT));
    const int64_t tokens = (int64_t)c.table_width * c.blocks_per_page * kKv4Block;  // of a sequence, at most
    const bool solo = tokens <= kWholeUnits * kUnit &&
                      items > (tokens <= kSoloUnits * kUnit ? ctas : 2 * ctas);
    return solo ? run<D, NT, true>(c, s) : run<D, NT, false>(c, s);
}

cudaError_t launch_kv4_attention(const Kv4Attention& c, cudaStream_t s) {
    // the fewest blocks of columns, and for these the fewest tiles
    const int64_t cols = (int64_t)c.max_q * (c.heads / c.kv_heads), most = 8 * most_tiles(c.D);
    const int64_t blocks = (cols + most - 1) / most;
    const int nt = (int)((cols + 8 * blocks - 1) / (8 * blocks));
    switch (c.D) {
        case 64:
            return nt == 1 ? short_or_long<64, 1>(c, s) : nt == 2 ? short_or_long<64, 2>(c, s)
                   : nt == 3 ? run<64, 3, false>(c, s) : run<64, 4, false>(c, s);
        case 128:
            return nt == 1 ? short_or_long<128, 1>(c, s) : nt == 2 ? short_or_long<128, 2>(c, s)
                           : run<128, 3, false>(c, s);
        case 256: return nt == 1 ? short_or_long<256, 1>(c, s) : run<256, 2, false>(c, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace rmsn
