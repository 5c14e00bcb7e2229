// rmsn_kv4_layout.h -- where a 4-bit cache keeps what (plain C++, host and device).
//
// The cache is [pages][kv heads][page / 16] records of 20 D bytes; a record holds 16
// consecutive tokens of one head.  Groups of 32 dims share a scale s and a minimum z (bf16);
// the value of a code c (0 .. 15) is c s + z.
//
//   bytes [0, 8D)      K codes      [16D, 18D)  K's (s, z) by token and group
//   bytes [8D, 16D)    V codes      [18D, 20D)  V's s, s, z, z of two tokens by group
//
// Codes are two to a byte, the even dim in the low half.  The order inside a record is that
// of the fragments the attention kernel feeds to the matrix instructions, so that its loads
// from shared memory are one wide access per lane without bank conflicts:
//   K: lane (g, t) of a warp (g = lane / 4, t = lane % 4) needs, of tokens g and g + 8, the
//      eight dims 32 j + 8 t .. + 7 of every group j: one 32-bit word per group, and the words
//      of a lane lie side by side.  D = 256: 16-byte units of odd tokens are swapped in pairs.
//   V: lane (g, t) needs of tokens 2t, 2t+1, 2t+8, 2t+9 the dims [g D/8, (g+1) D/8).  Token r
//      has row kv4_v_row(r), so the four lanes t read four neighbouring rows, and the units of
//      D/16 bytes inside a row are permuted by the row.
// Every token owns whole bytes (and whole 2-byte scales), so tokens are stored independently.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define RMSN_HD __host__ __device__ __forceinline__
#else
#define RMSN_HD inline
#endif

namespace rmsn {

constexpr int kKv4Block = 16;  // tokens per record
constexpr int kKv4Group = 32;  // dims per scale

RMSN_HD int kv4_record_bytes(int D) { return 20 * D; }

// Byte offset of the 32-bit word with the K codes of dims 8w .. 8w+7 of token r (w < D/8).
RMSN_HD int kv4_k_word(int D, int r, int w) {
    int at = (w & 3) * (D / 32) + (w >> 2);
    if (D == 256) at ^= (r & 1) << 2;
    return r * (D / 2) + 4 * at;
}

RMSN_HD int kv4_v_row(int r) { return (r & 8) + ((r & 7) >> 1) + 4 * (r & 1); }

// Byte offset of the unit with the V codes of dims [g D/8, (g+1) D/8) of token r (g < 8).
RMSN_HD int kv4_v_unit(int D, int r, int g) {
    const int row = kv4_v_row(r);
    if (D == 128) g ^= ((row >> 1) & 1) << 2;
    if (D == 256) g ^= (row & 3) << 1;
    return 8 * D + row * (D / 2) + g * (D / 16);
}

// Byte offsets of the scales of group j of token r; the minimum of K follows its scale, that
// of V is 4 bytes on.
RMSN_HD int kv4_k_scale(int D, int r, int j) { return 16 * D + r * (D / 8) + 4 * j; }
RMSN_HD int kv4_v_scale(int D, int r, int j) {
    return 18 * D + (r >> 1) * (D / 4) + 8 * j + 2 * (r & 1);
}

// Record of head 0 of a slot (slot = page * page_size + offset) that is inside the cache; head h
// is h * blocks_per_page records on.
RMSN_HD int64_t kv4_record_of(int64_t slot, int blocks_per_page, int kv_heads) {
    const int64_t block = slot >> 4;
    const int64_t page = block >> 31 ? block / blocks_per_page
                                     : (int64_t)((uint32_t)block / (uint32_t)blocks_per_page);
    return page * (kv_heads - 1) * blocks_per_page + block;
}

// Record of any slot and head; -1 outside the cache.
RMSN_HD int64_t kv4_record(int64_t slot, int64_t pages, int blocks_per_page, int kv_heads, int h) {
    if (slot < 0 || (slot >> 4) >= pages * blocks_per_page) return -1;
    return kv4_record_of(slot, blocks_per_page, kv_heads) + (int64_t)h * blocks_per_page;
}

}  // namespace rmsn
