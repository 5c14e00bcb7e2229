// rmsn_kv4.cuh -- checked calls on the 4-bit cache (what the entry points hand the launchers).
#pragma once

#include "rmsn_kv4_layout.h"
#include "rmsn_qk.cuh"

namespace rmsn {

struct Kv4Append {
    Heads x[3], y;  // q, k, v; q out
    const void* w[2];
    Rope rope;
    uint8_t* cache;
    const int64_t* slots;
    unsigned* err;
    int64_t tokens, pages;
    int heads, kv_heads, blocks_per_page, D, w_dt, sms;
    bool neighbours;
    float eps;
};

struct Kv4Read {
    const uint8_t* cache;
    const int64_t* slots;
    Heads k, v;
    unsigned* err;
    int64_t tokens, pages;
    int kv_heads, blocks_per_page, D, sms;
};

struct Kv4Attention {
    const void* q;
    int64_t q_st, q_sh, out_st, out_sh;  // strides in elements
    void* out;
    float* lse;
    const uint8_t* cache;
    const int* page_table;
    int64_t table_stride;
    const int* kv_lens;
    const int* cu_q;  // null: one query token per sequence
    void* ws;
    unsigned* err;
    uint64_t limit_ns;
    int64_t pages;
    int tokens, seqs, heads, kv_heads, table_width, blocks_per_page, max_q, D, sms;
    float scale;
};

cudaError_t launch_kv4_append(const Kv4Append& c, cudaStream_t s);
cudaError_t launch_kv4_read(const Kv4Read& c, cudaStream_t s);
cudaError_t launch_kv4_attention(const Kv4Attention& c, cudaStream_t s);
int64_t kv4_attention_workspace(int seqs, int D, int sms);

}  // namespace rmsn
