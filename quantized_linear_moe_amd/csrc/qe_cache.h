// Rotary positions, the paged key/value cache, attention over it and the verification of drafted tokens: launch
// wrappers of k_rope.hip, k_attn.hip and k_verify.hip (arguments validated by the caller).
#pragma once

#include "qe_internal.h"

namespace qe {

constexpr int kMaxHeadDim = 256;
constexpr int kVerifyMaxRows = 1024, kVerifyMaxVocab = 1 << 22;

// Heads to rotate or to store: q alone (qe_rope_apply), or keys and values to a cache with or without q
struct RopeLaunch {
    const void* x[3];        // q, k, v (NULL: none); token strides in elements
    int64_t x_stride[3];
    int heads[3];            // of q, k, v
    bool x_bf16;
    int T, head_dim;
    const qe_rope* rope;     // NULL: nothing rotates
    const int32_t* pos;
    void* q_out;
    int64_t q_out_stride;
    bool q_out_bf16;
    const qe_kv_cache* cache;  // NULL without k and v
    const int32_t* slot;
};
hipError_t launch_rope(const RopeLaunch& R, hipStream_t st);

struct AttnPlan {
    bool few_rows;   // all query rows of a sequence and key head in one tile whose waves divide the keys
    int row_tiles;   // query tiles per sequence and key head
    int splits;      // pieces of the keys (1: no partials)
    int chunk;       // keys of a piece
};
AttnPlan attn_plan(const qe_kv_cache* cache, int n_heads, int T, int n_seq, int max_q, int max_kv);
size_t attn_partial_bytes(const AttnPlan& P, int head_dim, int T, int n_heads);

struct AttnLaunch {
    const qe_kv_cache* cache;
    const uint16_t* q;
    int64_t q_stride;
    int T, n_heads, n_seq, max_pages, max_q, max_kv;
    const int32_t *q_start, *kv_len, *pages;
    const uint32_t* tree;
    int tree_words;
    float scale;
    uint16_t* out;
    int64_t out_stride;
    void* ws;
};
hipError_t launch_attention(const AttnLaunch& A, const AttnPlan& P, hipStream_t st);

int verify_chunks(int vocab);
hipError_t launch_verify(const float* p, int64_t p_stride, const float* draft_p, int64_t draft_stride, int vocab,
                         const int32_t* row_start, int n_rows, const int32_t* token, const int32_t* parent,
                         const float* u, int n_seq, int max_rows, int32_t* taken, int32_t* path, int32_t* next, void* ws,
                         hipStream_t st);

}  // namespace qe
