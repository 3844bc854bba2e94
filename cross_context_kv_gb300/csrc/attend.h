// attend.h -- the arguments of one kvfix_shared_attend or kvfix_tree_attend call, as the kernels take them.
#pragma once

#include "pool.cuh"

namespace kvfix {

struct AttendArgs {
    const uint16_t* q;
    Plane qp;  // chunks = agents, tokens = new_tokens, heads = q_heads
    uint16_t* out;
    Plane op;
    float* lse;  // [agents][new_tokens][q_heads], or null
    PoolView pool;
    int agents, new_tokens, q_heads, groups, page;
    int max_prefix_pages, max_suffix_pages;
    const int32_t* prefix_pages;  // [groups][max_prefix_pages]
    const int32_t* prefix_len;    // [groups]
    const int32_t* group_begin;   // [groups + 1]
    const int32_t* suffix_pages;  // [agents][max_suffix_pages]
    const int32_t* suffix_len;    // [agents]
    float scale_log2;             // softmax scale times log2 e
    void* workspace;
    // kvfix_tree_attend
    const uint32_t* tree;  // [agents][new_tokens][tree_words], or null: new tokens see all before them
    const int32_t* nodes;  // [agents], or null: new_tokens each
    int tree_words;
};

size_t attend_workspace_bytes(int agents, int new_tokens, int q_heads, int kv_heads, int head_dim, int groups);
cudaError_t launch_attend(const AttendArgs& a, cudaStream_t s);

}  // namespace kvfix
