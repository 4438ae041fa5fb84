// Internal interface between the paged-cache entry points (kv_api.cpp) and
// their kernels (kv_tables.hip, kv_rope.hip, kv_attention.hip). Not
// installed; callers use include/sgmv.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace sgmv {

struct TablesArgs {
    const int32_t *seq_len, *new_len;
    int num_requests;
    int32_t *block_table;
    int max_blocks, page_shift;
    int32_t *free_pages;
    int num_pages;
    const int32_t *pool_in;
    int32_t *pool_out, *q_start, *kv_len, *position, *slot;
    int T;
};

struct RopeTableArgs {
    float *table;
    int max_position, half;
    double base;
    int kind;
    double factor, low, high, magnitude;  // by parts: pairs up to `low` keep their frequency, from `high` on none
};

struct RopeArgs {
    void *q_out;
    int64_t q_out_stride;
    const void *q;
    int64_t q_stride;
    int q_heads;
    const void *k;
    int64_t k_stride;
    const void *v;
    int64_t v_stride;
    void *K, *V;
    int num_pages, kv_heads, page_shift, head_dim;
    const int32_t *position, *slot;
    int T;
    const float *table;
    int max_position, rot_dim, interleaved, dtype;
};

struct AttnArgs {
    void *out;
    int64_t out_stride;
    float *lse;
    const void *q;
    int64_t q_stride;
    int q_heads, group;  // group: query heads per cached head
    const void *K, *V;
    int num_pages, kv_heads, page_shift, head_dim;
    const int32_t *block_table;
    int max_blocks;
    const int32_t *q_start, *kv_len;
    int num_requests, T, max_q_len;
    float scale;
    int window, sinks, dtype;
    void *workspace;
};

// Partial-result slots of a launch: no launch splits its groups into more parts.
constexpr int kMostSplits = 1024;

// Workspace of sgmv_paged_attention: counters first, then the partial-result
// slots of the launch that splits the most.
size_t attention_workspace_bytes(int head_dim, int dtype);

int64_t attention_workgroups(const AttnArgs &a);  // of its launch

hipError_t launch_kv_tables(const TablesArgs &a, hipStream_t st);
hipError_t launch_rope_table(const RopeTableArgs &a, hipStream_t st);
int64_t rope_append_workgroups(const RopeArgs &a);
hipError_t launch_rope_append(const RopeArgs &a, hipStream_t st);
hipError_t launch_paged_attention(const AttnArgs &a, hipStream_t st);

}  // namespace sgmv
