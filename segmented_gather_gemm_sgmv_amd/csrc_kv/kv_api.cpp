// The paged key/value-cache entry points of the C ABI declared in
// include/sgmv.h: argument checks, then the gfx950 kernels.
#include "sgmv.h"

#include <hip/hip_runtime.h>

#include <math.h>

#include "kv_launch.h"
#include "sgmv_checks.h"

using namespace sgmv::abi;

namespace {

int hip_status(hipError_t e) { return e == hipSuccess ? SGMV_OK : SGMV_ERR_HIP; }

// One dispatch holds fewer than 2^32 work-items (its packet has 32 bits for them): 2^24 workgroups of 256 threads are one
// too many.
bool too_many(int64_t workgroups) { return workgroups >= sgmv::kMaxWorkgroups; }

// The exponent of a valid page size, or -1.
int page_shift(int32_t page_size) {
    for (int s = 4; s <= 8; ++s)
        if (page_size == 1 << s) return s;
    return -1;
}

int check_pages(int32_t num_pages, int32_t page_size) {
    if (page_shift(page_size) < 0 || num_pages <= 0 || (int64_t)num_pages * page_size > INT32_MAX)
        return SGMV_ERR_SHAPE;
    return SGMV_OK;
}

bool valid_head(int32_t head_dim) { return head_dim >= 8 && head_dim <= 128 && head_dim % 8 == 0; }
int64_t elem_size(int32_t dtype) { return dtype == SGMV_BF16 ? 2 : 4; }

// Rows of `heads` heads that start `stride` elements apart, T of them.
int check_rows(const void *p, int64_t stride, int32_t heads, int32_t head_dim, int32_t T, int32_t dtype) {
    if (stride < (int64_t)heads * head_dim || (double)stride * T > (double)kMaxElems) return SGMV_ERR_SHAPE;
    if (!aligned16(p) || stride * elem_size(dtype) % 16 != 0) return SGMV_ERR_ALIGN;
    return SGMV_OK;
}

// sgmv_paged_attention and sgmv_tree_attention.
int attention(void *out, int64_t out_stride, float *lse, const void *q, int64_t q_stride, int32_t q_heads,
              const void *K_cache, const void *V_cache, int32_t num_pages, int32_t kv_heads, int32_t page_size,
              int32_t head_dim, const int32_t *block_table, int32_t max_blocks, const int32_t *q_start,
              const int32_t *kv_len, int32_t num_requests, int32_t T, int32_t max_q_len, float scale,
              int32_t window, int32_t sinks, int32_t dtype, const uint32_t *mask, int32_t mask_words, bool tree,
              void *workspace, size_t workspace_bytes, void *stream) {
    if (!valid_dtype(dtype)) return SGMV_ERR_DTYPE;
    if (!valid_head(head_dim) || kv_heads <= 0 || q_heads <= 0 || q_heads % kv_heads != 0) return SGMV_ERR_SHAPE;
    if (num_requests < 0 || num_requests > SGMV_MAX_REQUESTS || T < 0 || T > 1 << 24 || max_q_len < 0 ||
        max_blocks < 0 || window < 0 || sinks < 0)
        return SGMV_ERR_SHAPE;
    // a tree's tokens have a bit each, and see all of their ancestors whatever the window
    if (tree && (mask_words <= 0 || mask_words > SGMV_MAX_TREE_WORDS || max_q_len > 32 * mask_words ||
                 (window > 0 && window < max_q_len)))
        return SGMV_ERR_SHAPE;
    if ((int64_t)T * q_heads > INT32_MAX || (int64_t)max_q_len * q_heads > INT32_MAX) return SGMV_ERR_SHAPE;
    // the kernels number their items, at most these, in 31 bits
    const int64_t rows = (int64_t)(max_q_len < T ? max_q_len : T) * (q_heads / kv_heads);
    if (((rows / 16 + 1) * kv_heads + sgmv::kMostSplits) * num_requests > INT32_MAX) return SGMV_ERR_SHAPE;
    int st = check_pages(num_pages, page_size);
    if (st != SGMV_OK) return st;
    // positions, and the ends of key tiles past them, in 31 bits; and a window past the longest context changes nothing
    const int far = 1 << 30;
    if ((int64_t)max_blocks * page_size > far) return SGMV_ERR_SHAPE;
    if (!(scale > 0.f) || !isfinite(scale)) return SGMV_ERR_SHAPE;
    if (T == 0 || num_requests == 0 || max_q_len == 0) return SGMV_OK;
    if (!out || !q || !K_cache || !V_cache || !q_start || !kv_len || (max_blocks > 0 && !block_table) || (tree && !mask))
        return SGMV_ERR_NULL;
    st = check_rows(q, q_stride, q_heads, head_dim, T, dtype);
    if (st == SGMV_OK) st = check_rows(out, out_stride, q_heads, head_dim, T, dtype);
    if (st != SGMV_OK) return st;
    if (!aligned16(K_cache) || !aligned16(V_cache)) return SGMV_ERR_ALIGN;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ||
        workspace_bytes < sgmv::attention_workspace_bytes(head_dim, dtype))
        return SGMV_ERR_WORKSPACE;
    const sgmv::AttnArgs a{out,       out_stride,   lse,         q,        q_stride,
                           q_heads,   q_heads / kv_heads, K_cache, V_cache, num_pages,
                           kv_heads,  page_shift(page_size), head_dim, block_table, max_blocks,
                           q_start,   kv_len,       num_requests, T,       max_q_len < T ? max_q_len : T,
                           scale,     window < far ? window : far, sinks < far ? sinks : far, dtype, workspace,
                           mask,      mask_words};
    if (too_many(tree ? sgmv::tree_attention_workgroups(a) : sgmv::attention_workgroups(a)))
        return SGMV_ERR_SHAPE;
    const hipStream_t on = static_cast<hipStream_t>(stream);
    return hip_status(tree ? sgmv::launch_tree_attention(a, on) : sgmv::launch_paged_attention(a, on));
}

}  // namespace

extern "C" {

int sgmv_kv_tables(const int32_t *seq_len, const int32_t *new_len, int32_t num_requests, int32_t *block_table,
                   int32_t max_blocks, int32_t page_size, int32_t *free_pages, int32_t num_pages,
                   const int32_t *pool_in, int32_t *pool_out, int32_t *q_start, int32_t *kv_len,
                   int32_t *position, int32_t *slot, int32_t T, void *stream) {
    if (num_requests < 0 || num_requests > SGMV_MAX_REQUESTS || max_blocks < 0 || T < 0) return SGMV_ERR_SHAPE;
    const int st = check_pages(num_pages, page_size);
    if (st != SGMV_OK) return st;
    if ((int64_t)num_requests * T > INT32_MAX || (int64_t)num_requests * max_blocks > INT32_MAX ||
        (int64_t)max_blocks * page_size > INT32_MAX)
        return SGMV_ERR_SHAPE;
    if (!free_pages || !pool_in || !pool_out || !q_start || (T > 0 && (!position || !slot))) return SGMV_ERR_NULL;
    if (num_requests > 0 && (!seq_len || !new_len || !kv_len || (max_blocks > 0 && !block_table)))
        return SGMV_ERR_NULL;
    const sgmv::TablesArgs a{seq_len,    new_len,   num_requests, block_table, max_blocks, page_shift(page_size),
                             free_pages, num_pages, pool_in,      pool_out,    q_start,    kv_len,
                             position,   slot,      T};
    return hip_status(sgmv::launch_kv_tables(a, static_cast<hipStream_t>(stream)));
}

int sgmv_rope_table(float *table, int32_t max_position, int32_t rot_dim, double base, int32_t kind, double factor,
                    double beta_fast, double beta_slow, int32_t original_max, void *stream) {
    if (max_position < 0 || rot_dim <= 0 || rot_dim % 2 != 0 || !(base > 1.0) || !isfinite(base)) return SGMV_ERR_SHAPE;
    if ((int64_t)max_position * rot_dim > kMaxElems) return SGMV_ERR_SHAPE;
    sgmv::RopeTableArgs a{table, max_position, rot_dim / 2, base, kind, 1.0, 0.0, 0.0, 1.0};
    if (kind == SGMV_ROPE_LINEAR || kind == SGMV_ROPE_BY_PARTS) {
        if (!(factor > 0.0) || !isfinite(factor)) return SGMV_ERR_SHAPE;
        a.factor = factor;
    } else if (kind != SGMV_ROPE_PLAIN) {
        return SGMV_ERR_SHAPE;
    }
    if (kind == SGMV_ROPE_BY_PARTS) {
        if (!(beta_slow > 0.0) || !(beta_fast > beta_slow) || !isfinite(beta_fast) || original_max <= 0 ||
            factor < 1.0)
            return SGMV_ERR_SHAPE;
        // The pair that turns n times over original_max positions: f_i * original_max = 2 pi n.
        const double turns = original_max / (2.0 * 3.14159265358979323846);
        const double low = floor(a.half * log(turns / beta_fast) / log(base));
        const double high = ceil(a.half * log(turns / beta_slow) / log(base));
        a.low = fmax(low, 0.0);
        a.high = fmax(fmin(high, rot_dim - 1.0), a.low + 0.001);
        a.magnitude = 0.1 * log(factor) + 1.0;
    }
    if (max_position == 0) return SGMV_OK;
    if (!table) return SGMV_ERR_NULL;
    if (!aligned16(table)) return SGMV_ERR_ALIGN;
    return hip_status(sgmv::launch_rope_table(a, static_cast<hipStream_t>(stream)));
}

int sgmv_rope_append(void *q_out, int64_t q_out_stride, const void *q, int64_t q_stride, int32_t q_heads,
                     const void *k, int64_t k_stride, const void *v, int64_t v_stride, void *K_cache,
                     void *V_cache, int32_t num_pages, int32_t kv_heads, int32_t page_size, int32_t head_dim,
                     const int32_t *position, const int32_t *slot, int32_t T, const float *table,
                     int32_t max_position, int32_t rot_dim, int32_t interleaved, int32_t dtype, void *stream) {
    if (!valid_dtype(dtype)) return SGMV_ERR_DTYPE;
    if (T < 0 || q_heads < 0 || kv_heads < 0 || max_position < 0 || !valid_head(head_dim)) return SGMV_ERR_SHAPE;
    if (rot_dim < 0 || rot_dim > head_dim || rot_dim % 2 != 0) return SGMV_ERR_SHAPE;
    if ((int64_t)q_heads + kv_heads > 65536) return SGMV_ERR_SHAPE;
    int st = kv_heads > 0 ? check_pages(num_pages, page_size) : (int)SGMV_OK;
    if (st != SGMV_OK) return st;
    if (T == 0 || q_heads + kv_heads == 0) return SGMV_OK;
    if (!position || (rot_dim > 0 && !table)) return SGMV_ERR_NULL;
    if (q_heads > 0 && (!q || !q_out)) return SGMV_ERR_NULL;
    if (kv_heads > 0 && (!k || !v || !K_cache || !V_cache || !slot)) return SGMV_ERR_NULL;
    if (rot_dim > 0 && !aligned16(table)) return SGMV_ERR_ALIGN;
    if (q_heads > 0) {
        st = check_rows(q, q_stride, q_heads, head_dim, T, dtype);
        if (st == SGMV_OK) st = check_rows(q_out, q_out_stride, q_heads, head_dim, T, dtype);
        if (st != SGMV_OK) return st;
    }
    if (kv_heads > 0) {
        st = check_rows(k, k_stride, kv_heads, head_dim, T, dtype);
        if (st == SGMV_OK) st = check_rows(v, v_stride, kv_heads, head_dim, T, dtype);
        if (st != SGMV_OK) return st;
        if (!aligned16(K_cache) || !aligned16(V_cache)) return SGMV_ERR_ALIGN;
    }
    const sgmv::RopeArgs a{q_out,     q_out_stride, q,          q_stride,  q_heads,   k,
                           k_stride,  v,            v_stride,   K_cache,   V_cache,   num_pages,
                           kv_heads,  kv_heads > 0 ? page_shift(page_size) : 4, head_dim, position, slot, T,
                           table,     max_position, rot_dim,    interleaved, dtype};
    if (too_many(sgmv::rope_append_workgroups(a))) return SGMV_ERR_SHAPE;
    return hip_status(sgmv::launch_rope_append(a, static_cast<hipStream_t>(stream)));
}

size_t sgmv_paged_attention_workspace_bytes(int32_t head_dim, int32_t dtype) {
    if (!valid_head(head_dim) || !valid_dtype(dtype)) return 0;
    return sgmv::attention_workspace_bytes(head_dim, dtype);
}

int sgmv_paged_attention(void *out, int64_t out_stride, float *lse, const void *q, int64_t q_stride,
                         int32_t q_heads, const void *K_cache, const void *V_cache, int32_t num_pages,
                         int32_t kv_heads, int32_t page_size, int32_t head_dim, const int32_t *block_table,
                         int32_t max_blocks, const int32_t *q_start, const int32_t *kv_len,
                         int32_t num_requests, int32_t T, int32_t max_q_len, float scale, int32_t window,
                         int32_t sinks, int32_t dtype, void *workspace, size_t workspace_bytes, void *stream) {
    return attention(out, out_stride, lse, q, q_stride, q_heads, K_cache, V_cache, num_pages, kv_heads,
                     page_size, head_dim, block_table, max_blocks, q_start, kv_len, num_requests, T, max_q_len,
                     scale, window, sinks, dtype, nullptr, 0, false, workspace, workspace_bytes, stream);
}

int sgmv_tree_attention(void *out, int64_t out_stride, float *lse, const void *q, int64_t q_stride,
                        int32_t q_heads, const void *K_cache, const void *V_cache, int32_t num_pages,
                        int32_t kv_heads, int32_t page_size, int32_t head_dim, const int32_t *block_table,
                        int32_t max_blocks, const int32_t *q_start, const int32_t *kv_len, const uint32_t *mask,
                        int32_t mask_words, int32_t num_requests, int32_t T, int32_t max_q_len, float scale,
                        int32_t window, int32_t sinks, int32_t dtype, void *workspace, size_t workspace_bytes,
                        void *stream) {
    return attention(out, out_stride, lse, q, q_stride, q_heads, K_cache, V_cache, num_pages, kv_heads,
                     page_size, head_dim, block_table, max_blocks, q_start, kv_len, num_requests, T, max_q_len,
                     scale, window, sinks, dtype, mask, mask_words, true, workspace, workspace_bytes, stream);
}

int sgmv_tree_tables(const int32_t *parent, const int32_t *q_start, const int32_t *kv_len, int32_t num_requests,
                     int32_t *position, uint32_t *mask, int32_t mask_words, int32_t T, void *stream) {
    if (num_requests < 0 || num_requests > SGMV_MAX_REQUESTS || T < 0 || T > 1 << 24) return SGMV_ERR_SHAPE;
    if (mask_words <= 0 || mask_words > SGMV_MAX_TREE_WORDS) return SGMV_ERR_SHAPE;
    if (T == 0) return SGMV_OK;
    if (!parent || !q_start || !position || !mask || (num_requests > 0 && !kv_len)) return SGMV_ERR_NULL;
    const sgmv::TreeTablesArgs a{parent, q_start, kv_len, num_requests, T, position, mask, mask_words};
    return hip_status(sgmv::launch_tree_tables(a, static_cast<hipStream_t>(stream)));
}

int sgmv_tree_accept(const int32_t *parent, const int32_t *token, const int32_t *target, const int32_t *slot,
                     const int32_t *q_start, const int32_t *kv_len, int32_t num_requests, int32_t page_size,
                     const int32_t *block_table, int32_t max_blocks, int32_t *free_pages, int32_t num_pages,
                     const int32_t *pool_in, int32_t *pool_out, int32_t *path, int32_t *accepted,
                     int32_t *next_token, int32_t *kept_len, int32_t T, void *stream) {
    if (num_requests < 0 || num_requests > SGMV_MAX_REQUESTS || max_blocks < 0 || T < 0 || T > 1 << 24)
        return SGMV_ERR_SHAPE;
    const int st = check_pages(num_pages, page_size);
    if (st != SGMV_OK) return st;
    if ((int64_t)num_requests * max_blocks > INT32_MAX || (int64_t)max_blocks * page_size > INT32_MAX)
        return SGMV_ERR_SHAPE;
    if (!q_start || !free_pages || !pool_in || !pool_out) return SGMV_ERR_NULL;
    if (T > 0 && (!parent || !token || !target || !slot || !path)) return SGMV_ERR_NULL;
    if (num_requests > 0 && (!kv_len || !accepted || !next_token || !kept_len || (max_blocks > 0 && !block_table)))
        return SGMV_ERR_NULL;
    const sgmv::AcceptArgs a{parent,      token,      target,     slot,      q_start, kv_len,   num_requests, T,
                             page_shift(page_size), block_table, max_blocks, free_pages, num_pages, pool_in, pool_out, path,
                             accepted,    next_token, kept_len};
    return hip_status(sgmv::launch_tree_accept(a, static_cast<hipStream_t>(stream)));
}

int sgmv_kv_commit(void *K_cache, void *V_cache, int32_t num_layers, int64_t layer_stride, int32_t num_pages,
                   int32_t kv_heads, int32_t page_size, int32_t head_dim, const int32_t *slot,
                   const int32_t *q_start, const int32_t *path, int32_t num_requests, int32_t T, int32_t dtype,
                   void *stream) {
    if (!valid_dtype(dtype)) return SGMV_ERR_DTYPE;
    if (!valid_head(head_dim) || kv_heads <= 0 || kv_heads > 65536 || num_layers < 0) return SGMV_ERR_SHAPE;
    if (num_requests < 0 || num_requests > SGMV_MAX_REQUESTS || T < 0 || T > 1 << 24) return SGMV_ERR_SHAPE;
    const int st = check_pages(num_pages, page_size);
    if (st != SGMV_OK) return st;
    const double layer = (double)num_pages * page_size * kv_heads * head_dim;
    if (num_layers > 1 && ((double)layer_stride < layer || (double)layer_stride * num_layers > (double)kMaxElems))
        return SGMV_ERR_SHAPE;
    if (num_layers == 0 || num_requests == 0 || T == 0) return SGMV_OK;
    if (!K_cache || !V_cache || !slot || !q_start || !path) return SGMV_ERR_NULL;
    if (!aligned16(K_cache) || !aligned16(V_cache) || (num_layers > 1 && layer_stride * elem_size(dtype) % 16 != 0))
        return SGMV_ERR_ALIGN;
    const sgmv::CommitArgs a{K_cache,  V_cache, num_layers, num_layers > 1 ? layer_stride : 0, num_pages, kv_heads,
                             page_shift(page_size), head_dim, dtype, slot, q_start, path, num_requests, T};
    const int64_t groups = sgmv::kv_commit_workgroups(a);
    if (too_many(groups) || groups / num_requests > 65535) return SGMV_ERR_SHAPE;
    return hip_status(sgmv::launch_kv_commit(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
