/*
 * sgmv.h — C ABI of the MI355X (gfx950) SGMV library.
 *
 * SGMV itself comes first; the paged key/value cache that a serving layer
 * needs next to it (block tables, rotary write, attention), the drafted trees
 * over it, and tokens under several adapters each have their own parts below.
 *
 * SGMV (segmented gather matrix-vector multiplication) applies many LoRA
 * adapters to one batch in one pass. The batch's rows are grouped into
 * contiguous segments; segment s covers rows seg_start[s] .. seg_start[s+1]-1
 * and uses adapter k = seg_adapter[s] from a pool reached through a table of
 * pointers. For every row m of segment s:
 *
 *     V[m, :] = X[m, :] . A_k                         (shrink, d_in -> r)
 *     Y[m, :] = Y[m, :] + (alpha / r) * V[m, :] . B_k  (expand, r -> d_out)
 *
 * Sources (Punica guide, aifetchly blog): the per-row LoRA equation for y_i
 * in section "The Heterogeneous Batching Bottleneck" (delta added to the base
 * output, scaled by alpha / r, A_k of logical shape d_in x r, B_k of logical
 * shape r x d_out); the segment offsets S = {s_0 .. s_N} and the pointer
 * array of section "The SGMV Mathematical Formulation"; the single kernel
 * that takes X and the pointers to A and B (figure "Punica: SGMV"); the two
 * launches per layer, one for all A and one for all B (section "Mathematical
 * Modeling", equation 2).
 *
 * Conventions shared by every call
 * --------------------------------
 * dtype        SGMV_F32 or SGMV_BF16. X, Y and every adapter share it. V is
 *              always fp32. Arithmetic accumulates in fp32; Y is rounded once,
 *              to nearest-even, when stored.
 * precision    bf16 segments of 16 rows or more expand on matrix cores, where
 *              each fp32 V value enters as the sum of two bf16 values,
 *              hi = rne(v) and lo = rne(v - hi): 16 significant bits, a
 *              relative error of at most 2^-16 per value (exact for integer
 *              V with |V| < 2^16). The expand error of such a row is then at
 *              most (alpha / r) * 2^-16 * sum_j |V[m, j]| |B_k(j, n)| beyond
 *              fp32 accumulation and the final rounding. Every other product
 *              takes its operands exactly.
 * X            device, row-major M x d_in, contiguous, 16-byte aligned.
 * Y            device, row-major M x d_out, contiguous, 16-byte aligned;
 *              read and written (the delta is added to what Y holds).
 * V            device, row-major M x r fp32, contiguous, 16-byte aligned.
 * A_ptrs       device array of num_adapters 64-bit device addresses. Entry k
 *              points to A_k stored as r rows of d_in elements: logical
 *              element (i, j) of A_k sits at j * d_in + i. 16-byte aligned.
 * B_ptrs       device array of num_adapters addresses. Entry k points to B_k
 *              stored as r rows of d_out elements: (j, n) at j * d_out + n.
 * seg_start    device int32[num_segments + 1], non-decreasing, with
 *              seg_start[0] = 0 and seg_start[num_segments] = M.
 * seg_adapter  device int32[num_segments], each in [0, num_adapters).
 * r            8, 16, 32 or 64.
 * d_in, d_out  positive multiples of 8.
 * stream       a hipStream_t (NULL = the default stream). Every call is
 *              asynchronous and stream-ordered: it only enqueues kernels, makes
 *              no host<->device copy and no synchronisation.
 *
 * Ownership: the caller owns every buffer and must keep it alive until the
 * stream work completes. The library allocates no memory and keeps no pointer
 * after a call returns.
 *
 * Errors: every call returns SGMV_OK (0) or a negative status; no call
 * aborts. Arguments are checked on the host before anything is enqueued; on
 * error nothing is enqueued. M == 0 or num_segments == 0 is a successful
 * no-op. Device-resident metadata cannot be checked without a
 * synchronisation, so the kernels defend themselves instead: segment bounds
 * are clamped into [0, M] (a decreasing pair is an empty segment) and a
 * segment whose adapter id lies outside [0, num_adapters) is skipped (its rows
 * are left as they were). Nothing outside the documented buffers is read or
 * written for any metadata values, and every kernel ends.
 *
 * Failures seen on the device (calls with a workspace): offsets that
 * decrease somewhere let two segments share rows; the values of such rows
 * are then unspecified, and the call sets SGMV_WS_BAD_OFFSETS in the
 * workspace's status word. Workgroups that wait for one another do so for a
 * bounded number of polls (sgmv_set_wait_limit); a wait that gives up leaves
 * its rows unchanged and sets SGMV_WS_WAIT_TIMEOUT. Either bit means the
 * workspace may hold leftovers: every later call on it does nothing (its
 * outputs are left as they were) until the caller zero-fills the workspace
 * again. sgmv_workspace_status reads the word.
 */
#ifndef SGMV_H
#define SGMV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum sgmv_dtype { SGMV_F32 = 0, SGMV_BF16 = 1 };

enum sgmv_status {
    SGMV_OK = 0,
    SGMV_ERR_NULL = -1,      /* a required pointer is NULL */
    SGMV_ERR_SHAPE = -2,     /* negative size, d not a multiple of 8, or too large */
    SGMV_ERR_RANK = -3,      /* r not in {8, 16, 32, 64} */
    SGMV_ERR_DTYPE = -4,     /* dtype not SGMV_F32 / SGMV_BF16 */
    SGMV_ERR_ALIGN = -5,     /* an operand (or a row of it) not 16-byte aligned */
    SGMV_ERR_WORKSPACE = -6, /* workspace missing or smaller than sgmv_workspace_bytes */
    SGMV_ERR_HIP = -7,       /* the HIP runtime reported an error at launch */
    SGMV_ERR_ADAPTER = -8,   /* host metadata: an adapter id that is negative (or outside the pool) */
    SGMV_ERR_SCRATCH = -9    /* sgmv_fused_noalloc: the batch needs more than SGMV_NOALLOC_SCRATCH_BYTES */
};

/*
 * Shrink (Punica guide, "The SGMV Mathematical Formulation": one launch for
 * every segment; "Mathematical Modeling" eq. 2: the launch for all A).
 * V[m, j] = sum_i X[m, i] * A_k(i, j) for every row m of every segment.
 * V is overwritten for rows that lie in a segment with a valid adapter, and
 * left untouched elsewhere.
 *
 * workspace: as for sgmv_fused (same size query, same zero-filled contract).
 * Long bf16 segments split the reduction over d_in between workgroups and
 * combine the parts there, in a fixed order. May be NULL with
 * workspace_bytes = 0 when sgmv_workspace_bytes(...) is 0.
 */
int sgmv_shrink(float *V, const void *X, const uint64_t *A_ptrs, int32_t num_adapters,
                const int32_t *seg_start, const int32_t *seg_adapter, int32_t num_segments,
                int32_t M, int32_t d_in, int32_t r, int32_t dtype, void *workspace,
                size_t workspace_bytes, void *stream);

/*
 * Expand (same sources; the launch for all B, and the equation for y_i: the
 * delta, scaled by alpha / r, is added to the base output).
 * Y[m, n] += (alpha / r) * sum_j V[m, j] * B_k(j, n). The scale alpha / r is
 * formed once in fp32.
 */
int sgmv_expand(void *Y, const float *V, const uint64_t *B_ptrs, int32_t num_adapters,
                const int32_t *seg_start, const int32_t *seg_adapter, int32_t num_segments,
                int32_t M, int32_t d_out, int32_t r, float alpha, int32_t dtype, void *stream);

/*
 * Fused shrink + expand in one launch (Punica guide, figure "Punica: SGMV":
 * one kernel call over X and the pointers to A and B).
 * Y[m, :] += (alpha / r) * X[m, :] . A_k . B_k. The intermediate V lives in
 * the workspace and is not returned. Same result as sgmv_shrink followed by
 * sgmv_expand, up to fp32 summation order.
 *
 * workspace: device memory of at least sgmv_workspace_bytes(...) bytes,
 * 256-byte aligned, zero-filled before its first use (for example by
 * hipMemset once after allocating it). Every call leaves the bytes it uses
 * all zero again when its kernel completes, so one workspace serves any later
 * call on the same stream, of any size that fits, without clearing. Calls
 * that overlap in time (different streams) must use different workspaces.
 */
int sgmv_fused(void *Y, const void *X, const uint64_t *A_ptrs, const uint64_t *B_ptrs,
               int32_t num_adapters, const int32_t *seg_start, const int32_t *seg_adapter,
               int32_t num_segments, int32_t M, int32_t d_in, int32_t d_out, int32_t r,
               float alpha, int32_t dtype, void *workspace, size_t workspace_bytes,
               void *stream);

/*
 * sgmv_fused without a workspace argument and without any allocation: for
 * callers that cannot allocate device memory (code under HIP graph capture,
 * tight serving loops, harnesses that forbid hipMalloc).
 *
 * Same arguments (minus the workspace), result and errors as sgmv_fused. The
 * workspace is a static array of SGMV_NOALLOC_SCRATCH_BYTES inside the
 * library, one per GPU (each GPU the call runs on holds its copy until the
 * process ends); a batch whose fused workspace (sgmv_workspace_bytes) is
 * larger is rejected with SGMV_ERR_SCRATCH and nothing is enqueued. The
 * stream must belong to the current device. Each call first enqueues a
 * one-workgroup kernel that zero-fills the array if an earlier call left a
 * failure status in it (otherwise earlier calls left it zero), then the
 * fused kernel. All calls on one GPU share the array: calls that overlap in
 * time on that GPU (different streams, or different threads) race and must
 * not be made; calls on one stream are ordered and safe. No hipMalloc,
 * hipFree or allocating library routine is called.
 */
#define SGMV_NOALLOC_SCRATCH_BYTES ((size_t)16 << 20)

int sgmv_fused_noalloc(void *Y, const void *X, const uint64_t *A_ptrs, const uint64_t *B_ptrs,
                       int32_t num_adapters, const int32_t *seg_start, const int32_t *seg_adapter,
                       int32_t num_segments, int32_t M, int32_t d_in, int32_t d_out, int32_t r,
                       float alpha, int32_t dtype, void *stream);

/*
 * Gathered forms: the batch stays in token order (Punica guide, figure "CUDA
 * Threadblock Tiling": the block of a segment gathers that segment's rows of
 * activations; section "Hardware-Level Optimizations in SGMV": grouping the
 * requests by adapter, which these calls do through an index instead of
 * moving X and Y).
 *
 * rows         device int32[M]: segment row p (p in [0, M), in segment order
 *              exactly as seg_start describes it for the calls above) is
 *              token row rows[p] of X and of Y. Normally the perm that
 *              sgmv_build_segments returns, i.e. a permutation of [0, M).
 * X, Y         token order, M rows each (same layout as above).
 * V            segment order: V row p belongs to token rows[p], as in the
 *              calls above.
 *
 * Each call computes what its contiguous counterpart computes on the batch
 * gathered into segment order, with Y's rows put back at their tokens:
 *     V[p, :]       = X[rows[p], :] . A_k                       (shrink_gather)
 *     Y[rows[p], :] += (alpha / r) * V[p, :] . B_k             (expand_scatter)
 *     Y[rows[p], :] += (alpha / r) * X[rows[p], :] . A_k . B_k  (fused_gather)
 * Arguments, workspace, errors and the device-side defences are those of
 * the contiguous call, plus: rows must not be NULL when M > 0. An entry of
 * rows outside [0, M) makes segment row p absent: no Y row is written for
 * it and V row p is unspecified (X is then read at row 0, never outside X).
 * If two entries name the same token, that token's Y row is unspecified
 * (the writes race); nothing outside the buffers is touched.
 */
int sgmv_shrink_gather(float *V, const void *X, const int32_t *rows, const uint64_t *A_ptrs,
                       int32_t num_adapters, const int32_t *seg_start, const int32_t *seg_adapter,
                       int32_t num_segments, int32_t M, int32_t d_in, int32_t r, int32_t dtype,
                       void *workspace, size_t workspace_bytes, void *stream);

int sgmv_expand_scatter(void *Y, const float *V, const int32_t *rows, const uint64_t *B_ptrs,
                        int32_t num_adapters, const int32_t *seg_start, const int32_t *seg_adapter,
                        int32_t num_segments, int32_t M, int32_t d_out, int32_t r, float alpha,
                        int32_t dtype, void *stream);

int sgmv_fused_gather(void *Y, const void *X, const int32_t *rows, const uint64_t *A_ptrs,
                      const uint64_t *B_ptrs, int32_t num_adapters, const int32_t *seg_start,
                      const int32_t *seg_adapter, int32_t num_segments, int32_t M, int32_t d_in,
                      int32_t d_out, int32_t r, float alpha, int32_t dtype, void *workspace,
                      size_t workspace_bytes, void *stream);

/*
 * Layer-batched fused call: every projection of one batch in one launch
 * (Punica guide, "Mathematical Modeling", equation 2: the execution latency
 * of a layer counts its launches, one per adapter matrix; here one per layer,
 * whatever the number of projections).
 *
 * For every projection q < num_projections, with p = projections[q]:
 *     p.Y[m, :] += (alpha / r) * p.X[m, :] . A_k . B_k
 * where A_k and B_k come from p's own pools (p.A_ptrs, p.B_ptrs, each of
 * p.num_adapters entries) and k is the adapter of m's segment. All
 * projections share the batch: M rows, the segments (seg_start,
 * seg_adapter), r, alpha and dtype; each has its own d_in and d_out, and X
 * and Y of the layouts above (p.X: M x p.d_in, p.Y: M x p.d_out). The
 * result is that of one sgmv_fused call per projection.
 *
 * rows         NULL: X and Y in segment order. Otherwise the token-order
 *              index of the gathered calls above, shared by every projection.
 * projections  host array of num_projections descriptors, read during the
 *              call only (the library keeps no pointer to it).
 * num_projections  0 .. SGMV_MAX_PROJECTIONS (0 is a no-op).
 * workspace    at least sgmv_layer_workspace_bytes(...) bytes, 256-byte
 *              aligned, zero-filled before first use; every call leaves it
 *              zero again (as for sgmv_fused).
 * The Y buffers of different projections must not overlap. Errors and
 * device-side defences as for sgmv_fused, checked for every projection;
 * num_projections outside [0, SGMV_MAX_PROJECTIONS] is SGMV_ERR_SHAPE.
 */
#define SGMV_MAX_PROJECTIONS 8

typedef struct sgmv_projection {
    void *Y;
    const void *X;
    const uint64_t *A_ptrs;
    const uint64_t *B_ptrs;
    int32_t num_adapters;
    int32_t d_in;
    int32_t d_out;
} sgmv_projection;

int sgmv_fused_layer(const sgmv_projection *projections, int32_t num_projections, const int32_t *rows,
                     const int32_t *seg_start, const int32_t *seg_adapter, int32_t num_segments, int32_t M,
                     int32_t r, float alpha, int32_t dtype, void *workspace, size_t workspace_bytes,
                     void *stream);

/* Workspace bytes sgmv_fused_layer needs (0 on invalid arguments). */
size_t sgmv_layer_workspace_bytes(const sgmv_projection *projections, int32_t num_projections,
                                  int32_t num_segments, int32_t M, int32_t r, int32_t dtype);

/* Bytes of workspace sgmv_shrink and sgmv_fused need for these sizes; one
 * buffer of this size serves both (0 on invalid sizes, or when neither needs
 * any). The gathered forms need the same. */
size_t sgmv_workspace_bytes(int32_t num_segments, int32_t M, int32_t d_in, int32_t d_out,
                            int32_t r, int32_t dtype);

/*
 * Host-side segment metadata (Punica guide, "Hardware-Level Optimizations in
 * SGMV": requests are grouped by adapter so that each adapter's rows are
 * contiguous; "The SGMV Mathematical Formulation": the offsets s_0 .. s_N).
 *
 * token_adapter: host int32[M], the adapter of each token, each >= 0.
 * perm:          host int32[M], out: the stable sort of token indices by
 *                adapter id; row p of the segmented batch is token perm[p].
 * seg_start:     host int32[M + 1], out: the first *num_segments + 1 entries
 *                are the segment offsets (seg_start[0] = 0, last = M).
 * seg_adapter:   host int32[M], out: the first *num_segments entries are the
 *                segments' adapter ids, strictly increasing.
 * num_segments:  host int32, out: the number of distinct adapters.
 * Returns SGMV_ERR_ADAPTER if an id is negative, SGMV_ERR_NULL / _SHAPE on
 * bad arguments. Runs in O(M log M) on the calling thread.
 */
int sgmv_build_segments(const int32_t *token_adapter, int32_t M, int32_t *perm,
                        int32_t *seg_start, int32_t *seg_adapter, int32_t *num_segments);

/*
 * Host-side check of segment metadata before it is copied to the device
 * (the conditions the calls above state for seg_start and seg_adapter; the
 * Punica guide, "The SGMV Mathematical Formulation": offsets s_0 .. s_N
 * that cover the batch, one adapter per segment).
 *
 * seg_start    host int32[num_segments + 1]; seg_adapter host int32[num_segments].
 * Returns SGMV_OK if seg_start[0] == 0, seg_start[num_segments] == M, the
 * offsets never decrease, and every id lies in [0, num_adapters);
 * SGMV_ERR_SHAPE for a bad offset (or negative sizes), SGMV_ERR_ADAPTER for
 * an id outside the pool, SGMV_ERR_NULL for a missing array. Reads only.
 */
int sgmv_check_segments(const int32_t *seg_start, const int32_t *seg_adapter, int32_t num_segments,
                        int32_t M, int32_t num_adapters);

/*
 * Adapter pool pointer table (Punica guide, figure "SGMV Kernel Memory
 * Layout": an array of pointers, each to one adapter's contiguous memory;
 * section "Core Innovation 2": one unified device buffer holds the hot
 * adapters). Fills ptrs_host[k] = base + k * slot_bytes for k < num_adapters,
 * for a pool whose slots are packed back to back. The caller copies the table
 * to the device. Tables for scattered slots may be filled by the caller
 * directly with any 16-byte aligned device addresses.
 */
int sgmv_pool_pointers(uint64_t *ptrs_host, const void *base, int32_t num_adapters,
                       int64_t slot_bytes);

/*
 * Adapter admission (Punica guide, "Core Innovation 2": the hot adapters live
 * in one unified device pool, and a cold one is copied in from host memory
 * on demand, in under 1.5 ms per adapter over the host link).
 *
 * Enqueues on `stream`, in this order: the copy of A_bytes from A_host to
 * the device slot A_slot, the copy of B_bytes from B_host to B_slot, and the
 * update A_ptrs[slot] = A_slot, B_ptrs[slot] = B_slot (a one-workgroup
 * kernel). An SGMV call enqueued after it on the same stream uses the new
 * adapter; one enqueued before it uses the old entries. The caller keeps
 * A_host and B_host unchanged until the copies complete; with pinned host
 * memory (hipHostMalloc) the call returns at once, with pageable memory the
 * runtime may finish the copy before returning.
 *
 * A_slot, B_slot  device memory of A_bytes / B_bytes, 16-byte aligned: A_k
 *                 as r rows of d_in, B_k as r rows of d_out (the layout above).
 * slot            0 <= slot < num_adapters (the table length).
 * Returns SGMV_ERR_NULL, _SHAPE (slot out of range, zero bytes), _ALIGN or
 * _HIP; nothing is enqueued on error.
 */
int sgmv_admit_adapter(void *A_slot, void *B_slot, const void *A_host, const void *B_host,
                       size_t A_bytes, size_t B_bytes, uint64_t *A_ptrs, uint64_t *B_ptrs,
                       int32_t slot, int32_t num_adapters, void *stream);

/*
 * Measurement helper, not part of SGMV: a streaming read of `bytes` bytes at
 * `src` (device, 16-byte aligned, bytes a multiple of 16) by `num_blocks`
 * workgroups of 256 threads, 16-byte loads, each workgroup writing the XOR
 * of the 32-bit words it read to sink[block] (device uint32[num_blocks]).
 * It gives the HBM rate a plain kernel reaches for a given size, the
 * ceiling the SGMV kernels are compared with. Returns SGMV_ERR_NULL,
 * _SHAPE or _ALIGN on bad arguments.
 */
int sgmv_stream_probe(const void *src, size_t bytes, uint32_t *sink, int32_t num_blocks, void *stream);

/*
 * Workspace status (the sticky word at the start of every workspace, see
 * "Failures seen on the device" above): 0 while every call on the workspace
 * succeeded, else the OR of the bits below.
 */
enum sgmv_ws_status {
    SGMV_WS_WAIT_TIMEOUT = 1, /* a bounded wait between workgroups gave up */
    SGMV_WS_BAD_OFFSETS = 2   /* seg_start decreases somewhere */
};

/*
 * Reads the status word of `workspace` (a workspace of sgmv_shrink,
 * sgmv_fused, the gathered calls or sgmv_fused_layer) into *status after
 * every call enqueued before it on `stream` has completed: it synchronises
 * the stream. A non-zero status stays until the caller zero-fills the
 * workspace (all of it: the failed call may have left leftovers anywhere in
 * it). Returns SGMV_ERR_NULL, or SGMV_ERR_HIP if the copy or the
 * synchronisation failed.
 */
int sgmv_workspace_status(const void *workspace, uint32_t *status, void *stream);

/*
 * Sets how many times a workgroup polls for another's result before it gives
 * up (default 32768, several milliseconds at the least); applies to calls
 * launched afterwards (a captured graph keeps the value it was captured
 * with). Process-wide; returns the previous value. 0 makes every wait give
 * up unless its result is there at the first poll: a way to test the failure
 * path from the host.
 */
uint32_t sgmv_set_wait_limit(uint32_t polls);

/* ---------------------------------------------------------------------------
 * The paged key/value cache between a layer's q/k/v and o projections
 * ---------------------------------------------------------------------------
 * What runs between the projections SGMV adapts: the step's tokens get cache
 * slots (sgmv_kv_tables, once per step), q and k are rotated and k and v
 * written to the cache (sgmv_rope_append, per layer), and the step's queries
 * attend to the cache (sgmv_paged_attention, per layer).
 *
 * K_cache, V_cache  device, [num_pages][kv_heads][page_size][head_dim],
 *               contiguous, 16-byte aligned: one head of one page is one run
 *               of memory.
 * page_size     16, 32, 64, 128 or 256; num_pages * page_size < 2^31.
 * head_dim      a positive multiple of 8, at most 128.
 * block_table   device int32[num_requests][max_blocks]: entry [b][i] is the
 *               page of positions i * page_size ... of request b.
 * q_start       device int32[num_requests + 1], non-decreasing from 0: request
 *               b's new tokens are rows q_start[b] .. q_start[b+1]-1 of the
 *               step's T rows.
 * kv_len        device int32[num_requests]: tokens of request b in the cache,
 *               its new ones included. New token i of n is at position
 *               kv_len[b] - n + i.
 * slot          device int32[T]: page * page_size + offset in the page, or a
 *               negative value for a token that has none.
 * q, k, v       rows of heads, [T][heads][head_dim] with a row stride in
 *               elements (rows may be slices of one fused projection's
 *               output); rows start 16-byte aligned.
 * Streams, ownership and errors are as above: nothing is allocated, nothing
 * synchronises, and no device-resident value makes a kernel read or write
 * outside the documented buffers. Page ids outside [0, num_pages) are never
 * followed (what such an entry's positions hold is then unspecified). */

/*
 * Block tables and slots of one step, built on the device from the requests'
 * lengths. For request b with seq_len[b] cached tokens:
 *   new_len[b] >= 0  adds that many tokens. Pages it needs beyond the ones it
 *                    has are taken from the ring of free pages, requests in
 *                    order, and entered in its row of block_table.
 *   new_len[b] < 0   the request has ended: its pages go back to the ring (for
 *                    later calls), and its length becomes 0.
 * A request whose pages do not fit what is free, or its row of block_table,
 * is refused: it gets no page and no slot and keeps its length. Requests are
 * served in order until one does not fit; after it only those that need no
 * page are. (One too long for its row of block_table takes no part in this.)
 * The tokens of a refused request keep their rows of the step (in q_start and
 * position) and have slot -1, the sign of it on the device. What the step's
 * other calls write to these rows has no meaning (sgmv_paged_attention takes
 * them to be at the end of the old length); offer them again in a later step.
 *
 * free_pages   device int32[num_pages], a ring of the free pages' ids.
 * pool_in      device int32[4]: [0] the ring's first free entry (in
 *              [0, num_pages)), [1] the number of free pages.
 * pool_out     device int32[4]: the same after the call, [2] the number of
 *              requests refused, [3] the step's tokens (q_start's last).
 * q_start      out; kv_len out: the lengths after the step.
 * position     out, int32[T]: each token's position, -1 past the last token.
 * slot         out, int32[T]: each token's slot, -1 where it has none.
 * The outputs must not overlap the inputs (the next call's seq_len and
 * pool_in are this one's kv_len and pool_out: keep two of each). Calling
 * twice with the same inputs and the same free_pages and block_table gives
 * the same result. num_requests: at most SGMV_MAX_REQUESTS.
 */
#define SGMV_MAX_REQUESTS 8192

int sgmv_kv_tables(const int32_t *seq_len, const int32_t *new_len, int32_t num_requests, int32_t *block_table,
                   int32_t max_blocks, int32_t page_size, int32_t *free_pages, int32_t num_pages,
                   const int32_t *pool_in, int32_t *pool_out, int32_t *q_start, int32_t *kv_len,
                   int32_t *position, int32_t *slot, int32_t T, void *stream);

/*
 * Rotary table: table[p][i] = (cos, sin) of position p's angle for pair i,
 * float[max_position][rot_dim / 2][2], formed in 64 bits and rounded once.
 * With inverse frequencies f_i = base^(-2i / rot_dim), the angle is
 *   SGMV_ROPE_PLAIN     p * f_i
 *   SGMV_ROPE_LINEAR    p * f_i / factor (positions interpolated)
 *   SGMV_ROPE_BY_PARTS  p * (f_i * w_i + f_i / factor * (1 - w_i)) (YaRN, Peng
 *                       et al. 2023): w_i falls linearly from 1 to 0 in i
 *                       between the pairs that turn beta_fast and beta_slow
 *                       times over original_max positions, and cos and sin are
 *                       multiplied by 0.1 ln(factor) + 1.
 * For SGMV_ROPE_PLAIN the scaling fields are not read.
 */
enum sgmv_rope_kind { SGMV_ROPE_PLAIN = 0, SGMV_ROPE_LINEAR = 1, SGMV_ROPE_BY_PARTS = 2 };

int sgmv_rope_table(float *table, int32_t max_position, int32_t rot_dim, double base, int32_t kind,
                    double factor, double beta_fast, double beta_slow, int32_t original_max, void *stream);

/*
 * Rotates the first rot_dim elements of every head of q and k by their
 * token's position and writes k and v to the cache:
 *     (a, b) -> (a cos - b sin, b cos + a sin)
 * with pairs (x[i], x[i + rot_dim/2]), or (x[2i], x[2i+1]) when interleaved.
 * Elements past rot_dim, and v, are copied. Arithmetic is fp32, rounded once.
 *
 * q_out        out, [T][q_heads][head_dim] with its own row stride; may be q.
 * table        of sgmv_rope_table; not read (may be NULL) when rot_dim is 0.
 * rot_dim      even, 0 .. head_dim (multiples of 16 in bf16 and of 8 in fp32 move
 *              16 bytes at a time, others less).
 * position     device int32[T]; a token whose position is outside
 *              [0, max_position) is left out (nothing of it is written).
 * slot         device int32[T]; a token without a slot (or one outside the
 *              cache) has its q rotated, and no k and v written.
 * q, q_out     may be NULL with q_heads = 0; k and v may be NULL with
 *              kv_heads = 0 (then the cache and slot may be too).
 * Two tokens must not have one slot.
 */
int sgmv_rope_append(void *q_out, int64_t q_out_stride, const void *q, int64_t q_stride, int32_t q_heads,
                     const void *k, int64_t k_stride, const void *v, int64_t v_stride, void *K_cache,
                     void *V_cache, int32_t num_pages, int32_t kv_heads, int32_t page_size, int32_t head_dim,
                     const int32_t *position, const int32_t *slot, int32_t T, const float *table,
                     int32_t max_position, int32_t rot_dim, int32_t interleaved, int32_t dtype, void *stream);

/*
 * Attention of the step's new tokens over the paged cache (which holds them
 * already). Query head h of a token at position p reads cached head
 * h / (q_heads / kv_heads) and sees key j of its request when
 *     0 <= j <= p,  and with window > 0 also  j > p - window  or  j < sinks:
 * a sliding window, with the first `sinks` tokens always visible.
 *     out = sum_j w_j V_j / sum_j w_j,   w_j = exp(scale * q . K_j)
 *     lse = log(sum_j w_j)
 * A row that sees no key gets out = 0 and lse = -infinity. A key that a row
 * does not see changes nothing of that row, whatever it holds. Rows of no
 * request are left as they were.
 *
 * Products accumulate in fp32 and the softmax's running maximum, sum and
 * output are fp32; out is rounded once. With bf16 the weights enter the second
 * product as two bf16 values each (16 significant bits).
 * Results do not depend on timing.
 *
 * out          [T][q_heads][head_dim] with its own row stride.
 * lse          device float[T][q_heads], or NULL.
 * q_heads      a multiple of kv_heads.
 * max_q_len    at least the largest number of new tokens of a request (the
 *              first max_q_len of more are computed).
 * scale        positive and finite. window, sinks: >= 0.
 * max_blocks   max_blocks * page_size at most 2^30.
 * workspace    as sgmv_paged_attention_workspace_bytes says for the same
 *              sizes, 256-byte aligned. Its first SGMV_ATTENTION_COUNTER_BYTES
 *              are counters: zero before its first use, and zero again after
 *              every call. Not to be shared with the calls above or between
 *              calls that overlap in time, replays of a captured call among
 *              them.
 */
#define SGMV_ATTENTION_COUNTER_BYTES 8192

int sgmv_paged_attention(void *out, int64_t out_stride, float *lse, const void *q, int64_t q_stride,
                         int32_t q_heads, const void *K_cache, const void *V_cache, int32_t num_pages,
                         int32_t kv_heads, int32_t page_size, int32_t head_dim, const int32_t *block_table,
                         int32_t max_blocks, const int32_t *q_start, const int32_t *kv_len,
                         int32_t num_requests, int32_t T, int32_t max_q_len, float scale, int32_t window,
                         int32_t sinks, int32_t dtype, void *workspace, size_t workspace_bytes, void *stream);

/* Workspace bytes of sgmv_paged_attention (0 on invalid arguments); the same
 * for every batch of the layout. */
size_t sgmv_paged_attention_workspace_bytes(int32_t head_dim, int32_t dtype);

/* ---------------------------------------------------------------------------
 * Drafted trees
 * ---------------------------------------------------------------------------
 * A step may verify a tree of drafted tokens per request instead of adding a
 * run of them. The step's tables are the same (sgmv_kv_tables gives every
 * drafted token a slot, in the order of its rows); what differs is where its
 * tokens are and what they see, and that most of them go again:
 *   sgmv_tree_tables     once: positions (by depth) and masks, then
 *   sgmv_rope_append     per layer, with these positions,
 *   sgmv_tree_attention  per layer;
 *   sgmv_tree_accept     once the model's own tokens are known: the drafted
 *                        ones it agrees with, lengths, pages given back,
 *   sgmv_kv_commit       the accepted tokens' keys and values to their places
 *                        (all layers), before the next step's sgmv_kv_tables.
 *
 * parent        device int32[T]: for new token i of a request (row q_start[b]
 *               + i) the index of its parent among the request's new tokens,
 *               less than i. Any other value makes it a root: it follows the
 *               cached tokens directly. Token 0 is the one that the model
 *               chose last; the others are drafted.
 * mask          device uint32[T][mask_words]: bit m % 32 of word m / 32 is the
 *               request's new token m, set where this token sees it.
 * mask_words    1 .. SGMV_MAX_TREE_WORDS; a tree has at most 32 * mask_words
 *               tokens.
 * Streams, ownership, errors and what is promised for any device-resident
 * values are as above.
 */
#define SGMV_MAX_TREE_WORDS 32

/*
 * Positions and masks of one step's trees, q_start and kv_len being those of
 * sgmv_kv_tables (kv_len with the new tokens): a token's position is
 * kv_len[b] - n + its depth, a root's depth being 0, and its mask holds its
 * ancestors and itself. Tokens past a request's first 32 * mask_words, and
 * rows past the last request, have position -1 and an empty mask.
 *
 * position     out, int32[T]. mask: out.
 */
int sgmv_tree_tables(const int32_t *parent, const int32_t *q_start, const int32_t *kv_len, int32_t num_requests,
                     int32_t *position, uint32_t *mask, int32_t mask_words, int32_t T, void *stream);

/*
 * sgmv_paged_attention with masks in the place of the causal order. With
 * c = kv_len[b] - n cached tokens before the step, a token sees key j < c when
 * window is 0, or j > p - window, or j < sinks, where p = c - 1 + the number
 * of new tokens it sees (its position in a tree), and key c + m (m < n) when
 * bit m of its mask is set. Any bits may be set, also of tokens behind it. A
 * row that sees nothing gets out = 0 and lse = -infinity.
 *
 * Everything else, the workspace too, is as for sgmv_paged_attention, and:
 * mask_words   32 * mask_words at least max_q_len.
 * window       0, or at least max_q_len (a window then holds every drafted
 *              token of a branch).
 */
int sgmv_tree_attention(void *out, int64_t out_stride, float *lse, const void *q, int64_t q_stride,
                        int32_t q_heads, const void *K_cache, const void *V_cache, int32_t num_pages,
                        int32_t kv_heads, int32_t page_size, int32_t head_dim, const int32_t *block_table,
                        int32_t max_blocks, const int32_t *q_start, const int32_t *kv_len, const uint32_t *mask,
                        int32_t mask_words, int32_t num_requests, int32_t T, int32_t max_q_len, float scale,
                        int32_t window, int32_t sinks, int32_t dtype, void *workspace, size_t workspace_bytes,
                        void *stream);

/*
 * Verification. With target[i] the model's own token after new token i (its
 * most likely one, or one sampled from its distribution: the accepted tokens
 * then follow that distribution), the accepted tokens of a request are token
 * 0 and, from an accepted token i on, its first child j (parent[j] = i) with
 * token[j] = target[i], until there is none.
 *   path        out, int32[T]: row q_start[b] + d holds the index of request
 *               b's accepted token d, -1 past the last one (and in rows past
 *               the last request).
 *   accepted    out, int32[num_requests]: how many.
 *   next_token  out, int32[num_requests]: target of the last accepted token,
 *               token 0 of the request's next step; -1 where there is none.
 *   kept_len    out, int32[num_requests]: kv_len[b] - n + accepted[b].
 * Of a request without new tokens, or that sgmv_kv_tables refused (its tokens
 * have no slot), nothing is accepted, and its length stays. At most the first
 * 32 * SGMV_MAX_TREE_WORDS tokens of a request are looked at.
 *
 * Every request of the step is verified, one that adds a run of tokens (a
 * prompt, or a chunk of one) too. To keep a run whole give it as a chain,
 * parent[i] = i - 1, with target[i] = token[i + 1] for all of its tokens but
 * the last; it is then no longer than a tree, 32 * mask_words tokens, and a
 * longer prompt goes in several steps or in one without trees.
 *
 * Pages that hold none of the kept_len[b] tokens go back behind the free ones
 * of the ring, requests in order. block_table is left as it is (sgmv_kv_commit
 * goes by slot, and entries past a request's length have no meaning to the
 * other calls).
 *
 * token, target   device int32[T], any values. slot, q_start, kv_len: of the
 *              step's sgmv_kv_tables (its outputs).
 * free_pages, pool_in, pool_out   as for sgmv_kv_tables, pool_in being the
 *              step's pool_out; pool_out[2] and [3] are pool_in's.
 * The outputs must not overlap the inputs; calling twice with the same inputs
 * gives the same result.
 */
int sgmv_tree_accept(const int32_t *parent, const int32_t *token, const int32_t *target, const int32_t *slot,
                     const int32_t *q_start, const int32_t *kv_len, int32_t num_requests, int32_t page_size,
                     const int32_t *block_table, int32_t max_blocks, int32_t *free_pages, int32_t num_pages,
                     const int32_t *pool_in, int32_t *pool_out, int32_t *path, int32_t *accepted,
                     int32_t *next_token, int32_t *kept_len, int32_t T, void *stream);

/*
 * Moves the accepted tokens' keys and values to where a plain step would have
 * written them: the row at slot[q_start[b] + d] becomes what the one at
 * slot[q_start[b] + path[q_start[b] + d]] held, in K_cache and V_cache and in
 * every layer. path is that of sgmv_tree_accept: it grows within a request
 * (entries that are less than their own index move nothing) and ends at its
 * first -1; slot and q_start are the step's. Once per step: a second call
 * would move rows again.
 *
 * K_cache, V_cache   num_layers caches each, layer_stride elements apart
 *              (not read when num_layers is 1).
 */
int sgmv_kv_commit(void *K_cache, void *V_cache, int32_t num_layers, int64_t layer_stride, int32_t num_pages,
                   int32_t kv_heads, int32_t page_size, int32_t head_dim, const int32_t *slot,
                   const int32_t *q_start, const int32_t *path, int32_t num_requests, int32_t T, int32_t dtype,
                   void *stream);

/* ---------------------------------------------------------------------------
 * Several adapters per token
 * ---------------------------------------------------------------------------
 * The grouping that sgmv_build_segments does on the host, on the device and
 * for a number of adapters per token, each with a weight (a mixture of
 * adapters, whose router chose them):
 *     Y[t] = base[t] + sum_j weight[t][j] * F_k(X[t]),  k = choice[t][j]
 * is sgmv_sort_tokens, sgmv_spread_rows (Xs, the rows in segment order), the
 * SGMV calls on Xs for Ys (cleared first), and sgmv_combine_rows. With one
 * adapter per token order is the index that the gathered calls take, and no
 * row need be moved.
 *
 * The gradients, given dY: of weight and of Ys, sgmv_combine_rows_grad; of Xs,
 * the SGMV calls on dYs with A_ptrs and B_ptrs exchanged (the adapters stay as
 * they are); of X, sgmv_combine_rows on dXs without weights, which is the
 * gradient of sgmv_spread_rows; of base, dY.
 *
 * choice        device int32[T][choices]: adapters; one outside
 *               [0, num_adapters) is no choice.
 * place         device int32[T][choices]: the choice's row in segment order,
 *               a negative value for none. Rows outside [0, rows) are never
 *               followed.
 * weight        device float[T][choices], or NULL: all 1.
 * Xs, Ys, dYs, dXs   `rows` rows of d elements, in segment order.
 * X, Y, base, dY, dX   T rows of d elements, in token order.
 * Row strides are in elements; rows start 16-byte aligned. d is a positive
 * multiple of 8, choices 1 .. SGMV_MAX_CHOICES, T * choices at most 2^24. A
 * launch has fewer than 2^24 workgroups (one per token in the gradient, and one
 * per token and 4 KB of its row in the others where a row has more than 512
 * bytes): a call that needs more is refused with SGMV_ERR_SHAPE. Sums are fp32,
 * in the order of the choices, and rounded once. Streams, ownership, errors and what is
 * promised for any device-resident values are as above.
 */
#define SGMV_MAX_CHOICES 64
#define SGMV_MAX_SORTED_ADAPTERS 4096

/*
 * Sorts the T * choices choices by adapter, those of one adapter in their
 * order (by token, then by choice).
 *   order        out, int32[T * choices]: row i in segment order is choice
 *                order[i] % choices of token order[i] / choices; -1 past the
 *                last row.
 *   place        out, int32[T][choices]: the inverse, -1 for no choice.
 *   seg_start    out, int32[num_segments + 1], seg_adapter: out,
 *                int32[num_segments]: one segment per adapter that was chosen,
 *                adapters rising; segments past the last are empty, with
 *                adapter 0, and seg_start's last entry is the number of rows.
 * num_adapters  0 .. SGMV_MAX_SORTED_ADAPTERS.
 * num_segments  at least the smaller of num_adapters and T * choices.
 * workspace     at least sgmv_sort_tokens_workspace_bytes(...), 16-byte
 *               aligned; what it holds before and after has no meaning. May be
 *               NULL where that is 0. T * choices: at most 2^24.
 */
int sgmv_sort_tokens(const int32_t *choice, int32_t T, int32_t choices, int32_t num_adapters, int32_t *seg_start,
                     int32_t *seg_adapter, int32_t num_segments, int32_t *order, int32_t *place, void *workspace,
                     size_t workspace_bytes, void *stream);

/* Workspace bytes of sgmv_sort_tokens (0 on invalid arguments, and where it
 * needs none). */
size_t sgmv_sort_tokens_workspace_bytes(int32_t T, int32_t choices, int32_t num_adapters);

/* Xs[place[t][j]] = X[t]. Rows of Xs that no choice has are left as they were;
 * one that two choices have (sgmv_sort_tokens gives each its own) holds
 * either's. Xs must not overlap X. */
int sgmv_spread_rows(void *Xs, int64_t Xs_stride, int32_t rows, const void *X, int64_t X_stride,
                     const int32_t *place, int32_t T, int32_t choices, int32_t d, int32_t dtype, void *stream);

/* Y[t] = base[t] + sum_j weight[t][j] * Ys[place[t][j]]. base: NULL (then 0),
 * Y itself or rows of its own; Y must not overlap Ys. Choices without a row
 * add nothing, whatever their weight. */
int sgmv_combine_rows(void *Y, int64_t Y_stride, const void *base, int64_t base_stride, const void *Ys,
                      int64_t Ys_stride, int32_t rows, const int32_t *place, const float *weight, int32_t T,
                      int32_t choices, int32_t d, int32_t dtype, void *stream);

/* dYs[place[t][j]] = weight[t][j] * dY[t], and dweight[t][j] = dY[t] .
 * Ys[place[t][j]] (0 for a choice without a row). dYs or dweight may be NULL;
 * without dweight Ys may be NULL, without dYs weight is not read. Rows of dYs
 * that no choice has are left as they were; one that two choices have holds
 * either's, which is then not the gradient (the sum of both). dYs must not
 * overlap dY or Ys. */
int sgmv_combine_rows_grad(void *dYs, int64_t dYs_stride, float *dweight, const void *dY, int64_t dY_stride,
                           const void *Ys, int64_t Ys_stride, int32_t rows, const int32_t *place,
                           const float *weight, int32_t T, int32_t choices, int32_t d, int32_t dtype,
                           void *stream);

/* A static, human-readable name for a status code. */
const char *sgmv_status_string(int status);

/* Library version, major * 10000 + minor * 100 + patch. */
int sgmv_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SGMV_H */
