// Drafted trees over the paged cache: positions and ancestor masks
// (sgmv_tree_tables), the walk along the model's own tokens with the pages past
// it given back (sgmv_tree_accept), and the accepted tokens' keys and values
// moved to their places (sgmv_kv_commit). Attention is kv_attention.hip's.
//
// What bounds them: latency. A step's trees are a few KB; each kernel is a
// chain of dependent reads, so a request's chain is walked in LDS or registers
// and requests go side by side, a workgroup or a wave each. An empty kernel
// takes 1.6 us.
#include "kv_launch.h"
#include "sgmv.h"
#include "sgmv_common.h"

namespace sgmv {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kMaxTree = 32 * SGMV_MAX_TREE_WORDS;

// Request b's rows of the step; b = num_requests: the rows past the last request.
__device__ __forceinline__ void rows_of(const int32_t *q_start, int B, int T, int b, int &lo, int &n) {
    lo = min(max(q_start[b], 0), T);
    const int hi = b < B ? min(max(q_start[b + 1], lo), T) : T;
    n = hi - lo;
}

// ----------------------------------------------------------------------------
// Positions and masks. A token's ancestors have falling indices, so its walk
// up the tree (parents in LDS) meets the words of its mask from the last to
// the first, and each is written once.
// Measured (kernel alone): 64 trees of 26 to 64 tokens 2.8 us; 512 of up to 256
// with 8 words each, 2.7 MB, 4.3 us. These trees are 3 to 10 deep; the walk is
// as long as a token is deep, and a thread's tokens come one after another: 64
// chains of 64 tokens 5.0 us, of 256 15.1, of 1024 140.
// ----------------------------------------------------------------------------
__global__ __launch_bounds__(kThreads) void tree_tables_kernel(TreeTablesArgs a) {
    __shared__ int s_parent[kMaxTree];
    const int b = blockIdx.x, tid = threadIdx.x;
    int q0, n;
    rows_of(a.q_start, a.num_requests, a.T, b, q0, n);
    const bool request = b < a.num_requests;
    const int size = request ? min(n, 32 * a.words) : 0;  // tokens of the tree
    const int first = request ? a.kv_len[b] - n : 0;
    for (int i = tid; i < size; i += kThreads) {
        const int p = a.parent[q0 + i];
        s_parent[i] = p < i ? p : -1;
    }
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
        const int64_t row = q0 + i;
        int at = i < size ? i : -1, depth = -1;
        for (int w = a.words - 1; w >= 0; --w) {
            uint32_t word = 0;
            while (at >= 32 * w) {
                word |= 1u << (at & 31);
                at = s_parent[at];
                ++depth;
            }
            a.mask[row * a.words + w] = word;
        }
        a.position[row] = i < size ? first + depth : -1;
    }
}

// ----------------------------------------------------------------------------
// Acceptance. A wave takes one request: its tree is read once to LDS, then each
// step looks for the first child of the present token that holds the model's
// own next one, 64 candidates at a time (children come after their parents).
// Giving pages back takes sums over all requests, which here would wait for
// every wave, and is a launch of its own.
// Measured (kernel alone): 64 requests of 26 to 64 tokens 4.3 us and 2.7 for
// the pages, 256 of up to 128 tokens 5.2 and 3.2, with 3 to 4 tokens accepted
// each. Every further one is a dependent step of 0.27 us: 64 chains accepted
// whole, of 64 tokens 20 us, of 256 70, of 1024 273.
// ----------------------------------------------------------------------------
struct Walk {
    int parent[kMaxTree], token[kMaxTree], target[kMaxTree];
};

__global__ __launch_bounds__(kThreads) void tree_accept_kernel(AcceptArgs a) {
    __shared__ Walk s_walk[kWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int b = blockIdx.x * kWaves + wave;
    if (b > a.num_requests) return;
    int q0, n;
    rows_of(a.q_start, a.num_requests, a.T, b, q0, n);
    int accepted = 0, next = -1;
    if (b < a.num_requests && n > 0) {
        Walk &t = s_walk[wave];
        const int size = min(n, kMaxTree);
        const bool served = a.slot[q0] >= 0;  // with its tree in one go
        for (int i = lane; i < size; i += 64) {
            const int parent = a.parent[q0 + i], token = a.token[q0 + i], target = a.target[q0 + i];
            t.parent[i] = parent;
            t.token[i] = token;
            t.target[i] = target;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
        __builtin_amdgcn_wave_barrier();
        int cur = 0;
        while (served) {  // cur grows
            next = t.target[cur];
            if (lane == 0) a.path[q0 + accepted] = cur;
            ++accepted;
            int child = size;
            for (int j0 = (cur + 1) & ~63; j0 < size; j0 += 64) {
                const int j = j0 + lane;
                const bool is = j > cur && j < size && t.parent[j] == cur && t.token[j] == next;
                const unsigned long long who = __ballot(is);
                if (who != 0) {
                    child = j0 + __ffsll(who) - 1;
                    break;
                }
            }
            if (child >= size) break;
            cur = child;
        }
    }
    for (int i = accepted + lane; i < n; i += 64) a.path[q0 + i] = -1;
    if (b < a.num_requests && lane == 0) {
        const int kv = a.kv_len[b];
        a.accepted[b] = accepted;
        a.next_token[b] = next;
        a.kept_len[b] = accepted > 0 ? kv - n + accepted : kv;
    }
}

// Pages past the kept tokens go behind the ring's free ones, requests in order: request b's from R_b on, R the prefix
// sum of the pages given back. As in kv_tables.hip every workgroup forms the sums over all requests for itself.
__device__ __forceinline__ int pages_of(const AcceptArgs &a, int len) {
    return (int)min(((int64_t)max(len, 0) + (1 << a.page_shift) - 1) >> a.page_shift, (int64_t)a.max_blocks);
}

__global__ __launch_bounds__(kThreads) void give_back_kernel(AcceptArgs a) {
    __shared__ int s_back[SGMV_MAX_REQUESTS];
    __shared__ int s_wave[kWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, B = a.num_requests, P = a.num_pages;
    const int head = min(max(a.pool_in[0], 0), P - 1), count = min(max(a.pool_in[1], 0), P);
    const int per = (B + kThreads - 1) / kThreads, b0 = min(tid * per, B), b1 = min(b0 + per, B);
    int back = 0;
    for (int b = b0; b < b1; ++b) {
        const int mine = max(pages_of(a, a.kv_len[b]) - pages_of(a, a.kept_len[b]), 0);
        s_back[b] = mine;
        back += mine;
    }
    int to = back;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int x = __shfl_up(to, o);
        to += lane >= o ? x : 0;
    }
    if (lane == 63) s_wave[wave] = to;
    __syncthreads();
    int at = to - back, returned = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        at += w < wave ? s_wave[w] : 0;
        returned += s_wave[w];
    }
    for (int b = b0; b < b1; ++b) {
        const int mine = s_back[b];
        s_back[b] = at;
        at += mine;
    }
    __syncthreads();
    returned = min(returned, P - count);
    if (blockIdx.x == 0 && tid == 0) {
        a.pool_out[0] = head;
        a.pool_out[1] = count + returned;
        a.pool_out[2] = a.pool_in[2];
        a.pool_out[3] = a.pool_in[3];
    }
    for (int f = blockIdx.x * kThreads + tid; f < returned; f += gridDim.x * kThreads) {
        int lo = 0, hi = B;  // the last request with s_back <= f
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s_back[mid] <= f)
                lo = mid;
            else
                hi = mid;
        }
        int to = head + count;
        to = (to >= P ? to - P : to) + f;
        a.free_pages[to >= P ? to - P : to] =
            a.block_table[(int64_t)lo * a.max_blocks + pages_of(a, a.kept_len[lo]) + (f - s_back[lo])];
    }
}

// ----------------------------------------------------------------------------
// Accepted rows to their places: row d of a request becomes row path[d]. A lane
// takes 16 bytes of one layer's heads, of K or of V, and moves them for every d
// in order: since path grows, path[d] >= d, a row is read before it is
// overwritten, and lanes have no bytes in common, so nothing else is waited
// for. Up to kDeep rows are in flight.
// Measured (kernel alone): 64 requests, one layer of 32 heads of 128, 4.4 us
// for some 143 rows that move (4.7 MB); 256 requests, eight layers of 8 heads,
// 570 to 630 rows, 37 to 41 MB read and written, 12.0 us (3.2 TB/s; a copy
// reaches 4.7).
// ----------------------------------------------------------------------------
constexpr int kDeep = 4;

__global__ __launch_bounds__(kThreads) void kv_commit_kernel(CommitArgs a, int vecs, int per_layer, int64_t columns) {
    const int lane = threadIdx.x & 63, b = blockIdx.x;
    int q0, n;
    rows_of(a.q_start, a.num_requests, a.T, b, q0, n);
    const int64_t column = (int64_t)blockIdx.y * kThreads + threadIdx.x;
    const bool on = column < columns;
    const int64_t layer = on ? column / per_layer : 0;
    const int in = on ? (int)(column % per_layer) : 0;
    const int head = in / (2 * vecs), is_v = in / vecs & 1, vec = in % vecs;
    const int size = a.dtype == SGMV_BF16 ? 2 : 4;
    char *base = static_cast<char *>(is_v ? a.V : a.K) + layer * a.layer_stride * size + 16 * vec;
    const auto row = [&](int slot) {
        const int64_t r = ((((int64_t)(slot >> a.page_shift) * a.kv_heads + head) << a.page_shift) + (slot & ((1 << a.page_shift) - 1)));
        return base + r * a.head_dim * size;
    };
    const int cells = a.num_pages << a.page_shift;
    for (int d0 = 0; d0 < n; d0 += 64) {
        const int d = d0 + lane;
        int from = -1, src = -1, dst = -1;
        if (d < n) {
            from = a.path[q0 + d];
            if (from > d && from < n) {
                src = a.slot[q0 + from];
                dst = a.slot[q0 + d];
            }
        }
        const bool move = (unsigned)src < (unsigned)cells && (unsigned)dst < (unsigned)cells;
        unsigned long long moves = __ballot(move);
        while (moves != 0) {
            uint4 x[kDeep];
            char *to[kDeep];
#pragma unroll
            for (int i = 0; i < kDeep; ++i) {
                const int l = moves != 0 ? __ffsll(moves) - 1 : -1;
                const int from_slot = __builtin_amdgcn_readlane(src, max(l, 0)), to_slot = __builtin_amdgcn_readlane(dst, max(l, 0));
                moves &= moves - 1;
                to[i] = nullptr;
                if (l >= 0 && on) {
                    x[i] = ld16(row(from_slot));
                    to[i] = row(to_slot);
                }
            }
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // every row is read before any is written
#pragma unroll
            for (int i = 0; i < kDeep; ++i)
                if (to[i]) st16(to[i], x[i]);
        }
        if (!__any(d + 1 == d0 + 64 && from >= 0)) break;  // the path ends here
    }
}

int commit_vecs(const CommitArgs &a) { return a.head_dim * (a.dtype == SGMV_BF16 ? 2 : 4) / 16; }
int64_t commit_columns(const CommitArgs &a) { return (int64_t)a.num_layers * a.kv_heads * 2 * commit_vecs(a); }

}  // namespace

hipError_t launch_tree_tables(const TreeTablesArgs &a, hipStream_t st) {
    hipLaunchKernelGGL(tree_tables_kernel, dim3(a.num_requests + 1), dim3(kThreads), 0, st, a);
    return hipGetLastError();
}

hipError_t launch_tree_accept(const AcceptArgs &a, hipStream_t st) {
    hipLaunchKernelGGL(tree_accept_kernel, dim3((a.num_requests + kWaves) / kWaves), dim3(kThreads), 0, st, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int blocks = (a.num_requests + kThreads - 1) / kThreads;
    hipLaunchKernelGGL(give_back_kernel, dim3(blocks < 1 ? 1 : blocks), dim3(kThreads), 0, st, a);
    return hipGetLastError();
}

int64_t kv_commit_workgroups(const CommitArgs &a) { return a.num_requests * ((commit_columns(a) + kThreads - 1) / kThreads); }

hipError_t launch_kv_commit(const CommitArgs &a, hipStream_t st) {
    const int64_t columns = commit_columns(a);
    const dim3 grid((unsigned)a.num_requests, (unsigned)((columns + kThreads - 1) / kThreads));
    hipLaunchKernelGGL(kv_commit_kernel, grid, dim3(kThreads), 0, st, a, commit_vecs(a), a.kv_heads * 2 * commit_vecs(a), columns);
    return hipGetLastError();
}

}  // namespace sgmv
