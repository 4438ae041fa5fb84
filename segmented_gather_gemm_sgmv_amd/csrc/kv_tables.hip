// Block tables and slots of one serving step, on the device (sgmv_kv_tables).
//
// Mathematics: with L_b cached and n_b new tokens, request b has
// h_b = ceil(L_b / page) pages and needs d_b = ceil((L_b + n_b) / page) - h_b
// more. Its pages are entries [D_b, D_b + d_b) of the ring of free pages, D
// the exclusive prefix sum of d; it is served when D_b + d_b fits what is
// free. Its tokens are rows [N_b, N_b + n_b), N the prefix sum of n. An ended
// request's h_b pages go behind the free ones, from R_b on, R the prefix sum
// of h over the ended.
//
// What bounds it: latency. A step's tables are a few hundred KB at most, and
// the work is a chain: lengths, three prefix sums, then independent writes.
// One launch does it all: every workgroup forms the same prefix sums over all
// requests in its own LDS (a read of 8 bytes per request, from L2 after the
// first workgroup) and writes its share of the tokens, fresh entries and
// returned pages, so nothing waits for another workgroup. That is also why
// the outputs have buffers of their own.
#include "kv_launch.h"

namespace sgmv {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxBlocks = 512;
constexpr int kFew = 2048;              // requests up to which the smaller LDS image serves

// Exclusive prefix sums of three values per thread over the workgroup, and
// their totals.
struct Three {
    int x, y, z;
};

__device__ __forceinline__ Three operator+(Three a, Three b) { return {a.x + b.x, a.y + b.y, a.z + b.z}; }
__device__ __forceinline__ Three operator-(Three a, Three b) { return {a.x - b.x, a.y - b.y, a.z - b.z}; }

__device__ __forceinline__ Three block_scan(Three v, Three &total, Three *s_wave) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    Three incl = v;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const Three up = {__shfl_up(incl.x, o), __shfl_up(incl.y, o), __shfl_up(incl.z, o)};
        if (lane >= o) incl = incl + up;
    }
    if (lane == 63) s_wave[wave] = incl;
    __syncthreads();
    Three before = {0, 0, 0};
    total = {0, 0, 0};
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        if (w < wave) before = before + s_wave[w];
        total = total + s_wave[w];
    }
    return before + incl - v;
}

struct Request {
    int seq, add;      // cached and new tokens
    int have, need;    // pages: held, and to be taken
    bool ended, fits;  // fits: its row of block_table is long enough
};

// Lengths are clamped so that no prefix sum passes 31 bits: a request holds at
// most max_blocks pages, adds at most T tokens, and needs more pages only if
// its row has room for them (the entry point bounds num_requests times each).
__device__ __forceinline__ Request request(const TablesArgs &a, int b) {
    const int page = 1 << a.page_shift;
    const int64_t room = (int64_t)a.max_blocks << a.page_shift;
    Request r;
    const int n = a.new_len[b];
    r.seq = max(a.seq_len[b], 0);
    r.ended = n < 0;
    r.add = min(max(n, 0), a.T);
    r.have = (int)min(((int64_t)r.seq + page - 1) >> a.page_shift, (int64_t)a.max_blocks);
    r.fits = (int64_t)r.seq + r.add <= room;
    r.need = r.ended || !r.fits ? 0 : (int)(((int64_t)r.seq + r.add + page - 1) >> a.page_shift) - r.have;
    return r;
}

// The last index i in [0, n) with start[i] <= at; start[0] <= at.
__device__ __forceinline__ int owner(const int *start, int n, int at) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= at)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

template <int kMax>
__global__ __launch_bounds__(kThreads) void kv_tables_kernel(TablesArgs a) {
    __shared__ int s_tok[kMax], s_need[kMax], s_back[kMax];
    __shared__ Three s_wave[kWaves];
    __shared__ int s_taken, s_refused;
    const int tid = threadIdx.x, B = a.num_requests, P = a.num_pages;
    const int head = min(max(a.pool_in[0], 0), P - 1), count = min(max(a.pool_in[1], 0), P);

    // Prefix sums, a block of kThreads requests at a time.
    Three base = {0, 0, 0};
    if (tid == 0) s_taken = s_refused = 0;
    for (int b0 = 0; b0 < B; b0 += kThreads) {
        const int b = b0 + tid;
        Request r = {0, 0, 0, 0, false, true};
        if (b < B) r = request(a, b);
        Three total;
        const Three ex = base + block_scan({r.add, r.need, r.ended ? r.have : 0}, total, s_wave);
        if (b < B) {
            s_tok[b] = ex.x;
            s_need[b] = ex.y;
            s_back[b] = ex.z;
            const bool granted = !r.ended && r.fits && (r.need == 0 || ex.y + r.need <= count);
            if (granted && r.need > 0) atomicMax(&s_taken, ex.y + r.need);
            if (blockIdx.x == 0) {
                a.q_start[b] = ex.x;
                a.kv_len[b] = r.ended ? 0 : r.seq + (granted ? r.add : 0);
                if (!r.ended && !granted) atomicAdd(&s_refused, 1);
            }
        }
        base = base + total;
        __syncthreads();
    }
    __syncthreads();
    const int tokens = base.x, fresh = s_taken, back = min(base.z, P - count);
    if (blockIdx.x == 0 && tid == 0) {
        a.q_start[B] = tokens;
        const int h = head + fresh;
        a.pool_out[0] = h >= P ? h - P : h;
        a.pool_out[1] = count - fresh + back;
        a.pool_out[2] = s_refused;
        a.pool_out[3] = tokens;
    }

    const int stride = gridDim.x * kThreads, first = blockIdx.x * kThreads + tid;
    for (int t = first; t < a.T; t += stride) {
        int pos = -1, slot = -1;
        if (t < tokens) {
            const int b = owner(s_tok, B, t);
            const Request r = request(a, b);
            pos = (int)((unsigned)r.seq + (unsigned)(t - s_tok[b]));
            const int block = pos >> a.page_shift, nth = block - r.have;
            const bool granted = r.fits && (r.need == 0 || s_need[b] + r.need <= count);
            if (granted) {
                int cell;
                if (nth >= 0) {
                    const int at = head + s_need[b] + nth;
                    cell = a.free_pages[at >= P ? at - P : at];
                } else {
                    cell = a.block_table[(int64_t)b * a.max_blocks + block];
                }
                if ((unsigned)cell < (unsigned)P) slot = (cell << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
            }
        }
        a.position[t] = pos;
        a.slot[t] = slot;
    }
    for (int f = first; f < fresh; f += stride) {
        const int b = owner(s_need, B, f), at = head + f;
        const Request r = request(a, b);
        a.block_table[(int64_t)b * a.max_blocks + r.have + (f - s_need[b])] = a.free_pages[at >= P ? at - P : at];
    }
    for (int f = first; f < back; f += stride) {
        const int b = owner(s_back, B, f);
        int at = head + count;
        at = at >= P ? at - P : at;
        at += f;
        a.free_pages[at >= P ? at - P : at] = a.block_table[(int64_t)b * a.max_blocks + (f - s_back[b])];
    }
}

}  // namespace

hipError_t launch_kv_tables(const TablesArgs &a, hipStream_t st) {
    // A token per thread: its chain of lookups (request, lengths, page) is then walked once, all tokens' at a time.
    int blocks = (a.T + kThreads - 1) / kThreads;
    const int by_requests = (a.num_requests + kThreads / 4 - 1) / (kThreads / 4);
    blocks = blocks > by_requests ? blocks : by_requests;
    blocks = blocks < 1 ? 1 : blocks > kMaxBlocks ? kMaxBlocks : blocks;
    if (a.num_requests <= kFew)
        hipLaunchKernelGGL((kv_tables_kernel<kFew>), dim3(blocks), dim3(kThreads), 0, st, a);
    else
        hipLaunchKernelGGL((kv_tables_kernel<8192>), dim3(blocks), dim3(kThreads), 0, st, a);
    return hipGetLastError();
}

}  // namespace sgmv
