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
// the outputs have buffers of their own. The scans run over a wave's lanes by
// lane shifts, and each thread handles about one token, entry or page.
//
// Measured (kernel alone): 64 requests of one token 3.0 us, 512 mixed ones
// with some 33000 tokens 5.4 us; an empty kernel takes 1.6. With shuffles
// through LDS and four tokens per thread they took 3.7 and 12.2 us.
#include "kv_launch.h"

namespace sgmv {

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kFew = 2048;        // requests up to which their lengths stay in LDS too
constexpr int kMaxBlocks = 512;

struct Request {
    int seq, add;      // cached and new tokens
    int have, need;    // pages: held, and to be taken
    bool ended, fits;  // fits: its row of block_table is long enough
};

// Lengths are clamped so that no prefix sum passes 31 bits: a request holds at
// most max_blocks pages, adds at most T tokens, and needs more pages only if
// its row has room for them (the entry point bounds num_requests times each).
__device__ __forceinline__ Request request(const TablesArgs &a, int seq_len, int new_len) {
    const int page = 1 << a.page_shift;
    const int64_t room = (int64_t)a.max_blocks << a.page_shift;
    Request r;
    r.seq = max(seq_len, 0);
    r.ended = new_len < 0;
    r.add = min(max(new_len, 0), a.T);
    r.have = (int)min(((int64_t)r.seq + page - 1) >> a.page_shift, (int64_t)a.max_blocks);
    r.fits = (int64_t)r.seq + r.add <= room;
    r.need = r.ended || !r.fits ? 0 : (int)(((int64_t)r.seq + r.add + page - 1) >> a.page_shift) - r.have;
    return r;
}

// Inclusive prefix sum over a wave's lanes.
template <int kCtrl, int kRowMask>
__device__ __forceinline__ int shifted(int v) {
    return __builtin_amdgcn_update_dpp(0, v, kCtrl, kRowMask, 0xf, false);
}
__device__ __forceinline__ int wave_scan(int v) {
    v += shifted<0x111, 0xf>(v);  // the lane 1, 2, 4, 8 below, within rows of 16 lanes
    v += shifted<0x112, 0xf>(v);
    v += shifted<0x114, 0xf>(v);
    v += shifted<0x118, 0xf>(v);
    v += shifted<0x142, 0xa>(v);  // row 0's last lane to row 1, row 2's to row 3
    v += shifted<0x143, 0xc>(v);  // lane 31 to rows 2 and 3
    return v;
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
    constexpr bool kKeep = kMax <= kFew;
    __shared__ int s_tok[kMax], s_need[kMax], s_back[kMax];
    __shared__ int s_seq[kKeep ? kMax : 1], s_new[kKeep ? kMax : 1];
    __shared__ int s_wave[kWaves][3], s_taken[kWaves], s_refused[kWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, B = a.num_requests, P = a.num_pages;
    const int head = min(max(a.pool_in[0], 0), P - 1), count = min(max(a.pool_in[1], 0), P);
    const auto get = [&](int b) {
        if constexpr (kKeep) return request(a, s_seq[b], s_new[b]);
        return request(a, a.seq_len[b], a.new_len[b]);
    };

    // Prefix sums of tokens, pages needed and pages returned; thread t has requests [t * per, (t + 1) * per).
    const int per = (B + kThreads - 1) / kThreads, b0 = min(tid * per, B), b1 = min(b0 + per, B);
    int tok = 0, need = 0, back = 0;
    for (int b = b0; b < b1; ++b) {
        const int seq = a.seq_len[b], add = a.new_len[b];
        if constexpr (kKeep) {
            s_seq[b] = seq;
            s_new[b] = add;
        }
        const Request r = request(a, seq, add);
        tok += r.add;
        need += r.need;
        back += r.ended ? r.have : 0;
    }
    const int tok_to = wave_scan(tok), need_to = wave_scan(need), back_to = wave_scan(back);
    if (lane == 63) {
        s_wave[wave][0] = tok_to;
        s_wave[wave][1] = need_to;
        s_wave[wave][2] = back_to;
    }
    __syncthreads();
    tok = tok_to - tok;
    need = need_to - need;
    back = back_to - back;
    int tokens = 0, returned = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        if (w < wave) {
            tok += s_wave[w][0];
            need += s_wave[w][1];
            back += s_wave[w][2];
        }
        tokens += s_wave[w][0];
        returned += s_wave[w][2];
    }
    int taken = 0, refused = 0;
    for (int b = b0; b < b1; ++b) {
        const Request r = get(b);
        s_tok[b] = tok;
        s_need[b] = need;
        s_back[b] = back;
        const bool granted = !r.ended && r.fits && (r.need == 0 || need + r.need <= count);
        if (blockIdx.x == 0) {
            a.q_start[b] = tok;
            a.kv_len[b] = r.ended ? 0 : r.seq + (granted ? r.add : 0);
        }
        if (granted && r.need > 0) taken = need + r.need;  // grows with b
        refused += !r.ended && !granted;
        tok += r.add;
        need += r.need;
        back += r.ended ? r.have : 0;
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) taken = max(taken, __shfl_xor(taken, o));
    refused = wave_scan(refused);
    if (lane == 63) {
        s_taken[wave] = taken;
        s_refused[wave] = refused;
    }
    __syncthreads();
    int fresh = 0;
    refused = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        fresh = max(fresh, s_taken[w]);
        refused += s_refused[w];
    }
    returned = min(returned, P - count);
    if (blockIdx.x == 0 && tid == 0) {
        a.q_start[B] = tokens;
        const int h = head + fresh;
        a.pool_out[0] = h >= P ? h - P : h;
        a.pool_out[1] = count - fresh + returned;
        a.pool_out[2] = refused;
        a.pool_out[3] = tokens;
    }

    // Tokens, then the fresh entries of block_table, then the returned pages: one at a time per thread.
    const int64_t all = (int64_t)a.T + fresh + returned;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + tid; i < all; i += (int64_t)gridDim.x * kThreads) {
        if (i < a.T) {
            const int t = (int)i;
            int pos = -1, slot = -1;
            if (t < tokens) {
                const int b = owner(s_tok, B, t);
                const Request r = get(b);
                pos = (int)((unsigned)r.seq + (unsigned)(t - s_tok[b]));
                const int block = pos >> a.page_shift, nth = block - r.have;
                if (r.fits && (r.need == 0 || s_need[b] + r.need <= count)) {
                    const int at = head + s_need[b] + nth;
                    const int cell = nth >= 0 ? a.free_pages[at >= P ? at - P : at]
                                              : a.block_table[(int64_t)b * a.max_blocks + block];
                    if ((unsigned)cell < (unsigned)P) slot = (cell << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
                }
            }
            a.position[t] = pos;
            a.slot[t] = slot;
        } else if (i - a.T < fresh) {
            const int f = (int)(i - a.T), b = owner(s_need, B, f), at = head + f;
            a.block_table[(int64_t)b * a.max_blocks + get(b).have + (f - s_need[b])] = a.free_pages[at >= P ? at - P : at];
        } else {
            const int f = (int)(i - a.T) - fresh, b = owner(s_back, B, f);
            int at = head + count;
            at = (at >= P ? at - P : at) + f;
            a.free_pages[at >= P ? at - P : at] = a.block_table[(int64_t)b * a.max_blocks + (f - s_back[b])];
        }
    }
}

}  // namespace

hipError_t launch_kv_tables(const TablesArgs &a, hipStream_t st) {
    // About one token, entry or page per thread: its chain of lookups (request, lengths, page) is then walked once,
    // all of them at a time.
    const int64_t about = (int64_t)a.T + (a.T >> a.page_shift) + a.num_requests;
    const int64_t want = (about + kThreads - 1) / kThreads;
    const int blocks = (int)(want < 1 ? 1 : want > kMaxBlocks ? kMaxBlocks : want);
    if (a.num_requests <= kFew)
        hipLaunchKernelGGL((kv_tables_kernel<kFew>), dim3(blocks), dim3(kThreads), 0, st, a);
    else
        hipLaunchKernelGGL((kv_tables_kernel<8192>), dim3(blocks), dim3(kThreads), 0, st, a);
    return hipGetLastError();
}

}  // namespace sgmv
