// Choices sorted by adapter, on the device (sgmv_sort_tokens).
//
// Mathematics: a stable counting sort. With c[k] choices of adapter k and
// C[k] = c[0] + .. + c[k-1], the i-th choice of adapter k (in the choices'
// order) goes to row C[k] + i. A wave takes 64 choices at a time: lanes with
// the same adapter find each other by ballots over the bits of its number, so
// a lane's rank among them is a count of bits, and their first lane alone
// moves the adapter's running count; nothing depends on the order of atomics.
//
// What bounds it: latency. Up to kOneBlock choices one workgroup does it all;
// beyond, workgroups count a run of choices each (to the workspace), and a
// second launch, in which every workgroup adds the others' counts up for
// itself, places them. A wave keeps what it found out about its choices, eight
// steps of 64 at most, from counting them to placing them.
//
// Measured (kernels alone): 128 choices of 64 adapters 3.3 us; 18332 of 2000
// 4.7 and 9.7 (25.9 with the workgroups' counts read one after another, 18 trips
// to memory that other XCDs wrote; they are read 16 at a time).
#include "route_launch.h"
#include "sgmv.h"
#include "sgmv_common.h"

namespace sgmv {

namespace {

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / kWave;
constexpr int kSteps = 8;                       // of 64 choices that a wave keeps
constexpr int kOneBlock = kSteps * kThreads;    // choices that one workgroup sorts by itself
constexpr int kMaxBlocks = 64;
constexpr int kRun = 2 * kThreads;  // choices per workgroup, at least, where there are several

constexpr int kBinsEach = 4;  // neighbouring adapters that a thread adds up: 16 bytes of every workgroup's counts

// Counts of one workgroup in the workspace.
__host__ __device__ __forceinline__ int stride_of(int num_adapters) { return (num_adapters + kBinsEach - 1) / kBinsEach * kBinsEach; }

struct Split {
    int blocks, run;  // run: choices per workgroup, a multiple of kThreads
};
Split split_of(int n) {
    if (n <= kOneBlock) return {1, (n + kThreads - 1) / kThreads * kThreads};
    int run = (n + kMaxBlocks - 1) / kMaxBlocks;
    run = (run < kRun ? kRun : run + kThreads - 1) / kThreads * kThreads;
    return {(n + run - 1) / run, run};
}

// Lanes of the wave whose key is this lane's, of those that have one (key >= 0).
__device__ __forceinline__ unsigned long long same_key(int key, int bits) {
    unsigned long long m = __ballot(key >= 0);
    for (int b = 0; b < bits; ++b) {
        const bool one = key >> b & 1;
        const unsigned long long ones = __ballot(one);
        m &= one ? ones : ~ones;
    }
    return m;
}

__device__ __forceinline__ int key_of(const SortArgs &a, int i, int end) {
    if (i >= end) return -1;
    const int k = a.choice[i];
    return (unsigned)k < (unsigned)a.num_adapters ? k : -1;
}

__device__ __forceinline__ unsigned long long lanes_below(int lane) { return (1ull << lane) - 1; }

// LDS operations of one wave complete in order; this only keeps the compiler from moving them across.
__device__ __forceinline__ void wave_lds_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
}

// 64 choices: this lane's key (-1: none), its rank among the lanes with the same key, and their number where it is their
// first (0 elsewhere).
struct Step {
    int key, rank, count;
};
__device__ __forceinline__ Step step_of(const SortArgs &a, int i, int end, int bits) {
    const int key = key_of(a, i, end);
    const unsigned long long who = same_key(key, bits);
    const int rank = (int)__popcll(who & lanes_below(threadIdx.x & 63));
    return {key, rank, key >= 0 && rank == 0 ? (int)__popcll(who) : 0};
}

// Calls f(step, index) for this wave's part [lo, hi) of the run, 64 choices at a time, in order. With kKeep the first
// kSteps steps are left in, or taken from, `kept`.
enum Kept { kFill, kUse };
template <Kept kKept, typename F>
__device__ __forceinline__ void each_step(const SortArgs &a, int lo, int hi, int bits, Step (&kept)[kSteps], F f) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
        const int i0 = lo + 64 * s;
        if (i0 >= hi) break;
        if constexpr (kKept == kFill) kept[s] = step_of(a, i0 + lane, hi, bits);
        f(kept[s], i0 + lane);
    }
    for (int i0 = lo + 64 * kSteps; i0 < hi; i0 += 64) f(step_of(a, i0 + lane, hi, bits), i0 + lane);
}

// Counts of one run, to the workspace.
template <int kBins>
__global__ __launch_bounds__(kThreads) void count_kernel(SortArgs a, int run, int bits) {
    __shared__ uint32_t s_count[kBins];
    const int tid = threadIdx.x, wave = tid >> 6;
    for (int k = tid; k < a.num_adapters; k += kThreads) s_count[k] = 0;
    __syncthreads();
    const int part = run / kWaves, lo = min(blockIdx.x * run + wave * part, (unsigned)a.n), hi = min(lo + part, a.n);
    Step kept[kSteps];
    each_step<kFill>(a, lo, hi, bits, kept, [&](const Step &s, int) {
        if (s.count > 0) atomicAdd(&s_count[s.key], (uint32_t)s.count);  // a sum: in any order
    });
    __syncthreads();
    for (int k = tid; k < a.num_adapters; k += kThreads) a.counts[(int64_t)blockIdx.x * stride_of(a.num_adapters) + k] = s_count[k];
}

// Inclusive sums of x and y over the workgroup's threads; adds them up with `base` (in, out: for the next round).
struct Pair {
    int x, y;
};
__device__ __forceinline__ Pair block_scan(Pair v, Pair (*s_wave)[kWaves], int round, Pair &total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int x = __shfl_up(v.x, o), y = __shfl_up(v.y, o);
        v.x += lane >= o ? x : 0;
        v.y += lane >= o ? y : 0;
    }
    Pair *mine = s_wave[round & 1];  // the round before may still be read
    if (lane == 63) mine[wave] = v;
    __syncthreads();
    total = Pair{0, 0};
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        if (w == wave) {
            v.x += total.x;
            v.y += total.y;
        }
        total.x += mine[w].x;
        total.y += mine[w].y;
    }
    return v;
}

constexpr int kAtOnce = 16;  // workgroups' counts that are read together

// kOne: the only workgroup, which counts for itself.
template <int kBins, bool kOne>
__global__ __launch_bounds__(kThreads) void place_kernel(SortArgs a, int run, int blocks, int bits) {
    __shared__ uint32_t s_at[kWaves][kBins];  // a wave's counts, then the rows that its next choices get
    __shared__ Pair s_wave[2][kWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, P = a.num_adapters;
    for (int k = lane; k < P; k += 64) s_at[wave][k] = 0;
    wave_lds_order();
    const int part = run / kWaves, lo = min(blockIdx.x * run + wave * part, (unsigned)a.n), hi = min(lo + part, a.n);
    Step kept[kSteps];
    each_step<kFill>(a, lo, hi, bits, kept, [&](const Step &s, int) {
        if (s.count > 0) s_at[wave][s.key] += s.count;
        wave_lds_order();
    });
    __syncthreads();

    // Rows before each adapter, and the segments, kBinsEach * kThreads adapters a round.
    Pair done = {0, 0};
    const int rounds = (P + kBinsEach * kThreads - 1) / (kBinsEach * kThreads);
    for (int r = 0; r < rounds; ++r) {
        const int k0 = (r * kThreads + tid) * kBinsEach, bins = min(P - k0, kBinsEach);
        uint32_t before[kBinsEach] = {0, 0, 0, 0}, all[kBinsEach] = {0, 0, 0, 0};
        if (bins > 0) {
            if constexpr (kOne) {
#pragma unroll
                for (int w = 0; w < kWaves; ++w)
#pragma unroll
                    for (int c = 0; c < kBinsEach; ++c) all[c] += s_at[w][k0 + c];
            } else {
                const uint32_t *counts = a.counts + k0;
                for (int b0 = 0; b0 < blocks; b0 += kAtOnce) {
                    uint4 x[kAtOnce];
#pragma unroll
                    for (int i = 0; i < kAtOnce; ++i) x[i] = ld16(counts + (int64_t)min(b0 + i, blocks - 1) * stride_of(P));
#pragma unroll
                    for (int i = 0; i < kAtOnce; ++i) {
                        const uint32_t y[kBinsEach] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
                        for (int c = 0; c < kBinsEach; ++c) {
                            before[c] += b0 + i < (int)blockIdx.x ? y[c] : 0;
                            all[c] += b0 + i < blocks ? y[c] : 0;
                        }
                    }
                }
            }
        }
        Pair mine = {0, 0};
#pragma unroll
        for (int c = 0; c < kBinsEach; ++c) {
            if (c >= bins) all[c] = 0;
            mine.x += all[c];
            mine.y += all[c] > 0;
        }
        Pair total;
        const Pair to = block_scan(mine, s_wave, r, total);
        int start = done.x + to.x - mine.x, seg = done.y + to.y - mine.y;
#pragma unroll
        for (int c = 0; c < kBinsEach; ++c) {
            if (c >= bins) continue;
            uint32_t at = start + before[c];
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const uint32_t here = s_at[w][k0 + c];
                s_at[w][k0 + c] = at;
                at += here;
            }
            if (blockIdx.x == 0 && all[c] > 0) {
                a.seg_start[seg] = start;
                a.seg_adapter[seg++] = k0 + c;
            }
            start += all[c];
        }
        done.x += total.x;
        done.y += total.y;
    }
    if (blockIdx.x == 0) {
        for (int64_t s = done.y + tid; s <= a.num_segments; s += kThreads) {  // up to 2^31 - 1 segments: past it an int would not end
            a.seg_start[s] = done.x;
            if (s < a.num_segments) a.seg_adapter[s] = 0;
        }
    }
    __syncthreads();

    each_step<kUse>(a, lo, hi, bits, kept, [&](const Step &s, int i) {
        if (i < hi) {
            int row = -1;
            if (s.key >= 0) {
                row = s_at[wave][s.key] + s.rank;
                a.order[row] = i;
            }
            a.place[i] = row;
            if (i >= done.x) a.order[i] = -1;
        }
        wave_lds_order();
        if (s.count > 0) s_at[wave][s.key] += s.count;
        wave_lds_order();
    });
}

template <int kBins>
void launch(const SortArgs &a, Split s, int bits, hipStream_t st) {
    if (s.blocks == 1) {
        hipLaunchKernelGGL((place_kernel<kBins, true>), dim3(1), dim3(kThreads), 0, st, a, s.run, 1, bits);
        return;
    }
    hipLaunchKernelGGL((count_kernel<kBins>), dim3(s.blocks), dim3(kThreads), 0, st, a, s.run, bits);
    hipLaunchKernelGGL((place_kernel<kBins, false>), dim3(s.blocks), dim3(kThreads), 0, st, a, s.run, s.blocks, bits);
}

}  // namespace

size_t sort_workspace_bytes(int n, int num_adapters) {
    const Split s = split_of(n);
    return s.blocks == 1 ? 0 : (size_t)s.blocks * stride_of(num_adapters) * sizeof(uint32_t);
}

hipError_t launch_sort_tokens(const SortArgs &a, hipStream_t st) {
    int bits = 0;
    while (1 << bits < a.num_adapters) ++bits;
    const Split s = split_of(a.n);
    if (a.num_adapters <= 256)
        launch<256>(a, s, bits, st);
    else if (a.num_adapters <= 1024)
        launch<1024>(a, s, bits, st);
    else if (a.num_adapters <= 2048)
        launch<2048>(a, s, bits, st);
    else
        launch<SGMV_MAX_SORTED_ADAPTERS>(a, s, bits, st);
    return hipGetLastError();
}

}  // namespace sgmv
