// Work mapping and small device helpers shared by the paged-attention
// kernels (kv_attention.hip).
//
// A launch knows neither the requests' lengths nor how many new tokens each
// has: both are on the device. Its workgroups therefore find their work
// themselves. The rows of a request's tokens for one cached head are packed
// (token, then query head of the group) and cut into row tiles; a (request,
// row tile, cached head) is a group. The key tiles of a long group are split
// into runs of `chunk` tiles, so that the whole batch makes about as many
// items as the GPU runs at once; chunk depends on the batch's total work
// alone, so a few long requests among many short ones still spread over the
// chip. Every workgroup forms the same sums over all requests (8 bytes per
// request, from L2) and picks the item of its own index.
#pragma once

#include "kv_launch.h"
#include "sgmv_common.h"

namespace sgmv {
namespace attn {

typedef __attribute__((ext_vector_type(4))) float f32x4_t;
typedef __attribute__((ext_vector_type(16))) float f32x16_t;
typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8_t;
typedef __attribute__((ext_vector_type(4))) short s16x4_t;

constexpr int kThreads = 256;
constexpr int kWaves = 4;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kNone = -__builtin_huge_valf();

// Which requests a launch takes, by their number of packed rows.
enum Take { kTakeAll = 0, kTakeShort = 1, kTakeLong = 2 };

// One request's share of a launch.
struct Share {
    int q0, n, p0;  // first row of q, computed tokens, position of the first
    int row_tiles, tiles;
};

// The key tiles that queries at positions [pa, pb] read: the tiles of the
// first `sinks` keys, then those of [first key of pa's window, pb]; a run of
// `count` virtual tiles, v < sink_tiles being tile v and the others tile
// v + skip.
struct TileRun {
    int sink_tiles, skip, count;
    __device__ __forceinline__ int tile(int v) const { return v < sink_tiles ? v : v + skip; }
};

template <int kKeys>
__device__ __forceinline__ TileRun tile_run(int pa, int pb, int window, int sinks) {
    TileRun t = {0, 0, 0};
    if (pb < 0) return t;
    const int end = pb / kKeys + 1;
    if (window > 0) {
        const int lo = max(pa - window + 1, 0) / kKeys;
        t.sink_tiles = min((int)(((int64_t)sinks + kKeys - 1) / kKeys), lo);
        t.skip = lo - t.sink_tiles;
    }
    t.count = end - t.skip;
    return t;
}

template <int kRows, int kKeys>
__device__ __forceinline__ Share share(const AttnArgs &a, int b, int take, int short_rows) {
    Share s;
    const int lo = min(max(a.q_start[b], 0), a.T), hi = min(max(a.q_start[b + 1], lo), a.T);
    const int kv = min(max(a.kv_len[b], 0), a.max_blocks << a.page_shift);
    s.q0 = lo;
    s.n = min(hi - lo, a.max_q_len);
    s.p0 = kv - (hi - lo);  // below 0 by at most T: such a token sees nothing
    const int64_t rows = (int64_t)s.n * a.group;
    const bool mine = rows > 0 && (take == kTakeAll || (take == kTakeShort) == (rows <= short_rows));
    s.row_tiles = mine ? (int)((rows + kRows - 1) / kRows) : 0;
    s.tiles = mine ? tile_run<kKeys>(s.p0, s.p0 + s.n - 1, a.window, a.sinks).count : 0;
    return s;
}

struct Item {
    int b, q0, n, p0;
    int row_tile, head;
    int split, chunk;  // this item's run of virtual tiles: [split * chunk, ...)
    int first_slot;    // partial-result slot of the group's split 0 of this request's first group
    int splits;        // splits every group of the request is given
};

struct PlanSmem {
    unsigned long long wave[kWaves];
    Item item;
    int found;
};

__device__ __forceinline__ unsigned long long wave_sum(unsigned long long v) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

// The item of this workgroup. Returns false if it has none (the grid is an
// upper bound), or if the sums do not fit the launch (only metadata outside
// the documented ranges does that): every workgroup then sees the same and
// none does anything.
template <int kRows, int kKeys>
__device__ __forceinline__ bool find_item(const AttnArgs &a, int take, int short_rows, int target, int min_chunk,
                                          int index, int grid, PlanSmem &sm, Item &out) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, B = a.num_requests;
    const unsigned long long heads = a.kv_heads;
    Share first = {0, 0, 0, 0, 0};
    unsigned long long work = 0;
    for (int b = tid; b < B; b += kThreads) {
        const Share s = share<kRows, kKeys>(a, b, take, short_rows);
        if (b == tid) first = s;
        work += (unsigned long long)s.row_tiles * max(s.tiles, 1) * heads;
    }
    work = wave_sum(work);
    if (lane == 0) sm.wave[wave] = work;
    if (tid == 0) sm.found = 0;
    __syncthreads();
    work = sm.wave[0] + sm.wave[1] + sm.wave[2] + sm.wave[3];
    const unsigned long long per = (work + target - 1) / target;
    const int chunk = per > (unsigned)min_chunk ? (int)min(per, 0x40000000ull) : min_chunk;

    // Items in the low 40 bits, partial-result slots above: a request gives
    // at most 2^20 items here, and all of them at most 2 * target slots,
    // since a group of t tiles is split only if t > chunk >= work / target.
    unsigned long long base = 0;
    for (int b0 = 0; b0 < B; b0 += kThreads) {
        const int b = b0 + tid;
        Share s = first;
        if (b0 > 0) s = b < B ? share<kRows, kKeys>(a, b, take, short_rows) : Share{0, 0, 0, 0, 0};
        const int splits = max((s.tiles + chunk - 1) / chunk, 1);
        const unsigned long long groups = (unsigned long long)s.row_tiles * heads;
        const unsigned long long items = min(groups * splits, 1ull << 20);
        const unsigned long long mine = items | (splits > 1 ? groups * splits : 0) << 40;
        unsigned long long incl = mine;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const unsigned long long up = __shfl_up(incl, o);
            if (lane >= o) incl += up;
        }
        __syncthreads();
        if (lane == 63) sm.wave[wave] = incl;
        __syncthreads();
        unsigned long long before = base;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            if (w < wave) before += sm.wave[w];
            base += sm.wave[w];
        }
        before += incl - mine;
        const long long at = (long long)index - (long long)(before & ((1ull << 40) - 1));
        if (at >= 0 && at < (long long)items) {
            const int j = (int)at / a.kv_heads;
            Item &it = sm.item;
            it.b = b;
            it.q0 = s.q0;
            it.n = s.n;
            it.p0 = s.p0;
            it.head = (int)at % a.kv_heads;
            it.row_tile = s.row_tiles - 1 - j / splits;  // the tiles that see the most keys first
            it.split = j % splits;
            it.chunk = chunk;
            it.splits = splits;
            it.first_slot = (int)(before >> 40) + (it.head * s.row_tiles + it.row_tile) * splits;
            sm.found = 1;
        }
    }
    __syncthreads();
    out = sm.item;
    return sm.found && (base & ((1ull << 40) - 1)) <= (unsigned long long)grid;
}

// Maximum and sum over the four lanes (l, l ^ 16, l ^ 32, l ^ 48) that hold
// one row's keys in the 16 x 16 product's layout, or the two (l, l ^ 32) of
// the 32 x 32 one.
__device__ __forceinline__ float swap32_max(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float swap16_max(float v) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float swap32_sum(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float swap16_sum(float v) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// v_exp_f32: 2^x to about one ulp; results below 2^-126 are 0.
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// The reference point of a row whose running maximum is m (in units of
// scale * log2 e): 0 while the row has seen nothing, so that no difference of
// two infinities is formed.
__device__ __forceinline__ float ref_of(float m) { return m == kNone ? 0.f : m; }

// Partial results go from one workgroup to another, possibly on another XCD:
// 16-byte accesses at device scope, past the caches that are not coherent.
constexpr int kDeviceScope = 16;
typedef uint32_t u32x4_raw __attribute__((ext_vector_type(4)));
__device__ __forceinline__ __amdgpu_buffer_rsrc_t part_rsrc(float *base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(base, 0, (int)bytes, 0x00020000);
}
__device__ __forceinline__ f32x4_t part_load(__amdgpu_buffer_rsrc_t r, uint32_t byte_off) {
    return __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, byte_off, 0, kDeviceScope));
}
__device__ __forceinline__ float part_load1(__amdgpu_buffer_rsrc_t r, uint32_t byte_off) {
    return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(r, byte_off, 0, kDeviceScope));
}
__device__ __forceinline__ void part_store(__amdgpu_buffer_rsrc_t r, uint32_t byte_off, f32x4_t v) {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_raw, v), r, byte_off, 0, kDeviceScope);
}
__device__ __forceinline__ void part_store1(__amdgpu_buffer_rsrc_t r, uint32_t byte_off, float v) {
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), r, byte_off, 0, kDeviceScope);
}

// Counts this workgroup in once all of its stores have completed; returns to
// every thread whether it was the last of `expected`.
__device__ __forceinline__ bool arrive_last(uint32_t *counter, uint32_t expected, int *s_flag) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this wave's stores have reached the device's memory
    __syncthreads();
    if (threadIdx.x == 0) {
        const uint32_t prev = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        *s_flag = prev == expected - 1;
    }
    __syncthreads();
    return *s_flag != 0;
}

}  // namespace attn
}  // namespace sgmv
