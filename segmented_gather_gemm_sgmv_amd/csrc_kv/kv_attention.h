// Work mapping and small device helpers shared by the paged-attention
// kernels (kv_attention.hip).
//
// A launch knows neither the requests' lengths nor how many new tokens each
// has: both are on the device. Its workgroups therefore find their work
// themselves. The rows of a request's tokens for one cached head are packed
// (token, then query head of the group) and cut into row tiles; a (request,
// row tile, cached head) is a group. The key tiles of a long group are split
// into runs of about `chunk` tiles, so that the whole batch makes about as
// many items as the GPU runs at once; chunk depends on the batch's total work
// alone, so a few long requests among many short ones still spread over the
// chip. Every wave forms the same sums over all requests (8 bytes per request,
// from L2; a scan over the wave's lanes, no LDS and no barrier) and picks the
// item of its workgroup's index.
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
    int split, size;   // this item's run of virtual tiles: [split * size, (split + 1) * size)
    int first_slot;    // partial-result slot of the group's split 0
};

template <int kCtrl, int kRowMask, typename V>
__device__ __forceinline__ V shifted(V v) {
    return __builtin_bit_cast(
        V, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), kCtrl, kRowMask, 0xf, false));
}

// Inclusive prefix sum over the wave's lanes.
template <typename V>
__device__ __forceinline__ V wave_scan(V v) {
    v += shifted<0x111, 0xf>(v);  // the lane 1, 2, 4, 8 below, within rows of 16 lanes
    v += shifted<0x112, 0xf>(v);
    v += shifted<0x114, 0xf>(v);
    v += shifted<0x118, 0xf>(v);
    v += shifted<0x142, 0xa>(v);  // row 0's last lane to row 1, row 2's to row 3
    v += shifted<0x143, 0xc>(v);  // lane 31 to rows 2 and 3
    return v;
}

// The item of workgroup `index` of a grid of `grid`, found by every wave for
// itself: lane i looks at requests i * per ... Returns false if there is none
// (the grid is an upper bound), or if the items do not fit the grid (only
// metadata outside the documented ranges does that): every workgroup then
// sees the same and none does anything. kBatch: requests per lane whose
// lengths are read at once.
template <int kRows, int kKeys, int kBatch>
__device__ __forceinline__ bool find_item_of(const AttnArgs &a, int take, int short_rows, int target, int min_chunk,
                                             int min_tiles, int max_splits, int index, int grid, Item &it) {
    const int lane = threadIdx.x & 63, B = a.num_requests;
    const int per = kBatch == 1 ? 1 : (B + 63) / 64, first = lane * per;
    Share s[kBatch];
    const auto read = [&](int j0) {
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int b = first + j0 + j;
            s[j] = j0 + j < per && b < B ? share<kRows, kKeys>(a, b, take, short_rows) : Share{0, 0, 0, 0, 0};
        }
    };
    // The batch's work in key tiles; its rounding is the same for every wave.
    float work = 0.f;
    for (int j0 = 0; j0 < per; j0 += kBatch) {
        read(j0);
#pragma unroll
        for (int j = 0; j < kBatch; ++j) work += (float)s[j].row_tiles * (float)max(s[j].tiles, 1);
    }
    work = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, wave_scan(work)), 63));
    const int chunk = max((int)fminf(ceilf(work * a.kv_heads / target), 1e9f), min_chunk);

    // A group is split where it is at least one and a half chunks long; the
    // groups that are split then have at most 4/3 * target parts together.
    const auto splits_of = [&](const Share &x) {
        return x.tiles < min_tiles ? 1 : min(max((x.tiles + chunk / 2) / chunk, 1), max_splits);
    };
    int items = 0, slots = 0;
    for (int j0 = 0; j0 < per; j0 += kBatch) {
        if (per > kBatch) read(j0);
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const int splits = splits_of(s[j]), parts = s[j].row_tiles * a.kv_heads * splits;
            items += parts;
            slots += splits > 1 ? parts : 0;
        }
    }
    const int items_to = wave_scan(items), slots_to = wave_scan(slots);
    if (__builtin_amdgcn_readlane(items_to, 63) > grid) return false;
    int at = index - (items_to - items), slot = slots_to - slots;
    bool mine = at >= 0 && at < items;
    const unsigned long long who = __ballot(mine);
    if (who == 0) return false;
    Share x = s[0];
    int b = first;
    if (kBatch > 1 && mine) {
        for (int j = 0; j < per; ++j) {
            x = share<kRows, kKeys>(a, first + j, take, short_rows);
            const int splits = splits_of(x), parts = x.row_tiles * a.kv_heads * splits;
            b = first + j;
            if (at < parts) break;
            at -= parts;
            slot += splits > 1 ? parts : 0;
        }
    }
    const int splits = splits_of(x), j = at / a.kv_heads, head = at % a.kv_heads;
    const int row_tile = x.row_tiles - 1 - j / splits;  // the tiles that see the most keys first
    const int size = (x.tiles + splits - 1) / splits;
    const int src = __ffsll((unsigned long long)who) - 1;
    const auto get = [&](int v) { return __builtin_amdgcn_readlane(v, src); };
    it.b = get(b);
    it.q0 = get(x.q0);
    it.n = get(x.n);
    it.p0 = get(x.p0);
    it.row_tile = get(row_tile);
    it.head = get(head);
    it.split = get(j % splits);
    it.size = get(size);
    it.first_slot = get(slot + (head * x.row_tiles + row_tile) * splits);
    return true;
}

template <int kRows, int kKeys>
__device__ __forceinline__ bool find_item(const AttnArgs &a, int take, int short_rows, int target, int min_chunk,
                                          int min_tiles, int max_splits, int index, int grid, Item &it) {
    return a.num_requests <= 64
               ? find_item_of<kRows, kKeys, 1>(a, take, short_rows, target, min_chunk, min_tiles, max_splits, index, grid, it)
               : find_item_of<kRows, kKeys, 8>(a, take, short_rows, target, min_chunk, min_tiles, max_splits, index, grid, it);
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
