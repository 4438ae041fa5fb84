// Work mapping and masks of the tree-attention kernels: kv_attention.hip where
// it is compiled for sgmv_tree_attention.
//
// As in kv_attention.h every wave finds its workgroup's item from the lengths
// on the device. Where there are more items than the GPU runs at once the
// longest requests come first: a long one that starts last would leave the
// rest idle. And the split items alone can be enumerated, for the launch that
// adds them up.
#pragma once

#include "kv_attention.h"

namespace sgmv {
namespace attn {

// A kind of items: rows and keys per tile, into how many items a launch is split, and splits' bounds (in key tiles).
template <int kRows_, int kKeys_, int kTarget_, int kMinChunk_, int kMinTiles_, int kMaxSplits_>
struct TreeKind {
    static constexpr int kRows = kRows_, kKeys = kKeys_, kTarget = kTarget_, kMinChunk = kMinChunk_, kMinTiles = kMinTiles_;
    static constexpr int kMaxSplits = kMaxSplits_;
};

// threadIdx.x, of which nothing is kept from one item to the next: what a loop over items computes from it, the compiler
// would otherwise compute before the loop, more than there are registers for.
__device__ __forceinline__ int this_thread() {
    int t = threadIdx.x;
    asm volatile("" : "+v"(t));
    return t;
}

// A launch's items of one kind. kBatch: requests per lane whose shares are kept.
template <typename Kind, int kBatch>
struct TreeItems {
    const AttnArgs &a;
    int per, first;       // requests per lane, and this lane's first one
    Share s[kBatch];      // of requests first + j0 ..
    int chunk;            // key tiles that a split has about
    int top;              // key tiles of the longest request; 0: requests in their order
    int items, splits;    // in all, and those of split groups

    // The lengths are read all at once.
    __device__ __forceinline__ void read(int j0) {
        int lo[kBatch], hi[kBatch], kv[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            lo[j] = hi[j] = kv[j] = 0;
            if (j0 + j < per) {
                const int b = min(first + j0 + j, a.num_requests - 1);
                lo[j] = a.q_start[b];
                hi[j] = a.q_start[b + 1];
                kv[j] = a.kv_len[b];
            }
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            s[j] = share_of<true, Kind::kRows, Kind::kKeys>(a, lo[j], hi[j], kv[j], kTakeAll, 0);
            if (j0 + j >= per || first + j0 + j >= a.num_requests) s[j].row_tiles = s[j].tiles = 0;
        }
    }
    __device__ __forceinline__ int splits_of(const Share &x) const {
        return x.tiles < Kind::kMinTiles ? 1 : min(max((x.tiles + chunk / 2) / chunk, 1), Kind::kMaxSplits);
    }
    // Four classes by length; all in one where top is 0.
    __device__ __forceinline__ int class_of(const Share &x) const {
        return top == 0 ? 0 : (4 * x.tiles > top) + (4 * x.tiles > 2 * top) + (4 * x.tiles > 3 * top);
    }

    __device__ __forceinline__ explicit TreeItems(const AttnArgs &args) : a(args) {
        per = kBatch == 1 ? 1 : (a.num_requests + 63) / 64;
        first = (this_thread() & 63) * per;
        float work = 0.f;  // in key tiles; its rounding is the same for every wave
        int longest = 0;
        for (int j0 = 0; j0 < per; j0 += kBatch) {
            read(j0);
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                work += (float)s[j].row_tiles * (float)max(s[j].tiles, 1);
                longest = max(longest, s[j].tiles);
            }
        }
        work = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, wave_scan(work)), 63));
        chunk = max((int)fminf(ceilf(work * a.kv_heads / Kind::kTarget), 1e9f), Kind::kMinChunk);
        items = splits = 0;
        for (int j0 = 0; j0 < per; j0 += kBatch) {
            if (per > kBatch) read(j0);
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int k = splits_of(s[j]), parts = s[j].row_tiles * a.kv_heads * k;
                items += parts;
                splits += k > 1 ? parts : 0;
            }
        }
        items = __builtin_amdgcn_readlane(wave_scan(items), 63);
        splits = __builtin_amdgcn_readlane(wave_scan(splits), 63);
        top = 0;
        if (items > Kind::kTarget && per <= kBatch) {  // (a class costs a pass over the requests, and there are four)
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) longest = max(longest, __shfl_xor(longest, o));
            top = __builtin_amdgcn_readfirstlane(longest);
        }
    }

    // Item `index` < items; with kSplit, of the `splits` ones of split groups.
    template <bool kSplit>
    __device__ __forceinline__ Item find(int index) {
        const auto parts_of = [&](const Share &x, int which) {
            const int k = splits_of(x);
            return class_of(x) != which || (kSplit && k == 1) ? 0 : x.row_tiles * a.kv_heads * k;
        };
        int at = 0, slot = 0, which = top == 0 ? 0 : 3, items_before = 0, slots_before = 0;
        unsigned long long who = 0;
        bool mine = false;
        for (;; --which) {
            int parts = 0, slots = 0;
            for (int j0 = 0; j0 < per; j0 += kBatch) {
                if (per > kBatch) read(j0);
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    const int x = parts_of(s[j], which);
                    parts += x;
                    slots += splits_of(s[j]) > 1 ? x : 0;
                }
            }
            const int parts_to = wave_scan(parts), slots_to = wave_scan(slots);
            at = index - items_before - (parts_to - parts);
            slot = slots_before + slots_to - slots;
            mine = at >= 0 && at < parts;
            who = __ballot(mine);
            if (who != 0 || which == 0) break;
            items_before += __builtin_amdgcn_readlane(parts_to, 63);
            slots_before += __builtin_amdgcn_readlane(slots_to, 63);
        }
        Share x = s[0];
        int b = first;
        if (kBatch > 1 && mine) {
            for (int j = 0; j < per; ++j) {
                b = first + j;
                x = share_of<true, Kind::kRows, Kind::kKeys>(a, a.q_start[b], a.q_start[b + 1], a.kv_len[b], kTakeAll, 0);
                const int parts = parts_of(x, which);
                if (at < parts) break;
                at -= parts;
                slot += splits_of(x) > 1 ? parts : 0;
            }
        }
        const int k = splits_of(x), j = at / a.kv_heads, head = at % a.kv_heads;
        const int row_tile = j / k, size = (x.tiles + k - 1) / k;
        const int src = __ffsll(who) - 1;
        const auto get = [&](int v) { return __builtin_amdgcn_readlane(v, src); };
        return {get(b), get(x.q0), get(x.n), get(x.p0), get(row_tile), get(head), get(j % k), get(size),
                get(slot + (head * x.row_tiles + row_tile) * k)};
    }
};

// Calls f(item) for item `index`, if there is one.
template <typename Kind, typename F>
__device__ __forceinline__ void one_item(const AttnArgs &a, int index, F f) {
    Item it;
    if (a.num_requests <= 64) {
        TreeItems<Kind, 1> x(a);
        if (index >= x.items) return;
        it = x.template find<false>(index);
    } else {
        TreeItems<Kind, 8> x(a);
        if (index >= x.items) return;
        it = x.template find<false>(index);
    }
    f(it);
}

// Calls f(item) for split items `start`, start + step, ...
template <typename Kind, typename F>
__device__ __forceinline__ void each_split(const AttnArgs &a, int start, int step, F f) {
    const auto go = [&](auto &x) {
        for (int i = start; i < x.splits; i += step) f(x.template find<true>(i));
    };
    if (a.num_requests <= 64) {
        TreeItems<Kind, 1> x(a);
        go(x);
    } else {
        TreeItems<Kind, 8> x(a);
        go(x);
    }
}

// One row's mask over its request's new tokens, which a token of a tree sees by.
struct TreeRow {
    const uint32_t *words;
    int count, n;  // words, none for a row past the last; new tokens

    // Bits m .. m + 31, those of tokens that there are not being 0; m is the same for every lane.
    __device__ __forceinline__ uint32_t bits(int m) const {
        const int left = n - m, w = m >> 5;
        if (left <= 0 || m <= -32) return 0;
        const uint32_t lo = (unsigned)w < (unsigned)count ? words[w] : 0, hi = (unsigned)(w + 1) < (unsigned)count ? words[w + 1] : 0;
        const uint32_t x = __builtin_amdgcn_alignbit(hi, lo, m & 31);
        return left < 32 ? x & ((1u << left) - 1) : x;
    }
    // How many it sees.
    __device__ __forceinline__ int seen() const {
        int sum = 0;
        for (int m = 0; m < n; m += 32) sum += __popc(bits(m));
        return sum;
    }
};

__device__ __forceinline__ TreeRow tree_row(const AttnArgs &a, const Item &it, int tok, bool valid) {
    return {a.tree + (int64_t)(it.q0 + (valid ? tok : 0)) * a.tree_words, valid ? a.tree_words : 0, it.n};
}

}  // namespace attn
}  // namespace sgmv
