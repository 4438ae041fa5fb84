// Attention of a step's new tokens over the paged key/value cache
// (sgmv_paged_attention).
//
// Mathematics: per row, out = sum_j p_j V_j / sum_j p_j with
// p_j = 2^(c s_j - c m), s_j = q . K_j, c = scale * log2 e, over one pass of
// the keys: m is a running reference point, and the sums are multiplied by
// 2^(c (m_old - m_new)) when it moves. It moves only when a score exceeds it
// by more than kSlack in the exponent, since any reference point gives the
// same quotient; weights then stay below 2^kSlack, which neither fp32 sums
// nor bf16 weights lose anything by. The products are formed transposed,
// S^T = K Q^T and O^T = V^T P^T, so that each lane holds one row's scores (the
// row's maximum is a maximum over a lane's registers and two or one lane
// swaps), the scores leave the first product in the layout in which the second
// takes its weights, and the order of keys within a product is free.
#include "kv_attention.h"
#include "sgmv.h"

namespace sgmv {

namespace {

using namespace attn;

constexpr float kSlack = 8.f;

// ----------------------------------------------------------------------------
// Streaming kernel: groups of few rows (decode, and every fp32 batch).
//
// What bounds it: HBM; a group reads its keys and values once. A workgroup
// takes one item, its four waves every fourth key tile, each with its own
// running softmax; the four results meet in LDS at the end. A wave's tile
// (32 keys in bf16, 16 in fp32: 8 KB of K and of V at head_dim 128) is loaded
// row-contiguously into registers while the previous one is worked on, then
// goes through the wave's own LDS region into the matrix instructions' layout,
// with no barrier in the loop. 16 rows go through v_mfma_*_16x16: with fewer
// rows the rest of the tile is idle, which costs nothing that HBM would not.
// Two workgroups fit a CU; their eight waves keep 128 KB in flight.
//
// Measured, bf16, heads of 128: 512 requests of 128 to 4096 keys, 64 heads on
// 8, 721 us (6.3 TB/s); 64 requests of 1 to 2048 keys, 32 heads, 162 us
// (6.2 TB/s); one request of 131001 keys, 64 heads on 8, 64 splits a head,
// 92 us (5.8 TB/s); a plain streaming read reaches 5.5 to 5.9 TB/s without
// the streaming hint. Where there is too little work to fill the GPU a wave's
// further tile costs 1.1 us (its loads' latency), and adding splits up 2.5:
// kStreamMinChunk and kStreamMinTiles follow from that (one request of 2000
// keys: 13.2 us in splits of 16 tiles, 11.0 in splits of 8).
// fp32 decode, 64 requests of 2000 keys: 32 heads 648 us (6.5 TB/s), 64 heads on
// 8 165 us (6.4). fp32 chunks: 88 to 93 TFLOP/s at 4 x 256 tokens, 32 heads on
// 8, of the 155 that a large fp32 product reaches; each 16 rows stream the keys
// by themselves, and a product step reads a fragment from LDS for 16 rows.
// ----------------------------------------------------------------------------
constexpr int kStreamRows = 16;
constexpr int kStreamTarget = 512;   // items a launch is split into: two workgroups on each of 256 CUs
constexpr int kStreamMinChunk = 8;   // key tiles a split has about at least (two per wave)
constexpr int kStreamMinTiles = 24;  // of a group that is split: fewer are done before the parts would be added up
constexpr int kStreamMaxSplits = 256;  // of one group

// bf16 requests of up to this many packed rows, two row tiles, are streamed; longer ones go to the tile kernel.
// Measured streamed and tiled, 2000 keys, 4 and 32 requests, us. 64 heads on 8: 24 rows 16.7 and 23.2, 46.6 and 52.4;
// 48 rows 18.9 and 26.3, 63.8 and 60.8; 64 rows 18.7 and 26.9, 71.9 and 64.9. 32 heads of their own: 32 rows 30.4 and
// 32.3, 202 and 193; 48 rows 35.0 and 38.2, 269 and 205. So a few requests are better streamed up to 64 rows at least
// (by 10 to 30%), many are not above 32 (5 to 30%); the bound is the many's, and a lone batch of few pays for it.
constexpr int kShortRows = 32;

struct StreamSmem {
    float m[kWaves][16], l[kWaves][16];  // the waves' running maxima and sums
    float part[2][kThreads];             // add_splits
    int flag;
    int odd;  // the tile kernel cleared values that are not finite
};

// D: columns of a row in LDS; U: columns that products run over, at least
// head_dim (96 for heads of 72 to 96 in rows of 128).
template <typename T, int D, int U = D>
struct Stream {
    static constexpr bool kBf16 = Elem<T>::kPerVec == 8;
    static constexpr int kBlocks = kBf16 ? 2 : 1;     // 16-key blocks per tile
    static constexpr int kKeys = 16 * kBlocks;
    static constexpr int kChunks = D / Elem<T>::kPerVec;  // 16-byte chunks per row
    static constexpr int kLoads = 16 * kChunks / 64;  // loads per lane and 16-key block
    static constexpr int kTileBytes = kKeys * kChunks * 16;
    static constexpr int kUsed = U / Elem<T>::kPerVec;    // chunks that products run over
    static constexpr int kOut = U / 16;               // 16-column blocks of the output
    static constexpr int kOutStride = D + 4;          // floats per row of the waves' results in LDS
    static constexpr int kOutBytes = 16 * kOutStride * 4;
    static constexpr int kWaveBytes = 2 * kTileBytes > kOutBytes ? 2 * kTileBytes : kOutBytes;  // one wave's LDS
    static constexpr int kSlotFloats = 16 * D + 32;   // partial result: 16 x D sums, 16 maxima, 16 weight sums

    // Chunk c of row r sits in chunk slot c ^ swizzle(r): the 16 rows that one
    // K read takes at one chunk index, and the 4 or 8 rows of one V read, lie
    // in different banks.
    static __device__ __forceinline__ int k_slot(int row, int c) {
        const int x = kChunks >= 16 ? row & 15 : (row >> 1) & 7;
        return row * kChunks + (c ^ x);
    }
    static __device__ __forceinline__ int v_slot(int row, int c) {
        int x;
        if (!kBf16)
            x = 4 * ((row >> 2) & 3);
        else if (kChunks >= 16)
            x = 4 * (row & 3) + 2 * ((row >> 2) & 1);
        else
            x = 4 * ((row >> 1) & 1) + 2 * ((row >> 2) & 1);
        return row * kChunks + (c ^ x);
    }
};

__device__ __forceinline__ f32x4_t mfma16(bf16x8_t a, bf16x8_t b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4_t mfma16(float a, float b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// LDS operations of one wave complete in order; this only keeps the compiler
// from moving them across.
__device__ __forceinline__ void wave_lds_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
}

typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;

// Four rows' values of one column per lane: lane i of a 16-lane group gives
// the address of four columns of row i / 4 and receives column i of the four
// rows.
__device__ __forceinline__ s16x4_t read_transposed(const void *p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t *)p);
}

// Values that are not finite. In a tile that some rows see and others do not they would reach all rows, since a zero
// weight does not take a NaN or an infinity out of a product: they enter it as 0, and are given to the rows that see
// them afterwards (any positive weight leaves such a value what it is). Measured: the check of the tiles on the mask's
// edge costs chunks 0 to 2%, and the test at a sum's end up to 1% of them (2 x 2048 tokens, the most) and 0.2 us of a
// decode step (one request of 2000 keys: 11.3 -> 11.7 us).
template <typename T>
__device__ __forceinline__ bool is_finite(T x) {
    if constexpr (sizeof(T) == 2)
        return (x.bits & 0x7f80u) != 0x7f80u;
    else
        return (__float_as_uint(x) & 0x7f800000u) != 0x7f800000u;
}

// Replaces them in a run of 16 bytes by 0; returns whether there were any.
template <typename T>
__device__ __forceinline__ bool clear_nonfinite(uint4 &v) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
    bool any = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t keep = 0;
        if constexpr (sizeof(T) == 2) {
            keep |= (w[i] & 0x7f80u) != 0x7f80u ? 0xffffu : 0u;
            keep |= (w[i] & 0x7f800000u) != 0x7f800000u ? 0xffff0000u : 0u;
        } else {
            keep = (w[i] & 0x7f800000u) != 0x7f800000u ? ~0u : 0u;
        }
        any |= keep != ~0u;
        w[i] &= keep;
    }
    v = make_uint4(w[0], w[1], w[2], w[3]);
    return any;
}

// Columns col .. col + 3 of a key's value, 0 where they are finite.
template <typename T>
__device__ __forceinline__ f32x4_t nonfinite4(const T *value, int col) {
    f32x4_t x;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const T v = value[col + e];
        if constexpr (sizeof(T) == 2)
            x[e] = is_finite(v) ? 0.f : __uint_as_float((uint32_t)v.bits << 16);
        else
            x[e] = is_finite(v) ? 0.f : v;
    }
    return x;
}

// Calls add(key, the key's value) for the keys of tiles v0, v0 + step, ... below v1 that lie in a 16-key block with
// values that are not finite. The wave looks for them 16 bytes per lane, so that a long context costs a read of its
// values and not a visit of every key.
template <typename T, int kKeys, typename Add>
__device__ __forceinline__ void each_nonfinite(const AttnArgs &a, const Item &it, const TileRun &run, int v0, int v1, int step,
                                               Add add) {
    for (int v = v0; v < v1; v += step) {
        const int first = run.tile(v) * kKeys;
        for (int key0 = first; key0 < first + kKeys; key0 += 16) {
            const int at = key0 >> a.page_shift;
            if (at >= a.max_blocks) break;  // past the request's last key
            const int p = a.block_table[(int64_t)it.b * a.max_blocks + at];
            const int page = (unsigned)p < (unsigned)a.num_pages ? p : 0;
            const int64_t row = (((int64_t)page * a.kv_heads + it.head) << a.page_shift) + (key0 & ((1 << a.page_shift) - 1));
            const T *values = static_cast<const T *>(a.V) + row * a.head_dim;
            bool odd = false;
            for (int f = threadIdx.x & 63; f < 16 * a.head_dim / Elem<T>::kPerVec; f += 64) {
                uint4 x = ld16(values + f * Elem<T>::kPerVec);
                odd |= clear_nonfinite<T>(x);
            }
            if (!__any(odd)) continue;
            for (int k = 0; k < 16; ++k) add(key0 + k, values + k * a.head_dim);
        }
    }
}

// Two weights as two bf16 values each, hi = rne(w) and lo = rne(w - hi): 16 significant bits, so that the result's only
// rounding that counts is the one to its own type. (Rounded once they would double the result's squared error.)
__device__ __forceinline__ void split_weights(float w0, float w1, uint32_t &hi, uint32_t &lo) {
    hi = pack_bf16x2(w0, w1);
    lo = pack_bf16x2(w0 - __uint_as_float(hi << 16), w1 - __uint_as_float(hi & 0xffff0000u));
}

// Writes one row's result: sum / weight, rounded once, and the log-sum-exp.
template <typename T>
__device__ __forceinline__ void store_row4(const AttnArgs &a, int64_t row, int head, int d, f32x4_t sum, float weight) {
    const float inv = weight > 0.f || weight != weight ? 1.f / weight : 0.f;
    const f32x4_t o = sum * inv;
    T *dst = static_cast<T *>(a.out) + row * a.out_stride + (int64_t)head * a.head_dim + d;
    if constexpr (Elem<T>::kPerVec == 8) {
        *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
    } else {
        *reinterpret_cast<float4 *>(dst) = make_float4(o[0], o[1], o[2], o[3]);
    }
}

__device__ __forceinline__ float lse_of(float m, float weight) {
    return weight > 0.f || weight != weight ? m * kLn2 + logf(weight) : kNone;
}

// The last of a group's items to arrive adds the splits up, in their order.
// Slots hold kRows x D sums, then the rows' maxima, then their weight sums.
// All of the maxima are read first, each thread's in one go, and the splits'
// factors left in LDS; then the sums, kAtOnce 4-column pieces and kDeep splits
// at a time: what this costs is the latency of reads from other XCDs, so as
// many as possible are in flight.
template <typename T, int D, int kRows, int kMaxSplits, int kAtOnce, typename Region>
__device__ __forceinline__ void add_splits(const AttnArgs &a, const Item &it, int splits, int row0, int live,
                                           __amdgpu_buffer_rsrc_t part, const Region &region, StreamSmem &sm) {
    constexpr int kSlot = kRows * D + 2 * kRows, kParts = kThreads / kRows, kEach = kMaxSplits / kParts;
    constexpr int kDeep = 16 / kAtOnce;  // splits read at a time
    const int tid = threadIdx.x;
    const auto factor = [&](int row) {  // splits' factors of a row, kMaxSplits apart
        return reinterpret_cast<float *>(region(row / (kRows / kWaves))) + row % (kRows / kWaves) * kMaxSplits;
    };
    {
        const int row = tid % kRows, p = tid / kRows;
        float m[kEach], l[kEach], top = kNone, weight = 0.f;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int k = min(p + i * kParts, splits - 1);  // a split read twice is not counted twice below
            m[i] = part_load1(part, ((uint32_t)k * kSlot + kRows * D + row) * 4);
            l[i] = part_load1(part, ((uint32_t)k * kSlot + kRows * D + kRows + row) * 4);
        }
#pragma unroll
        for (int i = 0; i < kEach; ++i) top = fmaxf(top, m[i]);
        sm.part[0][tid] = top;
        __syncthreads();
#pragma unroll
        for (int q = 0; q < kParts; ++q) top = fmaxf(top, sm.part[0][q * kRows + row]);
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int k = p + i * kParts;
            if (k < splits) {
                const float f = exp2_fast(m[i] - ref_of(top));
                factor(row)[k] = f;
                weight += f * l[i];
            }
        }
        sm.part[1][tid] = weight;
        __syncthreads();
        if (p == 0) {
            weight = 0.f;
#pragma unroll
            for (int q = 0; q < kParts; ++q) weight += sm.part[1][q * kRows + row];
            sm.part[0][row] = weight;  // only the threads p == 0 of this row read part[0][row] after the barrier above
            if (a.lse && row < live) {
                const int at = row0 + row;
                a.lse[(int64_t)(it.q0 + at / a.group) * a.q_heads + it.head * a.group + at % a.group] = lse_of(top, weight);
            }
        }
        __syncthreads();
    }
    const int vecs = a.head_dim / 4, pieces = live * vecs;
    for (int e0 = tid; e0 < pieces; e0 += kThreads * kAtOnce) {
        f32x4_t sum[kAtOnce];
        const float *f[kAtOnce];
        uint32_t at[kAtOnce];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const int e = min(e0 + u * kThreads, pieces - 1);
            sum[u] = f32x4_t{0.f, 0.f, 0.f, 0.f};
            f[u] = factor(e / vecs);
            at[u] = (e / vecs * D + e % vecs * 4) * 4;
        }
        const auto add = [&](int k0, auto deep) {  // splits k0 .. k0 + deep - 1, as far as there are
#pragma unroll
            for (int j = 0; j < deep(); ++j) {
                const int k = min(k0 + j, splits - 1);
#pragma unroll
                for (int u = 0; u < kAtOnce; ++u) {
                    const f32x4_t x = part_load(part, (uint32_t)k * kSlot * 4 + at[u]) * f[u][k];
                    sum[u] += k0 + j < splits ? x : f32x4_t{0.f, 0.f, 0.f, 0.f};
                }
            }
        };
        for (int k0 = 0; k0 < splits; k0 += kDeep) {
            if (splits - k0 > kDeep / 4)
                add(k0, [] { return kDeep; });
            else
                add(k0, [] { return kDeep / 4; });
        }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const int e = e0 + u * kThreads;
            if (e >= pieces) break;
            const int row = e / vecs, to = row0 + row;
            store_row4<T>(a, it.q0 + to / a.group, it.head * a.group + to % a.group, e % vecs * 4, sum[u], sm.part[0][row]);
        }
    }
}

// Item `index` of `grid`. The four LDS regions (kWaveBytes each) are the four
// waves' own. kOnce: no other row tile reads the same keys, so they are loaded
// past the caches' usual retention: at 64 heads on 8 and 512 requests of 128
// to 4096 keys 785 -> 720 us, 5.8 -> 6.3 TB/s.
template <typename T, int D, int U, bool kOnce>
__device__ __forceinline__ void stream_item(const AttnArgs &a, int take, int index, int grid, uint32_t *counters,
                                            float *slots, unsigned char *lds0, unsigned char *lds1,
                                            unsigned char *lds2, unsigned char *lds3, StreamSmem &sm) {
    using S = Stream<T, D, U>;
    constexpr int NB = S::kBlocks, CH = S::kChunks, NL = S::kLoads;
    Item it;
    if (!find_item<kStreamRows, S::kKeys>(a, take, kShortRows, kStreamTarget, kStreamMinChunk, kStreamMinTiles, kStreamMaxSplits, index,
                                              grid, it)) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, g = lane >> 4, r = lane & 15;
    const int rows = it.n * a.group, row0 = it.row_tile * kStreamRows;
    const int tok_a = row0 / a.group, tok_b = (min(row0 + kStreamRows, rows) - 1) / a.group;
    const int pa = it.p0 + tok_a, pb = it.p0 + tok_b;
    const TileRun run = tile_run<S::kKeys>(pa, pb, a.window, a.sinks);
    const int splits = run.count > it.size ? (run.count + it.size - 1) / it.size : 1;
    if (it.split >= splits) return;
    const int t1 = min(run.count, (it.split + 1) * it.size);

    // This lane's row: query fragments, position, first key of its window.
    const int my = row0 + r, tok = my / a.group;
    const bool valid = my < rows;
    const int q_head = it.head * a.group + my % a.group;
    const int pos = valid ? it.p0 + tok : -1;
    const int w_lo = a.window > 0 ? pos - a.window + 1 : 0;
    const int pa_lo = a.window > 0 ? pa - a.window + 1 : 0, pb_lo = a.window > 0 ? pb - a.window + 1 : 0;
    const int nch = a.head_dim / Elem<T>::kPerVec;
    uint4 qf[S::kUsed / 4];
    {
        const T *q = static_cast<const T *>(a.q) + (int64_t)(it.q0 + (valid ? tok : 0)) * a.q_stride +
                     (int64_t)(valid ? q_head : 0) * a.head_dim;
#pragma unroll
        for (int k = 0; k < S::kUsed / 4; ++k) {
            const int c = 4 * k + g;
            const uint4 v = ld16(q + (c < nch ? c : 0) * Elem<T>::kPerVec);
            qf[k] = valid && c < nch ? v : make_uint4(0, 0, 0, 0);
        }
    }

    const auto region = [&](int w) { return w == 0 ? lds0 : w == 1 ? lds1 : w == 2 ? lds2 : lds3; };
    unsigned char *k_lds = region(wave), *v_lds = k_lds + S::kTileBytes;
    if (nch < CH) {  // a narrower head: the chunks past it stay zero
        for (int i = lane; i < 2 * S::kTileBytes / 16; i += 64)
            reinterpret_cast<uint4 *>(k_lds)[i] = make_uint4(0, 0, 0, 0);
        wave_lds_order();
    }

    // Pages of this wave's next 64 16-key blocks, one per lane.
    const int row_bytes = a.head_dim * (int)sizeof(T);
    const int page_mask = (1 << a.page_shift) - 1;
    int pages = 0;
    const int first = it.split * it.size + wave;
    auto load_pages = [&](int i) {  // the wave's tiles i, i + 1, ...
        const int v = first + kWaves * (i + lane / NB);
        pages = 0;
        if (v < t1) {
            const int key = run.tile(v) * S::kKeys + 16 * (lane % NB), at = key >> a.page_shift;
            if (at < a.max_blocks) {
                const int p = a.block_table[(int64_t)it.b * a.max_blocks + at];
                pages = (unsigned)p < (unsigned)a.num_pages ? p : 0;
            }
        }
    };
    uint4 kr[NB * NL], vr[NB * NL];
    auto load_tile = [&](int i, int v) {
        const int key0 = run.tile(v) * S::kKeys;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            const int page = __builtin_amdgcn_readlane(pages, (i % (64 / NB)) * NB + nb);
            const int64_t row = (((int64_t)page * a.kv_heads + it.head) << a.page_shift) + ((key0 + 16 * nb) & page_mask);
            const char *kp = static_cast<const char *>(a.K) + row * row_bytes;
            const char *vp = static_cast<const char *>(a.V) + row * row_bytes;
#pragma unroll
            for (int j = 0; j < NL; ++j) {
                const int f = j * 64 + lane, c = f % CH;
                const uint32_t off = (uint32_t)(f / CH * row_bytes + (c < nch ? c : 0) * 16);
                kr[nb * NL + j] = kOnce ? ld16_stream(kp + off) : ld16(kp + off);
                vr[nb * NL + j] = kOnce ? ld16_stream(vp + off) : ld16(vp + off);
            }
        }
    };

    const float c2 = a.scale * kLog2e;
    float m = kNone, l = 0.f;  // m in units of scale * log2 e
    f32x4_t o[S::kOut];
#pragma unroll
    for (int d = 0; d < S::kOut; ++d) o[d] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    bool odd = false;  // values that are not finite, in a tile that not every row sees all of
    load_pages(0);
    if (first < t1) load_tile(0, first);
    for (int i = 0, v = first; v < t1; ++i, v += kWaves) {
        const int key0 = run.tile(v) * S::kKeys;
        // Every row of the tile sees every key.
        const bool whole = key0 + S::kKeys - 1 <= pa && (pb_lo <= key0 || key0 + S::kKeys <= a.sinks);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int j = 0; j < NL; ++j) {
                const int f = j * 64 + lane, row = 16 * nb + f / CH, c = f % CH, key = key0 + row;
                uint4 vv = vr[nb * NL + j];
                if (!whole) {
                    if (key > pb || (key < pa_lo && key >= a.sinks))
                        vv = make_uint4(0, 0, 0, 0);  // no row sees it
                    else if (pa != pb)  // rows of one token see the same keys
                        odd |= clear_nonfinite<T>(vv);
                }
                if (c < nch) {
                    reinterpret_cast<uint4 *>(k_lds)[S::k_slot(row, c)] = kr[nb * NL + j];
                    reinterpret_cast<uint4 *>(v_lds)[S::v_slot(row, c)] = vv;
                }
            }
        wave_lds_order();
        if (v + kWaves < t1) {
            if ((i + 1) % (64 / NB) == 0) load_pages(i + 1);
            load_tile(i + 1, v + kWaves);
        }

        f32x4_t s[NB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            s[nb] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < S::kUsed / 4; ++k) {
                const uint4 kf = reinterpret_cast<const uint4 *>(k_lds)[S::k_slot(16 * nb + r, 4 * k + g)];
                if constexpr (S::kBf16) {
                    s[nb] = mfma16(__builtin_bit_cast(bf16x8_t, kf), __builtin_bit_cast(bf16x8_t, qf[k]), s[nb]);
                } else {
                    s[nb] = mfma16(__uint_as_float(kf.x), __uint_as_float(qf[k].x), s[nb]);
                    s[nb] = mfma16(__uint_as_float(kf.y), __uint_as_float(qf[k].y), s[nb]);
                    s[nb] = mfma16(__uint_as_float(kf.z), __uint_as_float(qf[k].z), s[nb]);
                    s[nb] = mfma16(__uint_as_float(kf.w), __uint_as_float(qf[k].w), s[nb]);
                }
            }
        }
        if (!whole) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int key = key0 + 16 * nb + 4 * g + e;
                    const bool seen = key <= pos && (key >= w_lo || key < a.sinks);
                    s[nb][e] = seen ? s[nb][e] : kNone;
                }
        }
        float top = kNone;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 4; ++e) top = fmaxf(top, s[nb][e]);
        top = swap32_max(swap16_max(top)) * c2;
        const bool move = top > m + kSlack;  // of this row: the others keep their reference points, and so their bits
        if (__any(move)) {
            const float to = move ? top : m;
            const float keep = exp2_fast(m - ref_of(to));
            l *= keep;
#pragma unroll
            for (int d = 0; d < S::kOut; ++d) o[d] *= keep;
            m = to;
        }
        const float ref = ref_of(m);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[nb][e] = exp2_fast(__builtin_fmaf(s[nb][e], c2, -ref));
                l += s[nb][e];
            }

        if constexpr (S::kBf16) {
            // Weight slots 8 g + j of this lane: keys 4 g + j (j < 4) and 16 + 4 g + j - 4. HBM leaves the time for the
            // second product.
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) split_weights(s[i / 2][2 * (i % 2)], s[i / 2][2 * (i % 2) + 1], hi[i], lo[i]);
            const bf16x8_t p = __builtin_bit_cast(bf16x8_t, make_uint4(hi[0], hi[1], hi[2], hi[3]));
            const bf16x8_t p_lo = __builtin_bit_cast(bf16x8_t, make_uint4(lo[0], lo[1], lo[2], lo[3]));
            const int row = 4 * g + (r >> 2), half = 8 * (r & 1);
#pragma unroll
            for (int d = 0; d < S::kOut; ++d) {
                const int c = 2 * d + ((r & 3) >> 1);
                union {
                    s16x4_t h[2];
                    bf16x8_t v;
                } vf;
                vf.h[0] = read_transposed(v_lds + S::v_slot(row, c) * 16 + half);
                vf.h[1] = read_transposed(v_lds + S::v_slot(row + 16, c) * 16 + half);
                o[d] = mfma16(vf.v, p_lo, mfma16(vf.v, p, o[d]));
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int d = 0; d < S::kOut; ++d) {
                    const float *vp = reinterpret_cast<const float *>(v_lds + S::v_slot(4 * g + e, 4 * d + (r >> 2)) * 16);
                    o[d] = mfma16(vp[r & 3], s[0][e], o[d]);
                }
        }
        wave_lds_order();
    }
    l = swap32_sum(swap16_sum(l));
    // A sum over a value that is not finite is that value, which was cleared, or met a weight's zero low part.
#pragma unroll
    for (int d = 0; d < S::kOut; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) odd |= o[d][e] != o[d][e] && l == l;
    if (__any(odd)) {
        f32x4_t x[S::kOut];
#pragma unroll
        for (int d = 0; d < S::kOut; ++d) x[d] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        each_nonfinite<T, S::kKeys>(a, it, run, first, t1, kWaves, [&](int key, const T *value) {
            const bool seen = key <= pos && (key >= w_lo || key < a.sinks);
            if (!__any(seen)) return;
#pragma unroll
            for (int d = 0; d < S::kOut; ++d) {
                const int col = 16 * d + 4 * g;
                if (seen && col < a.head_dim) x[d] += nonfinite4(value, col);
            }
        });
#pragma unroll
        for (int d = 0; d < S::kOut; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[d][e] = x[d][e] != 0.f ? x[d][e] : o[d][e];
    }

    // The four waves' results meet in LDS, in wave order.
    if (g == 0) {
        sm.m[wave][r] = m;
        sm.l[wave][r] = l;
    }
    __syncthreads();
    const float m_all = fmaxf(fmaxf(sm.m[0][r], sm.m[1][r]), fmaxf(sm.m[2][r], sm.m[3][r]));
    const float keep = exp2_fast(m - ref_of(m_all));
    float *o_lds = reinterpret_cast<float *>(k_lds) + r * S::kOutStride;
#pragma unroll
    for (int d = 0; d < S::kOut; ++d) *reinterpret_cast<f32x4_t *>(o_lds + 16 * d + 4 * g) = o[d] * keep;
    __syncthreads();

    const __amdgpu_buffer_rsrc_t part =
        part_rsrc(slots + (int64_t)it.first_slot * S::kSlotFloats, (uint32_t)splits * S::kSlotFloats * 4);
    const int live = min(kStreamRows, rows - row0);
    const int vecs = a.head_dim / 4;  // 4-column pieces of a row
    for (int e = tid; e < live * vecs; e += kThreads) {
        const int row = e / vecs, d = e % vecs * 4;
        f32x4_t sum = f32x4_t{0.f, 0.f, 0.f, 0.f};
        float top = kNone, weight = 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) top = fmaxf(top, sm.m[w][row]);
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            sum += *reinterpret_cast<const f32x4_t *>(reinterpret_cast<const float *>(region(w)) + row * S::kOutStride + d);
            weight += sm.l[w][row] * exp2_fast(sm.m[w][row] - ref_of(top));
        }
        if (splits == 1) {
            const int at = row0 + row, head = it.head * a.group + at % a.group;
            const int64_t q_row = it.q0 + at / a.group;
            store_row4<T>(a, q_row, head, d, sum, weight);
            if (a.lse && d == 0) a.lse[q_row * a.q_heads + head] = lse_of(top, weight);
        } else {
            const uint32_t slot = (uint32_t)it.split * S::kSlotFloats * 4;
            part_store(part, slot + (row * D + d) * 4, sum);
            if (d == 0) {
                part_store1(part, slot + (16 * D + row) * 4, top);
                part_store1(part, slot + (16 * D + 16 + row) * 4, weight);
            }
        }
    }
    if (splits == 1) return;

    uint32_t *counter = counters + it.first_slot;
    if (!arrive_last(counter, (uint32_t)splits, &sm.flag)) return;
    add_splits<T, D, kStreamRows, kStreamMaxSplits, 1>(a, it, splits, row0, live, part, region, sm);
    if (tid == 0) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// ----------------------------------------------------------------------------
// Tile kernel: bf16 groups of many rows (prompt chunks).
//
// What bounds it: the matrix cores and the softmax beside them, at the clock
// that the power limit leaves. A workgroup takes 128 packed rows, 32 per wave, against key tiles of
// 64 that its waves share: the next tile is loaded straight to the other of
// two LDS buffers while the present one is worked on, one barrier per tile.
// 32 rows go through v_mfma_f32_32x32x16_bf16, whose transposed scores leave
// half of a row's keys on each of two lanes. Two workgroups share a CU (up to
// 228 registers, 68 KB of LDS), one's softmax beside the other's products.
// The weights enter the second product as two bf16 values, as in the streaming
// kernel, so a request's precision does not depend on its length; the flops
// below count the products that the operator has, not this third one.
//
// Measured, heads of 128, 64 on 8: 8 x 1024 tokens behind 4096 each 1770 to
// 1800 us, 690 to 700 TFLOP/s (1040 with the third product counted); one prompt
// of 8192 tokens 740; the largest library product reaches 1520. The matrix cores
// are busy 59% of the cycles. The cycles are the same with zeros for keys and
// values, 1.47 ms at 2.1 GHz; with random data the clock is 1.64 GHz. With
// weights of 8 bits: 870 and 960 TFLOP/s, 48% and 1.73 GHz, and the result's
// error against 64 bits 1.4 times as large (2.3e-3 of its norm, against 1.66e-3).
// Tried in that form, each against 867 TFLOP/s: the next tile's scores formed
// beside this tile's softmax (886), eight waves on 256 rows (+5% for long
// contexts, -3% for short, and 10% less at heads of 64), the same with its
// halves taking turns (856), 64 rows per wave (791; half the LDS reads, but one
// wave per SIMD), forced interleaving of products and softmax (698).
// ----------------------------------------------------------------------------
constexpr int kTileRows = 128;
constexpr int kTileKeys = 64;
constexpr int kTileTarget = 512;   // as kStreamTarget
constexpr int kTileMinChunk = 8;   // key tiles a split has about at least
constexpr int kTileMinTiles = 12;  // of a group that is split
constexpr int kTileMaxSplits = 64; // of one group

template <int D, int U = D>
struct Tile {
    static constexpr int kChunks = D / 8;
    static constexpr int kLoads = kTileKeys * kChunks / kThreads;  // per thread, of K and of V
    static constexpr int kBytes = kTileKeys * kChunks * 16;
    static constexpr int kSteps = U / 16;                          // 16-column steps of the scores
    static constexpr int kOut = U / 32;                            // 32-column blocks of the output
    static constexpr int kSlotFloats = kTileRows * D + 2 * kTileRows;
};

__device__ __forceinline__ f32x16_t mfma32(bf16x8_t a, bf16x8_t b, f32x16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// Eight rows' values of one column per lane: four rows at `p`, four `step` bytes on.
__device__ __forceinline__ bf16x8_t read_columns(const unsigned char *p, int step) {
    union {
        s16x4_t x[2];
        bf16x8_t v;
    } f;
    f.x[0] = read_transposed(p);
    f.x[1] = read_transposed(p + step);
    return f.v;
}

// 16 bytes per lane from base + off straight to LDS at `to` + 16 * lane (base and to uniform over the wave).
__device__ __forceinline__ void load_to_lds(const char *base, uint32_t off, unsigned char *to, bool on) {
    typedef const __attribute__((address_space(1))) char gchar_t;
    typedef __attribute__((address_space(3))) unsigned char lchar_t;
    if (on) __builtin_amdgcn_global_load_lds((gchar_t *)base + off, (lchar_t *)to, 16, 0, 0);
}

__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Every wave's loads to LDS have landed, and its reads of LDS are done.
__device__ __forceinline__ void loads_barrier() {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    lds_barrier();
}

// U as for Stream; kFull: head_dim is D.
template <int D, int U, bool kFull>
__device__ __forceinline__ void tile_item(const AttnArgs &a, int take, int index, int grid, uint32_t *counters,
                                          float *slots, unsigned char *k_even, unsigned char *v_even,
                                          unsigned char *k_odd, unsigned char *v_odd, StreamSmem &sm) {
    using L = Tile<D, U>;
    using S = Stream<bf16_t, D>;  // the LDS layouts of a row
    constexpr int CH = L::kChunks, NL = L::kLoads;
    Item it;
    if (!find_item<kTileRows, kTileKeys>(a, take, kShortRows, kTileTarget, kTileMinChunk, kTileMinTiles, kTileMaxSplits, index, grid, it)) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, h = lane >> 5, r = lane & 31;
    const int rows = it.n * a.group, row0 = it.row_tile * kTileRows;
    const int pa = it.p0 + row0 / a.group, pb = it.p0 + (min(row0 + kTileRows, rows) - 1) / a.group;
    const TileRun run = tile_run<kTileKeys>(pa, pb, a.window, a.sinks);
    const int splits = run.count > it.size ? (run.count + it.size - 1) / it.size : 1;
    if (it.split >= splits) return;
    const int t0 = it.split * it.size, t1 = min(run.count, t0 + it.size);

    const int wrow = row0 + 32 * wave;  // this wave's rows; past the last row it only helps loading
    const bool live_wave = wrow < rows;
    const int wa = it.p0 + wrow / a.group, wb = it.p0 + (min(wrow + 32, rows) - 1) / a.group;
    const int my = wrow + r, tok = my / a.group;
    const bool valid = my < rows;
    const int q_head = it.head * a.group + my % a.group;
    const int pos = valid ? it.p0 + tok : -1;
    const int w_lo = a.window > 0 ? pos - a.window + 1 : 0;
    const int pa_lo = a.window > 0 ? pa - a.window + 1 : 0, pb_lo = a.window > 0 ? pb - a.window + 1 : 0;
    const int wa_lo = a.window > 0 ? wa - a.window + 1 : 0, wb_lo = a.window > 0 ? wb - a.window + 1 : 0;
    const int head_dim = kFull ? D : a.head_dim, nch = head_dim / 8;
    bf16x8_t qf[L::kSteps];
    {
        const bf16_t *q = static_cast<const bf16_t *>(a.q) + (int64_t)(it.q0 + (valid ? tok : 0)) * a.q_stride +
                          (int64_t)(valid ? q_head : 0) * a.head_dim;
#pragma unroll
        for (int k = 0; k < L::kSteps; ++k) {
            const int c = 2 * k + h;
            const uint4 v = ld16(q + (c < nch ? c : 0) * 8);
            qf[k] = __builtin_bit_cast(bf16x8_t, valid && c < nch ? v : make_uint4(0, 0, 0, 0));
        }
    }
    if (!kFull) {  // the chunks past the head stay zero
        for (int i = tid; i < L::kBytes / 16; i += kThreads)
            for (unsigned char *buf : {k_even, v_even, k_odd, v_odd})
                reinterpret_cast<uint4 *>(buf)[i] = make_uint4(0, 0, 0, 0);
        __syncthreads();
    }

    const int row_bytes = head_dim * 2, page_mask = (1 << a.page_shift) - 1;
    int pages = 0;  // of the next 16 tiles' 64 16-key blocks, one per lane
    auto load_pages = [&](int i) {
        const int v = t0 + i + lane / 4;
        pages = 0;
        if (v < t1) {
            const int at = (run.tile(v) * kTileKeys + 16 * (lane % 4)) >> a.page_shift;
            if (at < a.max_blocks) {
                const int p = a.block_table[(int64_t)it.b * a.max_blocks + at];
                pages = (unsigned)p < (unsigned)a.num_pages ? p : 0;
            }
        }
    };
    // Tile i goes straight to LDS: thread t fills 16-byte slots t, t + 256, ... of a buffer with the chunks that the
    // swizzles put there. Rows of a 16-key block are one run of memory, so a thread's offset in it is the same for all.
    constexpr int kBlockThreads = 16 * CH;  // threads that fill one 16-key block
    const int slot_row = tid % kBlockThreads / CH, slot_chunk = tid % CH;
    const int k_chunk = S::k_slot(slot_row, slot_chunk) - slot_row * CH, v_chunk = S::v_slot(slot_row, slot_chunk) - slot_row * CH;
    const uint32_t k_off = slot_row * row_bytes + k_chunk * 16, v_off = slot_row * row_bytes + v_chunk * 16;
    const int wave_u = __builtin_amdgcn_readfirstlane(wave);
    auto load_tile = [&](int i, unsigned char *kb, unsigned char *vb) {
        const int key0 = run.tile(t0 + i) * kTileKeys;
#pragma unroll
        for (int j = 0; j < NL; ++j) {
            const int block = j * (kThreads / kBlockThreads) + wave_u * 64 / kBlockThreads;
            const int page = __builtin_amdgcn_readlane(pages, i % 16 * 4 + block);
            const int64_t row =
                (((int64_t)page * a.kv_heads + it.head) << a.page_shift) + ((key0 + 16 * block) & page_mask);
            const int at = (j * kThreads + wave_u * 64) * 16;
            load_to_lds(static_cast<const char *>(a.K) + row * row_bytes, k_off, kb + at, k_chunk < nch);
            load_to_lds(static_cast<const char *>(a.V) + row * row_bytes, v_off, vb + at, v_chunk < nch);
        }
    };

    const float c2 = a.scale * kLog2e;
    float m = kNone, l = 0.f;
    f32x16_t o[L::kOut];
#pragma unroll
    for (int d = 0; d < L::kOut; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[d][e] = 0.f;

    // Offsets of this lane's fragments in a buffer's first rows: K rows r (32 of a product), chunk 2 k + h; V rows
    // 4 h + 0..3, columns 32 d + 16 (lane / 16 % 2) + 0..15. Sixteen rows further on the swizzles are the same.
    uint32_t k_at[L::kSteps], v_at[L::kOut];
#pragma unroll
    for (int k = 0; k < L::kSteps; ++k) k_at[k] = S::k_slot(r, 2 * k + h) * 16;
#pragma unroll
    for (int d = 0; d < L::kOut; ++d)
        v_at[d] = S::v_slot(4 * h + ((lane & 15) >> 2), 4 * d + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1)) * 16 +
                  8 * (lane & 1);

    const int n = t1 - t0;
    const auto all_see = [&](int key0) {  // every row sees every key of the tile
        return key0 + kTileKeys - 1 <= pa && (pb_lo <= key0 || key0 + kTileKeys <= a.sinks);
    };
    auto step = [&](int i, unsigned char *kb, unsigned char *vb, unsigned char *k_next, unsigned char *v_next) {
        if (i + 1 < n) {
            if ((i + 1) % 16 == 0) load_pages(i + 1);
            load_tile(i + 1, k_next, v_next);
        }
        const int key0 = run.tile(t0 + i) * kTileKeys;
        if (!all_see(key0)) {
#pragma unroll
            for (int j = 0; j < NL; ++j) {
                const int f = j * kThreads + tid, key = key0 + f / CH;
                uint4 v = reinterpret_cast<uint4 *>(vb)[f];
                const bool unseen = key > pb || (key < pa_lo && key >= a.sinks);  // by every row
                if (unseen) v = make_uint4(0, 0, 0, 0);
                const bool cleared = clear_nonfinite<bf16_t>(v);
                if (unseen || cleared) reinterpret_cast<uint4 *>(vb)[f] = v;
                if (cleared) sm.odd = 1;
            }
            lds_barrier();
        }
        if (live_wave && key0 <= wb && (key0 + kTileKeys > wa_lo || key0 < a.sinks)) {
            bf16x8_t kf[2][L::kSteps];
#pragma unroll
            for (int k = 0; k < L::kSteps; ++k) kf[0][k] = *reinterpret_cast<const bf16x8_t *>(kb + k_at[k]);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int k = 0; k < L::kSteps; ++k) kf[1][k] = *reinterpret_cast<const bf16x8_t *>(kb + k_at[k] + 32 * CH * 16);
            __builtin_amdgcn_sched_barrier(0);
            f32x16_t s[2];
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int e = 0; e < 16; ++e) s[b][e] = 0.f;
#pragma unroll
            for (int k = 0; k < L::kSteps; ++k) s[0] = mfma32(kf[0][k], qf[k], s[0]);
#pragma unroll
            for (int k = 0; k < L::kSteps; ++k) s[1] = mfma32(kf[1][k], qf[k], s[1]);
            bf16x8_t vf[2][L::kOut];  // V fragments of two 16-key steps
#pragma unroll
            for (int d = 0; d < L::kOut; ++d) vf[0][d] = read_columns(vb + v_at[d], 8 * CH * 16);
            if (!(key0 + kTileKeys - 1 <= wa && (wb_lo <= key0 || key0 + kTileKeys <= a.sinks))) {
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int key = key0 + 32 * b + 8 * (e / 4) + 4 * h + e % 4;
                        const bool seen = (key <= pos) & ((key >= w_lo) | (key < a.sinks));
                        s[b][e] = seen ? s[b][e] : kNone;
                    }
            }
            float top = kNone;
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int e = 0; e < 16; ++e) top = fmaxf(top, s[b][e]);
            top = swap32_max(top) * c2;
            const bool move = top > m + kSlack;  // of this row, as above
            if (__any(move)) {
                const float to = move ? top : m;
                const float keep = exp2_fast(m - ref_of(to));
                l *= keep;
#pragma unroll
                for (int d = 0; d < L::kOut; ++d) o[d] *= keep;
                m = to;
            }
            const float ref = ref_of(m);
#pragma unroll
            for (int t = 0; t < 4; ++t) {  // 16 keys: this lane's weight slots are 16 t + 4 h + {0..3, 8..11}
                float w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    w[e] = exp2_fast(__builtin_fmaf(s[t / 2][t % 2 * 8 + e], c2, -ref));
                    l += w[e];
                }
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) split_weights(w[2 * i], w[2 * i + 1], hi[i], lo[i]);
                const bf16x8_t p = __builtin_bit_cast(bf16x8_t, make_uint4(hi[0], hi[1], hi[2], hi[3]));
                const bf16x8_t p_lo = __builtin_bit_cast(bf16x8_t, make_uint4(lo[0], lo[1], lo[2], lo[3]));
                if (t < 3) {
#pragma unroll
                    for (int d = 0; d < L::kOut; ++d)
                        vf[(t + 1) & 1][d] = read_columns(vb + v_at[d] + 16 * (t + 1) * CH * 16, 8 * CH * 16);
                }
#pragma unroll
                for (int d = 0; d < L::kOut; ++d) o[d] = mfma32(vf[t & 1][d], p, o[d]);
#pragma unroll
                for (int d = 0; d < L::kOut; ++d) o[d] = mfma32(vf[t & 1][d], p_lo, o[d]);
            }
        }
        loads_barrier();
    };
    if (tid == 0) sm.odd = 0;
    if (n > 0) {
        load_pages(0);
        load_tile(0, k_even, v_even);
    }
    loads_barrier();
    for (int i = 0; i < n; i += 2) {
        step(i, k_even, v_even, k_odd, v_odd);
        if (i + 1 < n) step(i + 1, k_odd, v_odd, k_even, v_even);
    }
    l = swap32_sum(l);
    // A sum over a value that is not finite is that value, which was cleared, or met a weight's zero low part.
    bool odd = sm.odd != 0;
#pragma unroll
    for (int d = 0; d < L::kOut; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) odd |= o[d][e] != o[d][e];
    if (__any(odd && valid && l == l)) {
        f32x16_t x[L::kOut];
#pragma unroll
        for (int d = 0; d < L::kOut; ++d)
#pragma unroll
            for (int e = 0; e < 16; ++e) x[d][e] = 0.f;
        each_nonfinite<bf16_t, kTileKeys>(a, it, run, t0, t1, 1, [&](int key, const bf16_t *value) {
            const bool seen = (key <= pos) & ((key >= w_lo) | (key < a.sinks));
            if (!__any(seen)) return;
#pragma unroll
            for (int d = 0; d < L::kOut; ++d)
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    const int col = 32 * d + 2 * e + 4 * h;
                    f32x4_t y = {0.f, 0.f, 0.f, 0.f};
                    if (seen && col < head_dim) y = nonfinite4(value, col);
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[d][e + i] += y[i];
                    __builtin_amdgcn_sched_barrier(0);  // a few at a time: rare, and no registers for more
                }
        });
#pragma unroll
        for (int d = 0; d < L::kOut; ++d)
#pragma unroll
            for (int e = 0; e < 16; ++e) o[d][e] = x[d][e] != 0.f ? x[d][e] : o[d][e];
    }

    const __amdgpu_buffer_rsrc_t part =
        part_rsrc(slots + (int64_t)it.first_slot * L::kSlotFloats, (uint32_t)splits * L::kSlotFloats * 4);
    if (valid) {
        const int64_t q_row = it.q0 + tok;
        const uint32_t slot = (uint32_t)it.split * L::kSlotFloats * 4;
        const int row = 32 * wave + r;
#pragma unroll
        for (int d = 0; d < L::kOut; ++d)
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
                const int at = 32 * d + 2 * e + 4 * h;
                const f32x4_t x = {o[d][e], o[d][e + 1], o[d][e + 2], o[d][e + 3]};
                if (at >= head_dim) continue;
                if (splits == 1)
                    store_row4<bf16_t>(a, q_row, q_head, at, x, l);
                else
                    part_store(part, slot + (row * D + at) * 4, x);
            }
        if (h == 0) {
            if (splits == 1) {
                if (a.lse) a.lse[q_row * a.q_heads + q_head] = lse_of(m, l);
            } else {
                part_store1(part, slot + (kTileRows * D + row) * 4, m);
                part_store1(part, slot + (kTileRows * D + kTileRows + row) * 4, l);
            }
        }
    }
    if (splits == 1) return;

    uint32_t *counter = counters + it.first_slot;
    if (!arrive_last(counter, (uint32_t)splits, &sm.flag)) return;
    const auto region = [&](int w) { return w == 0 ? k_even : w == 1 ? v_even : w == 2 ? k_odd : v_odd; };
    add_splits<bf16_t, D, kTileRows, kTileMaxSplits, 4>(a, it, splits, row0, min(kTileRows, rows - row0), part, region, sm);
    if (tid == 0) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

template <typename T, int D, int U, bool kOnce>
__global__ __launch_bounds__(kThreads, D == 64 ? 4 : 2) void stream_kernel(AttnArgs a, uint32_t *counters, float *slots) {
    using S = Stream<T, D, U>;
    __shared__ __align__(16) unsigned char lds[kWaves][S::kWaveBytes];
    __shared__ StreamSmem sm;
    stream_item<T, D, U, kOnce>(a, kTakeAll, blockIdx.x, gridDim.x, counters, slots, lds[0], lds[1], lds[2], lds[3], sm);
}

// Workgroups below `tiles` take the tile items, the others the streaming
// items, each with counters and slots of its own: in a batch of both, the
// ones compute while the others read.
template <int D, int U, bool kFull>
__global__ __launch_bounds__(kThreads, 2) void tile_kernel(AttnArgs a, int tiles, uint32_t *counters, float *slots) {
    // Two buffers of K and V. They are variables of their own, and the loop names them statically, so that the
    // compiler sees that a buffer's loads in flight have nothing to do with reads of the other one.
    constexpr int kBytes = Tile<D>::kBytes > Stream<bf16_t, D>::kWaveBytes ? Tile<D>::kBytes : Stream<bf16_t, D>::kWaveBytes;
    __shared__ __align__(16) unsigned char k_even[kBytes], v_even[kBytes], k_odd[kBytes], v_odd[kBytes];
    __shared__ StreamSmem sm;
    const int index = blockIdx.x;
    if (index < tiles)
        tile_item<D, U, kFull>(a, gridDim.x == (unsigned)tiles ? kTakeAll : kTakeLong, index, tiles, counters, slots,
                            k_even, v_even, k_odd, v_odd, sm);
    else
        stream_item<bf16_t, D, U, true>(a, kTakeShort, index - tiles, gridDim.x - tiles, counters + kMostSplits,
                               slots + (int64_t)kMostSplits * Tile<D>::kSlotFloats, k_even, v_even, k_odd, v_odd, sm);
}

// ----------------------------------------------------------------------------
// Launches and workspace
// ----------------------------------------------------------------------------
// The groups that a launch splits have at most 4/3 * its target parts.
constexpr size_t kCounterBytes = (size_t)2 * kMostSplits * sizeof(uint32_t);
static_assert(kCounterBytes == SGMV_ATTENTION_COUNTER_BYTES, "what callers clear");
static_assert(4 * kStreamTarget <= 3 * kMostSplits && 4 * kTileTarget <= 3 * kMostSplits, "slots for every split");

// The most groups of `rows` packed rows that requests of up to max_q_len
// tokens, T in all, can make: every request's last group may be part full.
int64_t most_groups(const AttnArgs &a, int64_t requests, int rows) {
    const int64_t per = ((int64_t)a.max_q_len * a.group + rows - 1) / rows;
    const int64_t by_rows = (int64_t)a.T * a.group / rows + requests;
    return per * requests < by_rows ? per * requests : by_rows;
}

// A launch: workgroups for tile items, then for streaming items.
struct Grid {
    int64_t tiles, streams;
};

Grid grid_of(const AttnArgs &a) {
    if (a.dtype != SGMV_BF16) return {0, most_groups(a, a.num_requests, kStreamRows) * a.kv_heads + kStreamTarget};
    // A batch whose requests are all short is the streaming kernel's alone.
    const int64_t rows = (int64_t)a.max_q_len * a.group;
    const int64_t tiles_each = ((rows < kShortRows ? rows : kShortRows) + kStreamRows - 1) / kStreamRows;
    const int64_t streams = tiles_each * a.num_requests * a.kv_heads + kStreamTarget;
    if (rows <= kShortRows) return {0, streams};
    // Otherwise requests go to the two kinds of items by their rows. At most T * group / (kShortRows + 1) are long; a
    // batch of one request has tile items only.
    const int64_t could = (int64_t)a.T * a.group / (kShortRows + 1);
    const bool one = a.num_requests == 1;
    const int64_t longs = one || could >= a.num_requests ? a.num_requests : could;
    return {most_groups(a, longs, kTileRows) * a.kv_heads + kTileTarget, one ? 0 : streams};
}

template <typename T>
auto stream_kernel_of(const AttnArgs &a) {
    const bool once = (int64_t)a.max_q_len * a.group <= kStreamRows;  // a request is one row tile
    if (a.head_dim <= 64) return once ? stream_kernel<T, 64, 64, true> : stream_kernel<T, 64, 64, false>;
    if (a.head_dim <= 96) return once ? stream_kernel<T, 128, 96, true> : stream_kernel<T, 128, 96, false>;
    return once ? stream_kernel<T, 128, 128, true> : stream_kernel<T, 128, 128, false>;
}

}  // namespace

size_t attention_workspace_bytes(int head_dim, int dtype) {
    const size_t d = head_dim <= 64 ? 64 : 128;
    const size_t stream = kStreamRows * d + 2 * kStreamRows;
    const size_t tile = dtype == SGMV_BF16 ? kTileRows * d + 2 * kTileRows : 0;
    return kCounterBytes + (size_t)kMostSplits * (stream + tile) * sizeof(float);
}

int64_t attention_workgroups(const AttnArgs &a) {
    const Grid g = grid_of(a);
    return g.tiles + g.streams;
}

hipError_t launch_paged_attention(const AttnArgs &a, hipStream_t st) {
    uint32_t *counters = static_cast<uint32_t *>(a.workspace);
    float *slots = reinterpret_cast<float *>(static_cast<char *>(a.workspace) + kCounterBytes);
    const Grid g = grid_of(a);
    const dim3 grid((unsigned)(g.tiles + g.streams));
    if (g.tiles == 0) {
        const auto kernel = a.dtype == SGMV_BF16 ? stream_kernel_of<bf16_t>(a) : stream_kernel_of<float>(a);
        hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, st, a, counters, slots);
    } else {
        const auto kernel = a.head_dim == 64    ? tile_kernel<64, 64, true>
                            : a.head_dim == 128 ? tile_kernel<128, 128, true>
                            : a.head_dim < 64   ? tile_kernel<64, 64, false>
                            : a.head_dim <= 96  ? tile_kernel<128, 96, false>
                                                : tile_kernel<128, 128, false>;
        hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, st, a, (int)g.tiles, counters, slots);
    }
    return hipGetLastError();
}

}  // namespace sgmv
