// The tile kernel of trees, and the launch that adds up split groups: part of
// kv_attention.hip where it is compiled for trees (it has the LDS layouts, the
// products and the launches).
//
// The tile kernel is the causal one's (128 rows on four waves, tiles of 64 keys
// in two buffers) with three differences. Its rows see the cached keys alike,
// so that a tile is bounded by the request, not by the row, and only tiles that
// reach past the cached keys (for n new tokens (n + 62) / 64 + 1 at most) or lie
// on a window's edge look at masks. A row tile of up to 64 rows, which a request
// with heads of its own has, would leave two waves idle: they take the other half
// of each tile's keys, and the halves' results meet in LDS. And a split group's
// parts are added up by another launch.
//
// What bounds it: with many rows the matrix cores and the softmax beside them,
// at the clock that the power limit leaves (128 trees of 64 tokens behind 127
// to 4095, 64 heads on 8: 955 us, 636 TFLOP/s, with the weights' second half
// 960; of the 35 tiles of a group the last two hold the tree, of which a token
// sees a tenth). With few rows HBM: 64 trees of 17 to 64 tokens behind up to
// 2047, 32 heads of their own, 239 us, 5.05 TB/s. There an item's loop runs at
// HBM's rate, 2.4 us a tile on two workgroups a CU, and its begin (finding it,
// pages, first tile) and end, 12 us of 53, are what is left.
// Tried for few rows, 64 requests of 64 rows and 1000 keys, 254 us as it is: K
// and V waited for separately and buffers filled as soon as they are read, 254;
// two waves of 32 rows and tiles of 32 keys, four workgroups a CU, 241, but 170
// for 139 where there are 512 groups, not 2048; workgroups that stay and take
// every 512th item, 264; three workgroups a CU, registers spilled.

// Every wave's loads to LDS have landed, and its reads and writes of LDS are done.
__device__ __forceinline__ void landed_barrier() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

using TileKind = TreeKind<kTileRows, kTileKeys, kTileTarget, kTileMinChunk, kTileMinTiles, kTileMaxSplits>;

// U as for Stream; kFull: head_dim is D.
template <int D, int U, bool kFull>
__device__ __forceinline__ void tree_tile_item(const AttnArgs &a, const Item &it, float *slots, unsigned char *k_even,
                                               unsigned char *v_even, unsigned char *k_odd, unsigned char *v_odd,
                                               StreamSmem &sm) {
    using L = Tile<D, U>;
    using S = Stream<bf16_t, D>;  // the LDS layouts of a row
    constexpr int CH = L::kChunks, NL = L::kLoads;
    const int tid = this_thread(), lane = tid & 63, wave = tid >> 6, h = lane >> 5, r = lane & 31;
    const int rows = it.n * a.group, row0 = it.row_tile * kTileRows;
    const int pa = it.p0 - 1, pb = it.p0 + it.n - 1;  // first and last position that a row can have
    const TileRun run = tile_run<kTileKeys>(pa, pb, a.window, a.sinks);
    const int splits = run.count > it.size ? (run.count + it.size - 1) / it.size : 1;
    if (it.split >= splits) return;
    const int t0 = it.split * it.size, t1 = min(run.count, t0 + it.size);

    // Up to 64 rows: two waves have them, for the first half of each key tile's keys, and two for the second half.
    const bool halves = rows - row0 <= kTileRows / 2;
    const int row_block = halves ? wave & 1 : wave, key_block = halves ? wave >> 1 : 0;
    const int wrow = row0 + 32 * row_block;  // this wave's rows; past the last row it only helps loading
    const bool live_wave = wrow < rows;
    const int my = wrow + r, tok = my / a.group;
    const bool valid = my < rows;
    const int q_head = it.head * a.group + my % a.group;
    const TreeRow mask = tree_row(a, it, tok, valid);
    const int cached = valid ? it.p0 : 0;  // keys that are seen for their position
    const int w_lo = a.window > 0 ? it.p0 + mask.seen() - a.window : 0;
    const int pa_lo = a.window > 0 ? pa - a.window + 1 : 0, pb_lo = a.window > 0 ? pb - a.window + 1 : 0;
    const int head_dim = kFull ? D : a.head_dim, nch = head_dim / 8;
    if (!kFull) {  // the chunks past the head stay zero
        for (int i = tid; i < L::kBytes / 16; i += kThreads)
            for (unsigned char *buf : {k_even, v_even, k_odd, v_odd})
                reinterpret_cast<uint4 *>(buf)[i] = make_uint4(0, 0, 0, 0);
        __syncthreads();
    }

    const int row_bytes = head_dim * 2, page_mask = (1 << a.page_shift) - 1;
    int pages = 0;  // of 16 tiles' 64 16-key blocks, one per lane
    const auto load_pages = [&](int i) {
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
    load_pages(0);
    // Tile i goes straight to LDS: thread t fills 16-byte slots t, t + 256, ... of a buffer with the chunks that the
    // swizzles put there. Rows of a 16-key block are one run of memory, so a thread's offset in it is the same for all.
    constexpr int kBlockThreads = 16 * CH;  // threads that fill one 16-key block
    const int slot_row = tid % kBlockThreads / CH, slot_chunk = tid % CH;
    const int k_chunk = S::k_slot(slot_row, slot_chunk) - slot_row * CH, v_chunk = S::v_slot(slot_row, slot_chunk) - slot_row * CH;
    const uint32_t k_off = slot_row * row_bytes + k_chunk * 16, v_off = slot_row * row_bytes + v_chunk * 16;
    const int wave_u = __builtin_amdgcn_readfirstlane(wave);
    const auto load_tile = [&](int i, unsigned char *kb, unsigned char *vb) {
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

    // The first tile's loads wait for their pages only, which the queries are read behind.
    const int n = t1 - t0;
    uint4 qv[L::kSteps];
    {
        const bf16_t *q = static_cast<const bf16_t *>(a.q) + (int64_t)(it.q0 + (valid ? tok : 0)) * a.q_stride +
                          (int64_t)(valid ? q_head : 0) * a.head_dim;
#pragma unroll
        for (int k = 0; k < L::kSteps; ++k) qv[k] = ld16(q + (2 * k + h < nch ? 2 * k + h : 0) * 8);
    }
    if (n > 0) load_tile(0, k_even, v_even);
    bf16x8_t qf[L::kSteps];
#pragma unroll
    for (int k = 0; k < L::kSteps; ++k)
        qf[k] = __builtin_bit_cast(bf16x8_t, valid && 2 * k + h < nch ? qv[k] : make_uint4(0, 0, 0, 0));

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

    const auto all_see = [&](int key0) {  // every row sees every key of the tile
        return key0 + kTileKeys - 1 <= pa && (pb_lo <= key0 || key0 + kTileKeys <= a.sinks);
    };
    // Tile i, whose K and V are there. kBlocks: 32-key blocks of it that a wave takes, from key_block on.
    auto step = [&](auto blocks, int i, unsigned char *kb, unsigned char *vb, unsigned char *k_next, unsigned char *v_next) {
        constexpr int kBlocks = decltype(blocks)::value;
        if (i + 1 < n) {
            if ((i + 1) % 16 == 0) load_pages(i + 1);
            load_tile(i + 1, k_next, v_next);
        }
        const int key0 = run.tile(t0 + i) * kTileKeys;
        const int first = kBlocks == 1 ? key_block : 0;  // 32-key block
        const unsigned char *k_from = kb + first * 32 * CH * 16, *v_from = vb + first * 32 * CH * 16;
        f32x16_t s[kBlocks];
        if (live_wave) {
            bf16x8_t kf[kBlocks][L::kSteps];
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
#pragma unroll
                for (int k = 0; k < L::kSteps; ++k) kf[b][k] = *reinterpret_cast<const bf16x8_t *>(k_from + k_at[k] + b * 32 * CH * 16);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int b = 0; b < kBlocks; ++b)
#pragma unroll
                for (int e = 0; e < 16; ++e) s[b][e] = 0.f;
#pragma unroll
            for (int b = 0; b < kBlocks; ++b)
#pragma unroll
                for (int k = 0; k < L::kSteps; ++k) s[b] = mfma32(kf[b][k], qf[k], s[b]);
        }
        const bool whole = all_see(key0);
        if (!whole) {
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
        if (live_wave) {
            bf16x8_t vf[2][L::kOut];  // V fragments of two 16-key steps
#pragma unroll
            for (int d = 0; d < L::kOut; ++d) vf[0][d] = read_columns(v_from + v_at[d], 8 * CH * 16);
            if (!whole) {
#pragma unroll
                for (int b = 0; b < kBlocks; ++b) {
                    const int key_b = key0 + 32 * (first + b);
                    const uint32_t bits = mask.bits(key_b - it.p0) >> (4 * h);
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int key = key_b + 8 * (e / 4) + 4 * h + e % 4;
                        bool seen = (key < cached) & ((key >= w_lo) | (key < a.sinks));
                        seen |= (bits >> (8 * (e / 4) + e % 4) & 1) != 0;
                        s[b][e] = seen ? s[b][e] : kNone;
                    }
                }
            }
            float top = kNone;
#pragma unroll
            for (int b = 0; b < kBlocks; ++b)
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
            for (int t = 0; t < 2 * kBlocks; ++t) {  // 16 keys: this lane's weight slots are 16 t + 4 h + {0..3, 8..11}
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
                if (t + 1 < 2 * kBlocks) {
#pragma unroll
                    for (int d = 0; d < L::kOut; ++d)
                        vf[(t + 1) & 1][d] = read_columns(v_from + v_at[d] + 16 * (t + 1) * CH * 16, 8 * CH * 16);
                }
#pragma unroll
                for (int d = 0; d < L::kOut; ++d) o[d] = mfma32(vf[t & 1][d], p, o[d]);
#pragma unroll
                for (int d = 0; d < L::kOut; ++d) o[d] = mfma32(vf[t & 1][d], p_lo, o[d]);
            }
        }
        landed_barrier();
    };
    if (tid == 0) sm.odd = 0;
    const auto steps = [&](auto blocks) {
        for (int i = 0; i < n; i += 2) {
            step(blocks, i, k_even, v_even, k_odd, v_odd);
            if (i + 1 < n) step(blocks, i + 1, k_odd, v_odd, k_even, v_even);
        }
    };
    landed_barrier();
    if (halves)
        steps(std::integral_constant<int, 1>{});
    else
        steps(std::integral_constant<int, 2>{});
    l = swap32_sum(l);
    if (halves) {  // the second halves' results, to the waves with the first
        f32x4_t *there = reinterpret_cast<f32x4_t *>(row_block == 0 ? k_even : v_even) + lane;
        float *more = reinterpret_cast<float *>(k_odd) + row_block * 128 + lane;
        if (key_block == 1) {
#pragma unroll
            for (int d = 0; d < L::kOut; ++d)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    there[(4 * d + e) * 64] = f32x4_t{o[d][4 * e], o[d][4 * e + 1], o[d][4 * e + 2], o[d][4 * e + 3]};
            more[0] = m;
            more[64] = l;
        }
        lds_barrier();
        if (key_block == 0) {
            const float m2 = more[0], top = fmaxf(m, m2);
            const float keep = exp2_fast(m - ref_of(top)), keep2 = exp2_fast(m2 - ref_of(top));
            m = top;
            l = l * keep + more[64] * keep2;
#pragma unroll
            for (int d = 0; d < L::kOut; ++d)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const f32x4_t x = there[(4 * d + e) * 64];
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[d][4 * e + i] = o[d][4 * e + i] * keep + x[i] * keep2;
                }
        }
    }
    const bool mine = valid && key_block == 0;  // this wave has its rows' results
    // A sum over a value that is not finite is that value, which was cleared, or met a weight's zero low part.
    bool odd = sm.odd != 0;
#pragma unroll
    for (int d = 0; d < L::kOut; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) odd |= o[d][e] != o[d][e];
    if (__any(odd && mine && l == l)) {
        f32x16_t x[L::kOut];
#pragma unroll
        for (int d = 0; d < L::kOut; ++d)
#pragma unroll
            for (int e = 0; e < 16; ++e) x[d][e] = 0.f;
        each_nonfinite<bf16_t, kTileKeys>(a, it, run, t0, t1, 1, [&](int key, const bf16_t *value) {
            const bool seen = ((key < cached) & ((key >= w_lo) | (key < a.sinks))) || (mask.bits(key - it.p0) & 1) != 0;
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
    if (mine) {
        const int64_t q_row = it.q0 + tok;
        const uint32_t slot = (uint32_t)it.split * L::kSlotFloats * 4;
        const int row = 32 * row_block + r;
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
}

// ----------------------------------------------------------------------------
// Adding up the splits of a tree's groups, in a launch of its own: a group of
// 128 rows in 32 splits is 2 MB, which the last of its workgroups alone would
// read at the latency of 16 loads a lane. Here split k's workgroup adds the k-th
// part of the group's rows; the workgroups look for their groups as the
// attention's do. One request of 25 tokens behind 31000, 64 heads on 8: 66 us
// in all, 8.2 of it here (31 MB), and 104 with the last workgroup's. A launch
// without splits costs 4.6 us, where the table of pages allows any.
// ----------------------------------------------------------------------------
// Waves of its workgroups. Of 128 rows a part has 4 or more, and with 8 waves fewer come one after another: 4 requests of
// 25 tokens behind 2000, 64 heads on 8, 43.6 -> 37.8 us in all, 32 of 16 behind up to 4000 128 -> 119; 16 waves 36.5 and 119,
// but start later: 72.7 for 70.3 with the one request above. Of 16 rows 4 waves have enough: one token behind 31000 32.4 us,
// with 8 waves 33.0.
template <typename Kind>
constexpr int join_waves = Kind::kRows > kStreamRows ? 8 : 4;

// Rows [begin, end) of a group in `splits` parts; a wave takes kR of them at once, 16 loads deep, so that few parts leave
// no load without use: 4 requests of 25 tokens behind 2000 12.4 -> 8.0 us here, 32 of 16 behind up to 4000 27.0 -> 15.5.
// What it reads first waits for nothing.
template <typename T, int D, typename Kind, int kR>
__device__ __forceinline__ void join_rows(const AttnArgs &a, const Item &it, const float *part, int splits, int begin, int end) {
    constexpr int kRows = Kind::kRows, kSlot = kRows * D + 2 * kRows, kPer = D / 64, kDeep = 16 / kR, kStep = join_waves<Kind>;
    constexpr int kRegs = kR > 1 ? 1 : (Kind::kMaxSplits + 63) / 64;
    const int tid = this_thread(), lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    for (int first = begin + wave; first < end; first += kStep * kR) {
        int row[kR];
        float x[kR][kDeep][kPer], f[kR][kRegs], l[kR][kRegs], top[kR], weight[kR], sum[kR][kPer];
        const auto load = [&](int k0) {
#pragma unroll
            for (int r = 0; r < kR; ++r)
#pragma unroll
                for (int j = 0; j < kDeep; ++j)
#pragma unroll
                    for (int c = 0; c < kPer; ++c)
                        x[r][j][c] = part[(int64_t)min(k0 + j, splits - 1) * kSlot + (int64_t)row[r] * D + kPer * lane + c];
        };
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            row[r] = min(first + r * kStep, end - 1);
#pragma unroll
            for (int i = 0; i < kRegs; ++i) {
                const int k = 64 * i + lane;
                f[r][i] = k < splits ? part[(int64_t)k * kSlot + kRows * D + row[r]] : kNone;
                l[r][i] = k < splits ? part[(int64_t)k * kSlot + kRows * D + kRows + row[r]] : 0.f;
            }
        }
        load(0);
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            top[r] = kNone;
            weight[r] = 0.f;
#pragma unroll
            for (int i = 0; i < kRegs; ++i) top[r] = fmaxf(top[r], f[r][i]);
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) top[r] = fmaxf(top[r], __shfl_xor(top[r], o));
#pragma unroll
            for (int i = 0; i < kRegs; ++i) {
                f[r][i] = exp2_fast(f[r][i] - ref_of(top[r]));
                weight[r] += f[r][i] * l[r][i];
            }
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) weight[r] += __shfl_xor(weight[r], o);
#pragma unroll
            for (int c = 0; c < kPer; ++c) sum[r][c] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < kRegs; ++i) {
            for (int k0 = 64 * i; k0 < min(splits, 64 * i + 64); k0 += kDeep) {
                if (k0 > 0) load(k0);
#pragma unroll
                for (int r = 0; r < kR; ++r)
#pragma unroll
                    for (int j = 0; j < kDeep; ++j) {
                        const float w = __builtin_bit_cast(
                            float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, f[r][i]), (k0 + j) & 63));
#pragma unroll
                        for (int c = 0; c < kPer; ++c)  // a value that is not finite is that value under any weight
                            sum[r][c] += k0 + j >= splits ? 0.f : is_finite(x[r][j][c]) ? x[r][j][c] * w : x[r][j][c];
                    }
            }
        }
#pragma unroll
        for (int r = 0; r < kR; ++r) {
            if (first + r * kStep >= end) break;
            const int at = it.row_tile * kRows + row[r], head = it.head * a.group + at % a.group, col = kPer * lane;
            const int64_t q_row = it.q0 + at / a.group;
            const float inv = weight[r] > 0.f || weight[r] != weight[r] ? 1.f / weight[r] : 0.f;
            if (col < a.head_dim) {
                T *dst = static_cast<T *>(a.out) + q_row * a.out_stride + (int64_t)head * a.head_dim + col;
#pragma unroll
                for (int c = 0; c < kPer; ++c) {
                    if constexpr (sizeof(T) == 2)
                        dst[c].bits = __builtin_bit_cast(uint16_t, (__bf16)(sum[r][c] * inv));
                    else
                        dst[c] = sum[r][c] * inv;
                }
            }
            if (a.lse && lane == 0) a.lse[q_row * a.q_heads + head] = lse_of(top[r], weight[r]);
        }
    }
}

template <typename T, int D, typename Kind>
__device__ __forceinline__ void join_item(const AttnArgs &a, const Item &it, const float *slots) {
    constexpr int kRows = Kind::kRows, kSlot = kRows * D + 2 * kRows;
    const TileRun run = tile_run<Kind::kKeys>(it.p0 - 1, it.p0 + it.n - 1, a.window, a.sinks);
    const int splits = (run.count + it.size - 1) / it.size;
    if (it.split >= splits) return;
    const int live = min(kRows, it.n * a.group - it.row_tile * kRows);
    const float *part = slots + (int64_t)it.first_slot * kSlot;
    const int begin = live * it.split / splits, end = live * (it.split + 1) / splits;
    if (splits <= 4)
        join_rows<T, D, Kind, 4>(a, it, part, splits, begin, end);
    else if (splits <= 8)
        join_rows<T, D, Kind, 2>(a, it, part, splits, begin, end);
    else
        join_rows<T, D, Kind, 1>(a, it, part, splits, begin, end);
}

template <typename T, int D, typename Kind>
__global__ __launch_bounds__(join_waves<Kind> * kWave) void join_kernel(AttnArgs a, const float *slots) {
    each_split<Kind>(a, blockIdx.x, gridDim.x, [&](const Item &it) { join_item<T, D, Kind>(a, it, slots); });
}

// The most key tiles that a group of the call can have.
int64_t most_tiles(const AttnArgs &a, int keys) {
    const int64_t all = (((int64_t)a.max_blocks << a.page_shift) + keys - 1) / keys;
    if (a.window == 0) return all;
    const int64_t seen = ((int64_t)a.window + a.max_q_len) / keys + 2 + ((int64_t)a.sinks + keys - 1) / keys;
    return seen < all ? seen : all;
}
