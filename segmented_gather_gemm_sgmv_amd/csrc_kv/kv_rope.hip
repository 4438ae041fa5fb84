// Rotary positions: the table of angles (sgmv_rope_table), and the rotation of
// q and k with the write of k and v to the paged cache (sgmv_rope_append).
//
// Mathematics: pair i of a head at position p turns by the angle p f_i,
// (a, b) -> (a cos - b sin, b cos + a sin). The angles come from a table
// formed once in 64 bits: at position 131071 an fp32 product p f_i is already
// off by up to 2^-8 rad, and its sine would cost more than the rotation.
//
// What bounds sgmv_rope_append: HBM. Every q, k and v element is read once
// and written once (3 flops per element between); a token's table row is read
// by all of its heads and comes from L2 after the first. A workgroup takes 256
// units of one token (16 bytes of a row or a pair of them), so a decode step
// of 64 tokens already makes 256 workgroups.
//
// Measured: 4583 tokens of 64 + 2 x 8 heads of 128 in bf16, 190 MB, 31.4 us
// (6.05 TB/s), interleaved 37.6 us (5.1), in fp32 60.1 us (6.3); 64 tokens of
// 32 + 2 x 32 heads 3.2 us (kernel alone). A rotated part whose halves are not
// multiples of 16 bytes moves shorter runs, v and the rest of the head with it:
// 80 of 80 elements turned 28.1 us, 40 of 80 39.5 us; 126 of 128 107 us.
// sgmv_rope_table: 131072 positions of 64 pairs 89 us, 94 pairs a ns, bounded by
// pow and sincos in 64 bits; once per model.
#include "kv_launch.h"
#include "sgmv.h"
#include "sgmv_common.h"

namespace sgmv {

namespace {

constexpr int kThreads = 256;

__global__ __launch_bounds__(kThreads) void rope_table_kernel(RopeTableArgs a) {
    const int64_t n = (int64_t)a.max_position * a.half;
    for (int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x; e < n; e += (int64_t)gridDim.x * kThreads) {
        const int p = (int)(e / a.half), i = (int)(e % a.half);
        double f = pow(a.base, -(double)i / a.half);
        if (a.kind == SGMV_ROPE_LINEAR) f /= a.factor;
        if (a.kind == SGMV_ROPE_BY_PARTS) {
            const double w = 1.0 - fmin(fmax((i - a.low) / (a.high - a.low), 0.0), 1.0);
            f = f * w + f / a.factor * (1.0 - w);
        }
        double s, c;
        sincos(p * f, &s, &c);
        const float2 cs = make_float2((float)(c * a.magnitude), (float)(s * a.magnitude));
        reinterpret_cast<float2 *>(a.table)[e] = cs;
    }
}

// N consecutive elements of storage type T, N * sizeof(T) up to 16 bytes and
// aligned to that: one load or store. Rows are read once, so they are loaded
// as streams (the 70B layer's 4583 rows: 36.6 -> 31.3 us).
template <int kBytes>
struct Chunk;
template <>
struct Chunk<16> {
    typedef u32x4_t type;
};
template <>
struct Chunk<8> {
    typedef uint32_t type __attribute__((ext_vector_type(2)));
};
template <>
struct Chunk<4> {
    typedef uint32_t type;
};
template <>
struct Chunk<2> {
    typedef uint16_t type;
};

template <typename T, int N>
struct Run {
    typedef typename Chunk<N * (int)sizeof(T)>::type raw_t;
    typedef __attribute__((address_space(1))) raw_t graw_t;
    typedef __attribute__((address_space(1))) const raw_t gconst_raw_t;
    raw_t raw;
    __device__ __forceinline__ void load(const T *p) { raw = __builtin_nontemporal_load((gconst_raw_t *)p); }
    __device__ __forceinline__ void store(T *p) const { *(graw_t *)p = raw; }
    __device__ __forceinline__ void widen(float *x) const {
        T e[N];
        __builtin_memcpy(e, &raw, sizeof e);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if constexpr (sizeof(T) == 2)
                x[i] = __uint_as_float((uint32_t)e[i].bits << 16);
            else
                x[i] = e[i];
        }
    }
    __device__ __forceinline__ void narrow(const float *x) {  // to nearest-even
        T e[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if constexpr (sizeof(T) == 2)
                e[i].bits = __builtin_bit_cast(uint16_t, (__bf16)x[i]);
            else
                e[i] = x[i];
        }
        __builtin_memcpy(&raw, e, sizeof e);
    }
};

// One unit of work, on one lane: in the rotated part of a head, N pairs (two
// runs of N elements: the pairs' halves, or 2 N neighbours when interleaved);
// elsewhere one run to copy. Lanes of a wave take neighbouring units, so a
// wave reads and writes whole rows. N is as large as 16 bytes and rot_dim
// allow: a rotated half of 20 bf16 values, for instance, goes by fours.
template <typename T, int N>
__global__ __launch_bounds__(kThreads) void rope_append_kernel(RopeArgs a, int rot_units, int copy_units, int v_units,
                                                               int units) {
    const int tok = blockIdx.x;
    const int u = blockIdx.y * kThreads + threadIdx.x;
    const int pos = a.position[tok];
    if ((unsigned)pos >= (unsigned)a.max_position || u >= units) return;
    const int per_head = rot_units + copy_units;
    const int qk_units = (a.q_heads + a.kv_heads) * per_head;
    const bool is_v = u >= qk_units;
    const int w = is_v ? u - qk_units : u;
    const int row = w / (is_v ? v_units : per_head), part = w % (is_v ? v_units : per_head);
    const bool is_q = !is_v && row < a.q_heads;
    const int head = is_v || is_q ? row : row - a.q_heads;

    const T *src;
    T *dst;
    if (is_q) {
        src = static_cast<const T *>(a.q) + tok * a.q_stride + (int64_t)head * a.head_dim;
        dst = static_cast<T *>(a.q_out) + tok * a.q_out_stride + (int64_t)head * a.head_dim;
    } else {
        const int slot = a.slot[tok], page = slot >> a.page_shift;
        if (slot < 0 || page >= a.num_pages) return;
        src = static_cast<const T *>(is_v ? a.v : a.k) + tok * (is_v ? a.v_stride : a.k_stride) +
              (int64_t)head * a.head_dim;
        dst = static_cast<T *>(is_v ? a.V : a.K) +
              ((((int64_t)page * a.kv_heads + head) << a.page_shift) + (slot & ((1 << a.page_shift) - 1))) * a.head_dim;
    }
    if (is_v || part >= rot_units) {
        const int at = is_v ? part * N : a.rot_dim + (part - rot_units) * N;
        Run<T, N> r;
        r.load(src + at);
        r.store(dst + at);
        return;
    }
    const int first = a.interleaved ? part * 2 * N : part * N;
    const int second = first + (a.interleaved ? N : a.rot_dim / 2);
    Run<T, N> lo, hi;
    lo.load(src + first);
    hi.load(src + second);
    // A run of 2 N table values is aligned to 16 bytes for N > 1: rot_dim / 2 is then even.
    const float *turn = a.table + ((int64_t)pos * (a.rot_dim / 2) + part * N) * 2;
    float x[2 * N], y[2 * N], cs[2 * N];
    if constexpr (N > 1) {
#pragma unroll
        for (int i = 0; i < 2 * N; i += 4) widen<float>(ld16(turn + i), reinterpret_cast<float(&)[4]>(cs[i]));
    } else {
        const float2 t = *reinterpret_cast<const float2 *>(turn);
        cs[0] = t.x;
        cs[1] = t.y;
    }
    lo.widen(x);
    hi.widen(x + N);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float c = cs[2 * i], s = cs[2 * i + 1];
        const float xa = a.interleaved ? x[2 * i] : x[i], xb = a.interleaved ? x[2 * i + 1] : x[i + N];
        const float ya = xa * c - xb * s, yb = xb * c + xa * s;
        if (a.interleaved) {
            y[2 * i] = ya;
            y[2 * i + 1] = yb;
        } else {
            y[i] = ya;
            y[i + N] = yb;
        }
    }
    lo.narrow(y);
    hi.narrow(y + N);
    lo.store(dst + first);
    hi.store(dst + second);
}

// The largest run of elements that `most` and rot_dim allow.
int run_of(const RopeArgs &a, int most) {
    int n = most;
    while (a.rot_dim % (2 * n) != 0) n /= 2;
    return n;
}

int units_of(const RopeArgs &a, int n) {
    return (a.q_heads + a.kv_heads) * (a.rot_dim / (2 * n) + (a.head_dim - a.rot_dim) / n) + a.kv_heads * (a.head_dim / n);
}

template <typename T, int N>
void launch_run(const RopeArgs &a, hipStream_t st) {
    const int units = units_of(a, N);
    const dim3 grid((unsigned)a.T, (unsigned)((units + kThreads - 1) / kThreads));
    hipLaunchKernelGGL((rope_append_kernel<T, N>), grid, dim3(kThreads), 0, st, a, a.rot_dim / (2 * N),
                       (a.head_dim - a.rot_dim) / N, a.head_dim / N, units);
}

}  // namespace

hipError_t launch_rope_table(const RopeTableArgs &a, hipStream_t st) {
    const int64_t n = (int64_t)a.max_position * a.half;
    const int64_t blocks = (n + kThreads - 1) / kThreads;
    hipLaunchKernelGGL(rope_table_kernel, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(kThreads), 0, st, a);
    return hipGetLastError();
}

int64_t rope_append_workgroups(const RopeArgs &a) {
    const int64_t units = units_of(a, run_of(a, a.dtype == SGMV_BF16 ? 8 : 4));
    return a.T * ((units + kThreads - 1) / kThreads);
}

hipError_t launch_rope_append(const RopeArgs &a, hipStream_t st) {
    if (a.dtype == SGMV_BF16) {
        switch (run_of(a, 8)) {
            case 8: launch_run<bf16_t, 8>(a, st); break;
            case 4: launch_run<bf16_t, 4>(a, st); break;
            case 2: launch_run<bf16_t, 2>(a, st); break;
            default: launch_run<bf16_t, 1>(a, st); break;
        }
    } else {
        switch (run_of(a, 4)) {
            case 4: launch_run<float, 4>(a, st); break;
            case 2: launch_run<float, 2>(a, st); break;
            default: launch_run<float, 1>(a, st); break;
        }
    }
    return hipGetLastError();
}

}  // namespace sgmv
