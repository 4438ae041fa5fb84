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
// by all of its heads and comes from L2 after the first.
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

// One unit of work, on one lane: in the rotated part of a head, kVec pairs
// (two 16-byte vectors: the pairs' halves, or 2 kVec neighbours when
// interleaved); elsewhere one 16-byte vector to copy. Lanes of a wave take
// neighbouring units, so a wave reads and writes whole rows.
template <typename T>
__global__ __launch_bounds__(kThreads) void rope_append_kernel(RopeArgs a, int rot_units, int copy_units, int v_units,
                                                               int units) {
    constexpr int kVec = Elem<T>::kPerVec;
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
        const int at = is_v ? part * kVec : a.rot_dim + (part - rot_units) * kVec;
        st16(dst + at, ld16_stream(src + at));
        return;
    }
    const int first = a.interleaved ? part * 2 * kVec : part * kVec;
    const int second = first + (a.interleaved ? kVec : a.rot_dim / 2);
    float x[2 * kVec], y[2 * kVec], cs[2 * kVec];
    const uint4 lo = ld16_stream(src + first), hi = ld16_stream(src + second);
    const float *turn = a.table + ((int64_t)pos * (a.rot_dim / 2) + part * kVec) * 2;
#pragma unroll
    for (int i = 0; i < 2 * kVec; i += 4) widen<float>(ld16(turn + i), reinterpret_cast<float(&)[4]>(cs[i]));
    widen<T>(lo, reinterpret_cast<float(&)[kVec]>(x[0]));
    widen<T>(hi, reinterpret_cast<float(&)[kVec]>(x[kVec]));
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        const float c = cs[2 * i], s = cs[2 * i + 1];
        const float xa = a.interleaved ? x[2 * i] : x[i], xb = a.interleaved ? x[2 * i + 1] : x[i + kVec];
        const float ya = xa * c - xb * s, yb = xb * c + xa * s;
        if (a.interleaved) {
            y[2 * i] = ya;
            y[2 * i + 1] = yb;
        } else {
            y[i] = ya;
            y[i + kVec] = yb;
        }
    }
    st16(dst + first, narrow<T>(reinterpret_cast<const float(&)[kVec]>(y[0])));
    st16(dst + second, narrow<T>(reinterpret_cast<const float(&)[kVec]>(y[kVec])));
}

}  // namespace

hipError_t launch_rope_table(const RopeTableArgs &a, hipStream_t st) {
    const int64_t n = (int64_t)a.max_position * a.half;
    const int64_t blocks = (n + kThreads - 1) / kThreads;
    hipLaunchKernelGGL(rope_table_kernel, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(kThreads), 0, st, a);
    return hipGetLastError();
}

hipError_t launch_rope_append(const RopeArgs &a, hipStream_t st) {
    const int vec = a.dtype == SGMV_BF16 ? 8 : 4;
    const int rot_units = a.rot_dim / (2 * vec), copy_units = (a.head_dim - a.rot_dim) / vec;
    const int v_units = a.head_dim / vec;
    const int units = (a.q_heads + a.kv_heads) * (rot_units + copy_units) + a.kv_heads * v_units;
    const dim3 grid((unsigned)a.T, (unsigned)((units + kThreads - 1) / kThreads));
    if (a.dtype == SGMV_BF16)
        hipLaunchKernelGGL((rope_append_kernel<bf16_t>), grid, dim3(kThreads), 0, st, a, rot_units, copy_units,
                           v_units, units);
    else
        hipLaunchKernelGGL((rope_append_kernel<float>), grid, dim3(kThreads), 0, st, a, rot_units, copy_units,
                           v_units, units);
    return hipGetLastError();
}

}  // namespace sgmv
