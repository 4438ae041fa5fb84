// Rows to segment order and back, with weights, and the gradients
// (sgmv_spread_rows, sgmv_combine_rows, sgmv_combine_rows_grad).
//
// What bounds them: HBM. A lane takes 16 bytes of a token's row: spread reads
// them once and writes them to each of the token's rows in segment order;
// combine reads them from each of these and writes their sum once; grad reads
// dY's and Ys's and keeps the products' sums. Going by tokens rather than by
// rows in segment order, every element is read once and written once, and a sum
// has one lane and one order; only grad reads a token's dY again for every four
// choices after the first four.
//
// Measured (kernels alone, bf16): 4583 tokens to 17415 rows of 8192, 360 MB, 69
// us (5.2 TB/s); back, weighted, onto a base, 435 MB, 66 us (6.5); the gradient
// of 4583 tokens over 8700 rows of 4096, 180 MB, 32 us (5.6); 64 tokens and 115
// rows of 4096 2.9 us each way. The halves of a workgroup, 128 threads, made
// no difference. The gradient of 4583 tokens a call, of eight choices over rows
// of 4096 115 us; of two over rows of 512 10.3 us, and of 64, where 8 lanes of a
// token's 256 have something to do, 8.9.
#include "route_launch.h"
#include "sgmv.h"
#include "sgmv_common.h"

namespace sgmv {

namespace {

constexpr int kThreads = 256;
constexpr int kAtOnce = 4;  // a token's choices whose rows are read together

// Rows in segment order are read once, as streams: 4583 tokens' gradient pass over 8700 rows of 4096 in bf16 (289 MB, two
// calls) 55 us, and 61 with ordinary loads. Results are written as streams by calls that move more than the last-level
// cache holds (256 MB), and left in the caches for the calls behind them by others: 17415 rows of 8192 (435 MB) combined
// in 67 us, and 73 with ordinary stores; 13300 of 4096 (109 MB) in 21 both ways.
constexpr int64_t kStreamBytes = (int64_t)256 << 20;

template <bool kStream>
__device__ __forceinline__ void store_row(void *p, uint4 v) {
    if constexpr (kStream)
        __builtin_nontemporal_store(u32x4_t{v.x, v.y, v.z, v.w}, (gvec_t *)p);
    else
        st16(p, v);
}

template <typename T>
__device__ __forceinline__ T *row_at(void *base, int64_t stride, int row, int vec) {
    return static_cast<T *>(base) + (int64_t)row * stride + vec * Elem<T>::kPerVec;
}
template <typename T>
__device__ __forceinline__ const T *row_at(const void *base, int64_t stride, int row, int vec) {
    return static_cast<const T *>(base) + (int64_t)row * stride + vec * Elem<T>::kPerVec;
}

// Unit u of the launch: 16 bytes `vec` of token t's row. A row's units are a multiple of 64 lanes apart, or rows of few
// units share a wave.
struct Unit {
    int t, vec;
    bool on;
};
__device__ __forceinline__ Unit unit_of(const RowsArgs &a, int vecs, int shift, int per_row) {
    const int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    Unit x;
    if (shift < 6) {  // 1 << shift lanes a row
        x.t = (int)min(u >> shift, (int64_t)INT32_MAX);
        x.vec = (int)(u & ((1 << shift) - 1));
    } else {
        x.t = (int)(blockIdx.x / per_row);
        x.vec = (int)(blockIdx.x % per_row) * kThreads + threadIdx.x;
    }
    x.on = x.t < a.T && x.vec < vecs;
    return x;
}

template <typename T, bool kStream>
__global__ __launch_bounds__(kThreads) void spread_kernel(RowsArgs a, int vecs, int shift, int per_row) {
    const Unit u = unit_of(a, vecs, shift, per_row);
    if (!u.on) return;
    const uint4 x = ld16_stream(row_at<T>(a.tokens, a.tokens_stride, u.t, u.vec));
    const int32_t *place = a.place + (int64_t)u.t * a.choices;
    for (int j = 0; j < a.choices; ++j) {
        const int p = place[j];
        if ((unsigned)p < (unsigned)a.rows) store_row<kStream>(row_at<T>(a.out, a.out_stride, p, u.vec), x);
    }
}

template <typename T, bool kStream>
__global__ __launch_bounds__(kThreads) void combine_kernel(RowsArgs a, int vecs, int shift, int per_row) {
    constexpr int N = Elem<T>::kPerVec;
    const Unit u = unit_of(a, vecs, shift, per_row);
    if (!u.on) return;
    float sum[N];
#pragma unroll
    for (int e = 0; e < N; ++e) sum[e] = 0.f;
    if (a.tokens) widen<T>(ld16(row_at<T>(a.tokens, a.tokens_stride, u.t, u.vec)), sum);
    const int64_t at = (int64_t)u.t * a.choices;
    for (int j0 = 0; j0 < a.choices; j0 += kAtOnce) {
        uint4 x[kAtOnce];
        float w[kAtOnce];
        bool has[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int j = j0 + i;
            const int p = j < a.choices ? a.place[at + j] : -1;
            has[i] = (unsigned)p < (unsigned)a.rows;
            if (has[i]) {
                w[i] = a.weight ? a.weight[at + j] : 1.f;
                x[i] = ld16_stream(row_at<T>(a.sorted, a.sorted_stride, p, u.vec));
            }
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            if (!has[i]) continue;
            float y[N];
            widen<T>(x[i], y);
#pragma unroll
            for (int e = 0; e < N; ++e) sum[e] = __builtin_fmaf(w[i], y[e], sum[e]);
        }
    }
    store_row<kStream>(row_at<T>(a.out, a.out_stride, u.t, u.vec), narrow<T>(sum));
}

// A workgroup takes a token, whose row its lanes share; a choice's products are summed per lane over the row, then over
// the wave and over the waves, in that order.
template <typename T, bool kStream>
__global__ __launch_bounds__(kThreads) void grad_kernel(RowsArgs a, int vecs) {
    constexpr int N = Elem<T>::kPerVec, kW = kThreads / kWave;
    __shared__ float s_sum[kAtOnce][kW];
    const int t = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t at = (int64_t)t * a.choices;
    for (int j0 = 0; j0 < a.choices; j0 += kAtOnce) {
        int p[kAtOnce];
        float w[kAtOnce], dot[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int j = j0 + i;
            p[i] = j < a.choices ? a.place[at + j] : -1;
            if ((unsigned)p[i] >= (unsigned)a.rows) p[i] = -1;
            w[i] = a.out && a.weight && p[i] >= 0 ? a.weight[at + j] : 1.f;
            dot[i] = 0.f;
        }
        for (int v = tid; v < vecs; v += kThreads) {
            float g[N];
            widen<T>(ld16(row_at<T>(a.tokens, a.tokens_stride, t, v)), g);
            uint4 x[kAtOnce];
            if (a.dweight) {
#pragma unroll
                for (int i = 0; i < kAtOnce; ++i)
                    if (p[i] >= 0) x[i] = ld16_stream(row_at<T>(a.sorted, a.sorted_stride, p[i], v));
            }
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                if (p[i] < 0) continue;
                float y[N];
                if (a.out) {
#pragma unroll
                    for (int e = 0; e < N; ++e) y[e] = w[i] * g[e];
                    store_row<kStream>(row_at<T>(a.out, a.out_stride, p[i], v), narrow<T>(y));
                }
                if (a.dweight) {
                    widen<T>(x[i], y);
#pragma unroll
                    for (int e = 0; e < N; ++e) dot[i] = __builtin_fmaf(g[e], y[e], dot[i]);
                }
            }
        }
        if (!a.dweight) continue;
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
#pragma unroll
            for (int o = 32; o > 0; o >>= 1) dot[i] += __shfl_xor(dot[i], o);
            if (lane == 0) s_sum[i][wave] = dot[i];
        }
        __syncthreads();
        if (tid < kAtOnce && j0 + tid < a.choices) {
            float sum = 0.f;
#pragma unroll
            for (int q = 0; q < kW; ++q) sum += s_sum[tid][q];
            a.dweight[at + j0 + tid] = sum;
        }
        __syncthreads();
    }
}

int vecs_of(const RowsArgs &a) { return a.d / (a.dtype == SGMV_BF16 ? 8 : 4); }

struct Shape {
    int vecs, shift, per_row;  // as Unit
    int64_t blocks;
};
Shape shape_of(const RowsArgs &a) {
    Shape s;
    s.vecs = vecs_of(a);
    s.shift = 0;
    while (s.shift < 6 && 1 << s.shift < s.vecs) ++s.shift;
    s.per_row = (s.vecs + kThreads - 1) / kThreads;
    s.blocks = s.shift < 6 ? (((int64_t)a.T << s.shift) + kThreads - 1) / kThreads : (int64_t)a.T * s.per_row;
    return s;
}

}  // namespace

int64_t rows_workgroups(const RowsArgs &a) {
    const int64_t n = shape_of(a).blocks;
    return n > a.T ? n : a.T;
}

// Launches the call's form of a kernel and returns its error; `rows`: rows of d elements that the call moves at most.
#define SGMV_ROWS_LAUNCH(kernel, rows, ...)                                                        \
    do {                                                                                           \
        const bool bf16 = a.dtype == SGMV_BF16;                                                    \
        const bool stream = (int64_t)(rows) * a.d * (bf16 ? 2 : 4) > kStreamBytes;                 \
        const auto k = bf16 ? (stream ? kernel<bf16_t, true> : kernel<bf16_t, false>)              \
                            : (stream ? kernel<float, true> : kernel<float, false>);               \
        hipLaunchKernelGGL(k, __VA_ARGS__);                                                        \
        return hipGetLastError();                                                                  \
    } while (0)

hipError_t launch_spread_rows(const RowsArgs &a, hipStream_t st) {
    const Shape s = shape_of(a);
    SGMV_ROWS_LAUNCH(spread_kernel, (int64_t)a.T * (a.choices + 1), dim3((unsigned)s.blocks), dim3(kThreads), 0, st, a, s.vecs,
                     s.shift, s.per_row);
}

hipError_t launch_combine_rows(const RowsArgs &a, hipStream_t st) {
    const Shape s = shape_of(a);
    SGMV_ROWS_LAUNCH(combine_kernel, (int64_t)a.T * (a.choices + (a.tokens ? 2 : 1)), dim3((unsigned)s.blocks), dim3(kThreads), 0,
                     st, a, s.vecs, s.shift, s.per_row);
}

hipError_t launch_combine_rows_grad(const RowsArgs &a, hipStream_t st) {
    SGMV_ROWS_LAUNCH(grad_kernel, (int64_t)a.T * (a.choices * ((a.out != nullptr) + (a.dweight != nullptr)) + 1),
                     dim3((unsigned)a.T), dim3(kThreads), 0, st, a, vecs_of(a));
}

#undef SGMV_ROWS_LAUNCH

}  // namespace sgmv
