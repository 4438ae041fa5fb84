// The entry points for several adapters per token, of the C ABI declared in
// include/sgmv.h: argument checks, then the gfx950 kernels.
#include "sgmv.h"

#include <hip/hip_runtime.h>

#include "route_launch.h"
#include "sgmv_checks.h"

using namespace sgmv::abi;

namespace {

int hip_status(hipError_t e) { return e == hipSuccess ? SGMV_OK : SGMV_ERR_HIP; }

// One dispatch holds fewer than 2^32 work-items (its packet has 32 bits for them): 2^24 workgroups of 256 threads are one
// too many.
bool too_many(int64_t workgroups) { return workgroups >= sgmv::kMaxWorkgroups; }

constexpr int64_t kMostChoices = 1 << 24;

// Sizes that the calls share.
int check_sizes(int32_t T, int32_t choices, int32_t rows, int32_t d, int32_t dtype) {
    if (!valid_dtype(dtype)) return SGMV_ERR_DTYPE;
    if (T < 0 || rows < 0 || choices < 1 || choices > SGMV_MAX_CHOICES || !valid_dim(d)) return SGMV_ERR_SHAPE;
    if ((int64_t)T * choices > kMostChoices) return SGMV_ERR_SHAPE;
    return SGMV_OK;
}

int check_rows(const void *p, int64_t stride, int64_t rows, int32_t d, int32_t dtype) {
    if (rows > 1 && (stride < d || (double)stride * rows > (double)kMaxElems)) return SGMV_ERR_SHAPE;
    if (!aligned16(p) || (rows > 1 && stride * (dtype == SGMV_BF16 ? 2 : 4) % 16 != 0)) return SGMV_ERR_ALIGN;
    return SGMV_OK;
}

}  // namespace

extern "C" {

size_t sgmv_sort_tokens_workspace_bytes(int32_t T, int32_t choices, int32_t num_adapters) {
    if (T < 0 || choices < 1 || choices > SGMV_MAX_CHOICES || (int64_t)T * choices > kMostChoices || num_adapters < 0 ||
        num_adapters > SGMV_MAX_SORTED_ADAPTERS)
        return 0;
    return sgmv::sort_workspace_bytes(T * choices, num_adapters);
}

int sgmv_sort_tokens(const int32_t *choice, int32_t T, int32_t choices, int32_t num_adapters, int32_t *seg_start,
                     int32_t *seg_adapter, int32_t num_segments, int32_t *order, int32_t *place, void *workspace,
                     size_t workspace_bytes, void *stream) {
    if (T < 0 || choices < 1 || choices > SGMV_MAX_CHOICES || (int64_t)T * choices > kMostChoices) return SGMV_ERR_SHAPE;
    if (num_adapters < 0 || num_adapters > SGMV_MAX_SORTED_ADAPTERS) return SGMV_ERR_SHAPE;
    const int32_t n = T * choices;
    if (num_segments < (num_adapters < n ? num_adapters : n)) return SGMV_ERR_SHAPE;
    if (!seg_start || (num_segments > 0 && !seg_adapter) || (n > 0 && (!choice || !order || !place))) return SGMV_ERR_NULL;
    const size_t need = sgmv::sort_workspace_bytes(n, num_adapters);
    if (need > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < need)) return SGMV_ERR_WORKSPACE;
    const sgmv::SortArgs a{choice, n, num_adapters, seg_start, seg_adapter, num_segments, order, place,
                           static_cast<uint32_t *>(workspace)};
    return hip_status(sgmv::launch_sort_tokens(a, static_cast<hipStream_t>(stream)));
}

int sgmv_spread_rows(void *Xs, int64_t Xs_stride, int32_t rows, const void *X, int64_t X_stride,
                     const int32_t *place, int32_t T, int32_t choices, int32_t d, int32_t dtype, void *stream) {
    int st = check_sizes(T, choices, rows, d, dtype);
    if (st != SGMV_OK) return st;
    if (T == 0 || rows == 0) return SGMV_OK;
    if (!Xs || !X || !place) return SGMV_ERR_NULL;
    st = check_rows(Xs, Xs_stride, rows, d, dtype);
    if (st == SGMV_OK) st = check_rows(X, X_stride, T, d, dtype);
    if (st != SGMV_OK) return st;
    const sgmv::RowsArgs a{Xs, Xs_stride, X, X_stride, nullptr, 0, rows, place, nullptr, nullptr, T, choices, d, dtype};
    if (too_many(sgmv::rows_workgroups(a))) return SGMV_ERR_SHAPE;
    return hip_status(sgmv::launch_spread_rows(a, static_cast<hipStream_t>(stream)));
}

int sgmv_combine_rows(void *Y, int64_t Y_stride, const void *base, int64_t base_stride, const void *Ys,
                      int64_t Ys_stride, int32_t rows, const int32_t *place, const float *weight, int32_t T,
                      int32_t choices, int32_t d, int32_t dtype, void *stream) {
    int st = check_sizes(T, choices, rows, d, dtype);
    if (st != SGMV_OK) return st;
    if (T == 0) return SGMV_OK;
    if (!Y || !place || (rows > 0 && !Ys)) return SGMV_ERR_NULL;
    st = check_rows(Y, Y_stride, T, d, dtype);
    if (st == SGMV_OK && base) st = check_rows(base, base_stride, T, d, dtype);
    if (st == SGMV_OK && rows > 0) st = check_rows(Ys, Ys_stride, rows, d, dtype);
    if (st != SGMV_OK) return st;
    const sgmv::RowsArgs a{Y, Y_stride, base, base_stride, Ys, Ys_stride, rows, place, weight, nullptr, T, choices, d, dtype};
    if (too_many(sgmv::rows_workgroups(a))) return SGMV_ERR_SHAPE;
    return hip_status(sgmv::launch_combine_rows(a, static_cast<hipStream_t>(stream)));
}

int sgmv_combine_rows_grad(void *dYs, int64_t dYs_stride, float *dweight, const void *dY, int64_t dY_stride,
                           const void *Ys, int64_t Ys_stride, int32_t rows, const int32_t *place,
                           const float *weight, int32_t T, int32_t choices, int32_t d, int32_t dtype,
                           void *stream) {
    int st = check_sizes(T, choices, rows, d, dtype);
    if (st != SGMV_OK) return st;
    if (T == 0) return SGMV_OK;
    if (!dY || !place || (!dYs && !dweight) || (dweight && rows > 0 && !Ys)) return SGMV_ERR_NULL;
    st = check_rows(dY, dY_stride, T, d, dtype);
    if (st == SGMV_OK && dYs && rows > 0) st = check_rows(dYs, dYs_stride, rows, d, dtype);
    if (st == SGMV_OK && dweight && rows > 0) st = check_rows(Ys, Ys_stride, rows, d, dtype);
    if (st != SGMV_OK) return st;
    const sgmv::RowsArgs a{dYs, dYs_stride, dY, dY_stride, Ys, Ys_stride, rows, place, weight, dweight, T, choices, d, dtype};
    if (too_many(sgmv::rows_workgroups(a))) return SGMV_ERR_SHAPE;
    return hip_status(sgmv::launch_combine_rows_grad(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
