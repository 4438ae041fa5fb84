// Internal interface between the entry points for several adapters per token
// (route_api.cpp) and their kernels (route_sort.hip, route_rows.hip). Not
// installed; callers use include/sgmv.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace sgmv {

struct SortArgs {
    const int32_t *choice;
    int n, num_adapters;  // n choices in all
    int32_t *seg_start, *seg_adapter;
    int num_segments;
    int32_t *order, *place;
    uint32_t *counts;  // workspace: [blocks][num_adapters]
};

// T rows in token order, `rows` in segment order; a pointer that a call does not have is NULL.
struct RowsArgs {
    void *out;  // spread: Xs; combine: Y; grad: dYs
    int64_t out_stride;
    const void *tokens;  // spread: X; combine: base; grad: dY
    int64_t tokens_stride;
    const void *sorted;  // combine, grad: Ys
    int64_t sorted_stride;
    int rows;
    const int32_t *place;
    const float *weight;
    float *dweight;
    int T, choices, d, dtype;
};

size_t sort_workspace_bytes(int n, int num_adapters);
hipError_t launch_sort_tokens(const SortArgs &a, hipStream_t st);
int64_t rows_workgroups(const RowsArgs &a);  // at most, of any of the three
hipError_t launch_spread_rows(const RowsArgs &a, hipStream_t st);
hipError_t launch_combine_rows(const RowsArgs &a, hipStream_t st);
hipError_t launch_combine_rows_grad(const RowsArgs &a, hipStream_t st);

}  // namespace sgmv
