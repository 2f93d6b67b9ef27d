// grouped.cuh -- launch interface of the experts' operators: products grouped
// by expert (16-bit and 8-bit), and the row operators between them.
#pragma once

#include "moe_internal.cuh"

namespace moe {

// Sticky bits of the operators' error word (moe_grouped_status) are the
// kErr* bits of moe_internal.cuh: kErrBadId for an offsets table that does not
// ascend from >= 0 to <= rows, kErrTimeout for a bounded wait that ran out.

// One product: `a` is the row-major left side (x or dy), `w` the weights (the
// second row-major side of a weight gradient), `out` the result.
struct GroupedCall {
    int64_t rows;
    int E, d_in, d_out;
    int dtype, out_dtype, accumulate;
    const int32_t* offsets;
    int64_t x_stride, y_stride;
    const void* a;
    const void* w;
    void* out;
    const float* a_scale;      // 8-bit: scale of each row, of each output channel
    const float* w_scale;
};

enum GroupedOp { kOpGemm = 0, kOpDgrad = 1, kOpWgrad = 2 };

moe_status_t launch_grouped(GroupedOp op, const GroupedCall& c, cudaStream_t stream);

struct RowsCall {
    int64_t rows;
    int cols, dtype;
    const void* a;             // x, or gate
    const void* b;             // up, or nullptr
    int64_t in_stride;
    const void* dh;            // gradient of h (swiglu_grad)
    int64_t dh_stride;
    void* out;                 // h, codes or dgate
    void* out2;                // dup
    int64_t out_stride;
    float* scale;
};
cudaError_t launch_swiglu(const RowsCall& c, cudaStream_t stream);
cudaError_t launch_swiglu_grad(const RowsCall& c, cudaStream_t stream);
cudaError_t launch_i8_rows(const RowsCall& c, cudaStream_t stream);

// Reads and clears the current device's error word.
moe_status_t grouped_status_read();

}  // namespace moe
