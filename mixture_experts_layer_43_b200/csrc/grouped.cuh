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

// Programmatic dependent launch.  The operators are launched so that a kernel may
// start while the one before it in the stream still runs: it sets itself up
// (barriers, tensor memory, descriptors) and then waits, before its first access
// to global memory, until that kernel has finished and its writes are visible.
// Each lets its successor do the same from its own start on.
#ifdef __CUDACC__
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_let_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_chained(void (*kernel)(P...), dim3 grid, int threads, size_t smem, int cluster,
                           cudaStream_t stream, const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster; attr[1].val.clusterDim.y = 1; attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    if (e != cudaSuccess) cudaGetLastError();          // reported by the caller's status alone
    return e;
}
#endif

// Reads and clears the current device's error word.
moe_status_t grouped_status_read();

}  // namespace moe
