// grouped_api.cu -- C ABI of the experts' operators (declared in
// include/moe.h): argument checks and launches.  No kernel code lives here.
#include <initializer_list>

#include "grouped.cuh"

using namespace moe;

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 30;
constexpr int kMaxDim = 1 << 20;
constexpr int kMaxDimI8 = 131056;      // 128 * 128 * kMaxDimI8 < 2^31: the int32 sums are exact
constexpr int64_t kMaxStride = int64_t(1) << 31;

inline bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool tensor_ok(const void* p) { return p && aligned(p, 16); }
inline bool is16(int dtype) { return dtype == MOE_DTYPE_BF16 || dtype == MOE_DTYPE_F16; }
inline bool stride_ok(int64_t stride, int64_t cols, int mult) {
    return stride >= cols && stride <= kMaxStride && stride % mult == 0;
}

// Every pointer is memory of the current device (or managed memory): work on
// another device's stream or a host pointer is refused here, before a launch.
moe_status_t on_device(std::initializer_list<const void*> ptrs) {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return MOE_ERR_CUDA;
    }
    for (const void* p : ptrs) {
        cudaPointerAttributes at{};
        if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
            cudaGetLastError();
            return MOE_ERR_CUDA;
        }
        if (at.type == cudaMemoryTypeManaged) continue;
        if (at.type != cudaMemoryTypeDevice || at.device != dev) return MOE_ERR_INVALID_ARG;
    }
    return MOE_OK;
}

moe_status_t check_grouped(const moe_grouped_t* g, bool i8, bool wgrad) {
    if (!g) return MOE_ERR_INVALID_ARG;
    if (g->rows < 0 || g->rows > kMaxRows || g->n_experts < 1 || g->n_experts > kMaxExperts)
        return MOE_ERR_INVALID_ARG;
    const int m_in = i8 ? 16 : 8;
    if (g->d_in < 1 || g->d_in % m_in || g->d_in > (i8 ? kMaxDimI8 : kMaxDim) || g->d_out < 1 ||
        g->d_out % 8 || g->d_out > kMaxDim)
        return MOE_ERR_INVALID_ARG;
    if (!stride_ok(g->x_stride, g->d_in, m_in) || !stride_ok(g->y_stride, g->d_out, 8))
        return MOE_ERR_INVALID_ARG;
    if (i8 ? g->dtype != MOE_DTYPE_I8 : !is16(g->dtype)) return MOE_ERR_INVALID_ARG;
    const bool out_ok = g->out_dtype == MOE_DTYPE_F32 || (i8 ? is16(g->out_dtype) : g->out_dtype == g->dtype);
    if (!out_ok) return MOE_ERR_INVALID_ARG;
    if (g->accumulate != 0 && !(wgrad && g->accumulate == 1 && g->out_dtype == MOE_DTYPE_F32))
        return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

GroupedCall call_of(const moe_grouped_t* g, const void* a, const void* w, void* out) {
    GroupedCall c{};
    c.rows = g->rows;
    c.E = g->n_experts;
    c.d_in = g->d_in;
    c.d_out = g->d_out;
    c.dtype = g->dtype;
    c.out_dtype = g->out_dtype;
    c.accumulate = g->accumulate;
    c.offsets = g->offsets;
    c.x_stride = g->x_stride;
    c.y_stride = g->y_stride;
    c.a = a;
    c.w = w;
    c.out = out;
    return c;
}

moe_status_t check_rows(int64_t rows, int32_t cols, int32_t dtype) {
    if (rows < 0 || rows > kMaxRows || cols < 1 || cols % 8 || cols > kMaxDim || !is16(dtype))
        return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

moe_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

}  // namespace

extern "C" {

moe_status_t moe_grouped_gemm(const moe_grouped_t* g, const void* x, const void* w, void* y, void* stream) {
    moe_status_t s = check_grouped(g, false, false);
    if (s) return s;
    if (g->rows == 0) return MOE_OK;
    if (!tensor_ok(x) || !tensor_ok(w) || !tensor_ok(y) || !g->offsets || !aligned(g->offsets, 4))
        return MOE_ERR_INVALID_ARG;
    s = on_device({x, w, y, g->offsets});
    if (s) return s;
    return launch_grouped(kOpGemm, call_of(g, x, w, y), static_cast<cudaStream_t>(stream));
}

moe_status_t moe_grouped_dgrad(const moe_grouped_t* g, const void* dy, const void* w, void* dx, void* stream) {
    moe_status_t s = check_grouped(g, false, false);
    if (s) return s;
    if (g->rows == 0) return MOE_OK;
    if (!tensor_ok(dy) || !tensor_ok(w) || !tensor_ok(dx) || !g->offsets || !aligned(g->offsets, 4))
        return MOE_ERR_INVALID_ARG;
    s = on_device({dy, w, dx, g->offsets});
    if (s) return s;
    return launch_grouped(kOpDgrad, call_of(g, dy, w, dx), static_cast<cudaStream_t>(stream));
}

moe_status_t moe_grouped_wgrad(const moe_grouped_t* g, const void* dy, const void* x, void* dw, void* stream) {
    moe_status_t s = check_grouped(g, false, true);
    if (s) return s;
    if (!tensor_ok(dw)) return MOE_ERR_INVALID_ARG;
    if (g->rows == 0) {
        s = on_device({dw});
    } else {
        if (!tensor_ok(dy) || !tensor_ok(x) || !g->offsets || !aligned(g->offsets, 4)) return MOE_ERR_INVALID_ARG;
        s = on_device({dy, x, dw, g->offsets});
    }
    if (s) return s;
    return launch_grouped(kOpWgrad, call_of(g, dy, x, dw), static_cast<cudaStream_t>(stream));
}

moe_status_t moe_i8_grouped_gemm(const moe_grouped_t* g, const void* xq, const float* x_scale, const void* wq,
                                 const float* w_scale, void* y, void* stream) {
    moe_status_t s = check_grouped(g, true, false);
    if (s) return s;
    if (g->rows == 0) return MOE_OK;
    if (!tensor_ok(xq) || !tensor_ok(wq) || !tensor_ok(y) || !g->offsets || !aligned(g->offsets, 4) ||
        !x_scale || !aligned(x_scale, 4) || !w_scale || !aligned(w_scale, 4))
        return MOE_ERR_INVALID_ARG;
    s = on_device({xq, x_scale, wq, w_scale, y, g->offsets});
    if (s) return s;
    GroupedCall c = call_of(g, xq, wq, y);
    c.a_scale = x_scale;
    c.w_scale = w_scale;
    return launch_grouped(kOpGemm, c, static_cast<cudaStream_t>(stream));
}

moe_status_t moe_grouped_status(void) { return grouped_status_read(); }

moe_status_t moe_i8_quantize(int64_t rows, int32_t cols, int32_t dtype, const void* x, int64_t x_stride, void* q,
                             int64_t q_stride, float* scale, void* stream) {
    moe_status_t s = check_rows(rows, cols, dtype);
    if (s) return s;
    if (!stride_ok(x_stride, cols, 8) || !stride_ok(q_stride, cols, 8)) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if (!tensor_ok(x) || !tensor_ok(q) || !scale || !aligned(scale, 4)) return MOE_ERR_INVALID_ARG;
    s = on_device({x, q, scale});
    if (s) return s;
    RowsCall c{};
    c.rows = rows;
    c.cols = cols;
    c.dtype = dtype;
    c.a = x;
    c.in_stride = x_stride;
    c.out = q;
    c.out_stride = q_stride;
    c.scale = scale;
    return cuda_status(launch_i8_rows(c, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_swiglu_i8(int64_t rows, int32_t cols, int32_t dtype, const void* gate, const void* up,
                           int64_t in_stride, void* q, int64_t q_stride, float* scale, void* stream) {
    moe_status_t s = check_rows(rows, cols, dtype);
    if (s) return s;
    if (!stride_ok(in_stride, cols, 8) || !stride_ok(q_stride, cols, 8)) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if (!tensor_ok(gate) || !tensor_ok(up) || !tensor_ok(q) || !scale || !aligned(scale, 4))
        return MOE_ERR_INVALID_ARG;
    s = on_device({gate, up, q, scale});
    if (s) return s;
    RowsCall c{};
    c.rows = rows;
    c.cols = cols;
    c.dtype = dtype;
    c.a = gate;
    c.b = up;
    c.in_stride = in_stride;
    c.out = q;
    c.out_stride = q_stride;
    c.scale = scale;
    return cuda_status(launch_i8_rows(c, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_swiglu(int64_t rows, int32_t cols, int32_t dtype, const void* gate, const void* up,
                        int64_t in_stride, void* h, int64_t h_stride, void* stream) {
    moe_status_t s = check_rows(rows, cols, dtype);
    if (s) return s;
    if (!stride_ok(in_stride, cols, 8) || !stride_ok(h_stride, cols, 8)) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if (!tensor_ok(gate) || !tensor_ok(up) || !tensor_ok(h)) return MOE_ERR_INVALID_ARG;
    s = on_device({gate, up, h});
    if (s) return s;
    RowsCall c{};
    c.rows = rows;
    c.cols = cols;
    c.dtype = dtype;
    c.a = gate;
    c.b = up;
    c.in_stride = in_stride;
    c.out = h;
    c.out_stride = h_stride;
    return cuda_status(launch_swiglu(c, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_swiglu_grad(int64_t rows, int32_t cols, int32_t dtype, const void* dh, int64_t dh_stride,
                             const void* gate, const void* up, int64_t in_stride, void* dgate, void* dup,
                             int64_t grad_stride, void* stream) {
    moe_status_t s = check_rows(rows, cols, dtype);
    if (s) return s;
    if (!stride_ok(in_stride, cols, 8) || !stride_ok(dh_stride, cols, 8) || !stride_ok(grad_stride, cols, 8))
        return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if (!tensor_ok(dh) || !tensor_ok(gate) || !tensor_ok(up) || !tensor_ok(dgate) || !tensor_ok(dup))
        return MOE_ERR_INVALID_ARG;
    s = on_device({dh, gate, up, dgate, dup});
    if (s) return s;
    RowsCall c{};
    c.rows = rows;
    c.cols = cols;
    c.dtype = dtype;
    c.a = gate;
    c.b = up;
    c.in_stride = in_stride;
    c.dh = dh;
    c.dh_stride = dh_stride;
    c.out = dgate;
    c.out2 = dup;
    c.out_stride = grad_stride;
    return cuda_status(launch_swiglu_grad(c, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
