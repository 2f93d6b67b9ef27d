// rows.cu -- the row operators around the experts' products: SwiGLU, its
// gradient, and the rounding of rows to 8-bit codes with a scale for each row.
//
// All are bound by the bytes they read and write.  Every thread moves 16-byte
// vectors (8 elements), computes in fp32 and rounds each result once.
#include "grouped.cuh"

namespace moe {
namespace {

constexpr int kRowThreads = 256;

template <bool F16>
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (F16) {
            const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            f[2 * i] = p.x;
            f[2 * i + 1] = p.y;
        } else {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
}
template <bool F16>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = F16 ? pack_f16x2(f[2 * i], f[2 * i + 1]) : pack_bf16x2(f[2 * i], f[2 * i + 1]);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// sigmoid: e^-g is +inf for g < -88.7, and 1 / (1 + inf) = 0, its limit
__device__ __forceinline__ float sigmoid_f(float g) { return 1.f / (1.f + expf(-g)); }

// h = g sig(g) u.  g = -inf gives -inf * 0 = NaN, as the formula does.
template <bool F16>
__global__ void __launch_bounds__(kRowThreads) swiglu_kernel(const RowsCall c) {
    const int vec = c.cols / 8;
    const int64_t n = c.rows * vec;
    const uint16_t* gate = static_cast<const uint16_t*>(c.a);
    const uint16_t* up = static_cast<const uint16_t*>(c.b);
    for (int64_t i = blockIdx.x * static_cast<int64_t>(kRowThreads) + threadIdx.x; i < n;
         i += static_cast<int64_t>(gridDim.x) * kRowThreads) {
        const int64_t r = i / vec;
        const int col = static_cast<int>(i - r * vec) * 8;
        float g[8], u[8];
        unpack8<F16>(*reinterpret_cast<const uint4*>(gate + r * c.in_stride + col), g);
        unpack8<F16>(*reinterpret_cast<const uint4*>(up + r * c.in_stride + col), u);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = g[j] * sigmoid_f(g[j]) * u[j];
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(c.out) + r * c.out_stride + col) = pack8<F16>(g);
    }
}

// dgate = dh u sig(g) (1 + g (1 - sig(g))),  dup = dh g sig(g)
template <bool F16>
__global__ void __launch_bounds__(kRowThreads) swiglu_grad_kernel(const RowsCall c) {
    const int vec = c.cols / 8;
    const int64_t n = c.rows * vec;
    const uint16_t* gate = static_cast<const uint16_t*>(c.a);
    const uint16_t* up = static_cast<const uint16_t*>(c.b);
    const uint16_t* dh = static_cast<const uint16_t*>(c.dh);
    for (int64_t i = blockIdx.x * static_cast<int64_t>(kRowThreads) + threadIdx.x; i < n;
         i += static_cast<int64_t>(gridDim.x) * kRowThreads) {
        const int64_t r = i / vec;
        const int col = static_cast<int>(i - r * vec) * 8;
        float g[8], u[8], d[8];
        unpack8<F16>(*reinterpret_cast<const uint4*>(gate + r * c.in_stride + col), g);
        unpack8<F16>(*reinterpret_cast<const uint4*>(up + r * c.in_stride + col), u);
        unpack8<F16>(*reinterpret_cast<const uint4*>(dh + r * c.dh_stride + col), d);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float s = sigmoid_f(g[j]);
            const float t = d[j] * s;
            const float dg = t * u[j] * (1.f + g[j] * (1.f - s));
            u[j] = t * g[j];
            g[j] = dg;
        }
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(c.out) + r * c.out_stride + col) = pack8<F16>(g);
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(c.out2) + r * c.out_stride + col) = pack8<F16>(u);
    }
}

// Codes of a row v (x itself, or SwiGLU of gate and up, in fp32): with
// a = max |v|, s = a / 127 and q = rint(v / s), both divisions rounded to
// nearest (the codes are then those of any fp32 evaluation of the formula).
// a = 0: s = 0 and codes 0.  A row with an infinity or a NaN: s = NaN, codes 0,
// so that the product shows it.  |v| is compared by its bits: a NaN is larger
// than an infinity, and an infinity than every number.
// TPR threads share a row, each keeping up to VPT vectors of it in registers
// between the two passes; what a longer row has beyond that is read again.
template <bool F16, bool GLU, int TPR, int VPT>
__global__ void __launch_bounds__(kRowThreads) i8_rows_kernel(const RowsCall c) {
    constexpr int kRows = kRowThreads / TPR;          // rows of a block
    __shared__ uint32_t s_max[kRowThreads / 32];
    const int vec = c.cols / 8;
    const int t = threadIdx.x % TPR;
    const int64_t r = blockIdx.x * static_cast<int64_t>(kRows) + threadIdx.x / TPR;
    const bool live = r < c.rows;
    const uint16_t* pa = static_cast<const uint16_t*>(c.a) + (live ? r : 0) * c.in_stride;
    const uint16_t* pb = GLU ? static_cast<const uint16_t*>(c.b) + (live ? r : 0) * c.in_stride : nullptr;

    auto value = [&](int j, float (&f)[8]) {
        unpack8<F16>(__ldg(reinterpret_cast<const uint4*>(pa + j * 8)), f);
        if constexpr (GLU) {
            float u[8];
            unpack8<F16>(__ldg(reinterpret_cast<const uint4*>(pb + j * 8)), u);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = f[i] * sigmoid_f(f[i]) * u[i];
        }
    };
    uint32_t m = 0;
    auto widen = [&](const float (&f)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7FFFFFFFu);
    };
    float keep[VPT][8];
    if (live) {
#pragma unroll
        for (int v = 0; v < VPT; ++v)
            if (t + v * TPR < vec) { value(t + v * TPR, keep[v]); widen(keep[v]); }
        for (int j = t + VPT * TPR; j < vec; j += TPR) {
            float f[8];
            value(j, f);
            widen(f);
        }
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if constexpr (TPR > 32) {
        if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
        __syncthreads();
        m = 0;
#pragma unroll
        for (int w = 0; w < TPR / 32; ++w) m = max(m, s_max[(threadIdx.x / TPR) * (TPR / 32) + w]);
    }
    if (!live) return;
    const bool finite = m < 0x7F800000u;
    const float s = finite ? __fdiv_rn(__uint_as_float(m), 127.f) : __uint_as_float(0x7FC00000u);
    if (t == 0) c.scale[r] = s;
    int8_t* q = static_cast<int8_t*>(c.out) + r * c.out_stride;
    auto store = [&](int j, const float (&f)[8]) {
        uint32_t w[2] = {0u, 0u};
        if (finite && s > 0.f) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int code = max(-127, min(127, __float2int_rn(__fdiv_rn(f[i], s))));
                w[i >> 2] |= (static_cast<uint32_t>(code) & 0xFFu) << (8 * (i & 3));
            }
        }
        *reinterpret_cast<uint2*>(q + j * 8) = make_uint2(w[0], w[1]);
    };
#pragma unroll
    for (int v = 0; v < VPT; ++v)
        if (t + v * TPR < vec) store(t + v * TPR, keep[v]);
    for (int j = t + VPT * TPR; j < vec; j += TPR) {
        float f[8];
        value(j, f);
        store(j, f);
    }
}

template <bool F16, bool GLU>
cudaError_t i8_rows(const RowsCall& c, cudaStream_t stream) {
    // a warp for a row of up to 1024 elements; a block for longer ones
    if (c.cols <= 1024) {
        const int64_t blocks = (c.rows + 7) / 8;
        i8_rows_kernel<F16, GLU, 32, 4><<<static_cast<unsigned>(blocks), kRowThreads, 0, stream>>>(c);
    } else {
        i8_rows_kernel<F16, GLU, 256, 4><<<static_cast<unsigned>(c.rows), kRowThreads, 0, stream>>>(c);
    }
    return cudaGetLastError();
}

unsigned flat_blocks(const RowsCall& c) {
    const int64_t n = (c.rows * (c.cols / 8) + kRowThreads - 1) / kRowThreads;
    return static_cast<unsigned>(n < 148 * 64 ? n : 148 * 64);
}

}  // namespace

cudaError_t launch_swiglu(const RowsCall& c, cudaStream_t stream) {
    if (c.dtype == MOE_DTYPE_F16) swiglu_kernel<true><<<flat_blocks(c), kRowThreads, 0, stream>>>(c);
    else swiglu_kernel<false><<<flat_blocks(c), kRowThreads, 0, stream>>>(c);
    return cudaGetLastError();
}

cudaError_t launch_swiglu_grad(const RowsCall& c, cudaStream_t stream) {
    if (c.dtype == MOE_DTYPE_F16) swiglu_grad_kernel<true><<<flat_blocks(c), kRowThreads, 0, stream>>>(c);
    else swiglu_grad_kernel<false><<<flat_blocks(c), kRowThreads, 0, stream>>>(c);
    return cudaGetLastError();
}

cudaError_t launch_i8_rows(const RowsCall& c, cudaStream_t stream) {
    if (c.b) return c.dtype == MOE_DTYPE_F16 ? i8_rows<true, true>(c, stream) : i8_rows<false, true>(c, stream);
    return c.dtype == MOE_DTYPE_F16 ? i8_rows<true, false>(c, stream) : i8_rows<false, false>(c, stream);
}

}  // namespace moe
