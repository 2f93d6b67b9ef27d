// rows.cu -- the row operators around the experts' products: SwiGLU, its
// gradient, and the rounding of rows to 8-bit codes with a scale for each row.
//
// All are bound by the bytes they read and write, if the arithmetic stays
// small beside them: every thread moves 16-byte vectors (8 elements), computes
// in fp32 and rounds each result once.
#include "grouped.cuh"

namespace moe {
namespace {

constexpr int kRowThreads = 256;

template <bool F16>
__device__ __forceinline__ void unpack2(uint32_t w, float (&f)[2]) {
    if (F16) {
        const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w));
        f[0] = p.x;
        f[1] = p.y;
    } else {
        f[0] = __uint_as_float(w << 16);
        f[1] = __uint_as_float(w & 0xFFFF0000u);
    }
}
template <bool F16>
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) unpack2<F16>(w[i], reinterpret_cast<float (&)[2]>(f[2 * i]));
}
template <bool F16>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = F16 ? pack_f16x2(f[2 * i], f[2 * i + 1]) : pack_bf16x2(f[2 * i], f[2 * i + 1]);
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 load16(const uint16_t* p) { return *reinterpret_cast<const uint4*>(p); }

// sigmoid(g) = 1 / (1 + 2^t), t = -g log2(e).  t is formed in two parts, since
// the rounding of t alone would cost |g| half steps of the result: 2^t =
// 2^hi (1 + lo ln 2).  Errors in units of 2^-24: 2^hi 4 (ex2.approx), 1 + lo
// ln 2 and the product 1 each, 1 + 2^t 1, the reciprocal 2: at most 9.  Below
// g = -87.3 the result is under 2^-126 and comes out as 0 (sigmoid_tail has those).
// At an infinity lo is NaN: fminf drops it (the factor is never above 1.0001
// otherwise).
__device__ __forceinline__ float sigmoid_f(float g) {
    constexpr float kL = -1.44269504f, kLlo = -1.92596299e-8f, kLn2 = 0.693147181f;
    const float hi = g * kL;
    const float lo = fmaf(g, kLlo, fmaf(g, kL, -hi));
    float p, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p) : "f"(hi));
    p *= fminf(fmaf(lo, kLn2, 1.f), 1.0001f);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + p));
    return r;
}

// (g + plus) sig(g) b for gates whose sigmoid is below the smallest normal number
// while its product with g and b need not be: there sig(g) = e^g = q 2^-n with q near
// 1, and the powers of two are multiplied in behind g and b, a normal number at a
// time.  Gates of -300 and below give 0 with every finite b (e^-300 < 2^-432).
constexpr float kTail = -87.f, kTailEnd = -300.f;
__device__ __forceinline__ bool in_tail(float g) { return g < kTail && g > kTailEnd; }
__device__ __forceinline__ float sigmoid_tail(float g, float plus, float b) {
    constexpr float kL = -1.44269504f, kLlo = -1.92596299e-8f, kLn2 = 0.693147181f;
    const float hi = g * kL;
    const float lo = fmaf(g, kLlo, fmaf(g, kL, -hi));
    const float whole = rintf(hi);
    float q;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(q) : "f"(whole - hi));
    q *= fmaf(lo, -kLn2, 1.f);
    int n = static_cast<int>(whole);
    float v = (g + plus) * q;
#pragma unroll
    for (int i = 0; i < 4; ++i) {                      // n <= 433
        const int k = min(n, 126);
        v *= __int_as_float((127 - k) << 23);
        if (i == 0) v *= b;
        n -= k;
    }
    return v;
}
// Whether one of 8 gates is below kTail, by the maximum of their bits: negative
// 16-bit numbers order by them, above the positive ones (a negative NaN passes, too).
template <bool F16>
__device__ __forceinline__ bool any_tail(const uint4& v) {
    const uint32_t m = __vmaxu2(__vmaxu2(v.x, v.y), __vmaxu2(v.z, v.w));
    return max(m & 0xFFFFu, m >> 16) > (F16 ? 0xD570u : 0xC2AEu);
}
// The words of a vector move up one place.
__device__ __forceinline__ void turn(uint4& v, uint32_t last) { v = make_uint4(v.y, v.z, v.w, last); }

// f = g sig(g) u of 8 values.  A vector with a gate in the tail is rare and takes a
// loop over its words, which keeps the kernels' registers as they are without it
// (a branch behind the common path took 40 instead of 32 in SwiGLU, 58 in its
// gradient).  The look at the gates costs nothing measurable there (24576 x 1408
// bf16: 31.0 us, gradient 52.0) and 2.3 us of 42 where codes follow; one look for
// all of a thread's vectors, with a second pass, cost 9.5.
template <bool F16>
__device__ __forceinline__ void glu8(uint4 gate, uint4 up, float (&f)[8]) {
    if (any_tail<F16>(gate)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = 0.f;
#pragma unroll 1
        for (int w = 0; w < 4; ++w) {
            float g[2], u[2];
            unpack2<F16>(gate.x, g);
            unpack2<F16>(up.x, u);
#pragma unroll
            for (int i = 0; i < 6; ++i) f[i] = f[i + 2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                f[6 + i] = in_tail(g[i]) ? sigmoid_tail(g[i], 0.f, u[i]) : g[i] * sigmoid_f(g[i]) * u[i];
            turn(gate, 0);
            turn(up, 0);
        }
        return;
    }
    float u[8];
    unpack8<F16>(gate, f);
    unpack8<F16>(up, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = f[i] * sigmoid_f(f[i]) * u[i];
}

// Vector i of `n` as a row and a first column, for fewer than 2^31 vectors:
// i / vec by a multiplication (d = vec: mul = floor(2^32 (2^s - d) / d) + 1,
// s = ceil(log2 d); the quotient is then (umulhi(mul, i) + i) >> s).
struct FastDiv {
    uint32_t d, mul, s;
    explicit FastDiv(uint32_t v) : d(v), s(0) {
        while ((uint64_t(1) << s) < d) ++s;
        mul = static_cast<uint32_t>((((uint64_t(1) << s) - d) << 32) / d + 1);
    }
};
template <bool BIG>
__device__ __forceinline__ void place(int64_t i, const FastDiv& f, int64_t& r, int& col) {
    if (BIG) {
        r = i / f.d;
        col = static_cast<int>(i - r * f.d) * 8;
    } else {
        const uint32_t k = static_cast<uint32_t>(i);
        const uint32_t q = (__umulhi(f.mul, k) + k) >> f.s;
        r = q;
        col = static_cast<int>(k - q * f.d) * 8;
    }
}

// h = g sig(g) u.  g = -inf gives -inf * 0 = NaN, as the formula does.
template <bool F16, bool BIG>
__global__ void __launch_bounds__(kRowThreads) swiglu_kernel(const RowsCall c, const FastDiv f) {
    const int64_t n = c.rows * f.d;
    const uint16_t* gate = static_cast<const uint16_t*>(c.a);
    const uint16_t* up = static_cast<const uint16_t*>(c.b);
    grid_let_next();
    grid_wait();
    for (int64_t i = blockIdx.x * static_cast<int64_t>(kRowThreads) + threadIdx.x; i < n;
         i += static_cast<int64_t>(gridDim.x) * kRowThreads) {
        int64_t r;
        int col;
        place<BIG>(i, f, r, col);
        const uint4 vg = load16(gate + r * c.in_stride + col), vu = load16(up + r * c.in_stride + col);
        float h[8];
        glu8<F16>(vg, vu, h);
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(c.out) + r * c.out_stride + col) = pack8<F16>(h);
    }
}

// dgate = dh u sig(g) (1 + g (1 - sig(g))),  dup = dh g sig(g), in the place of g and u
template <bool TAIL>
__device__ __forceinline__ void grad_of(float& g, float& u, float d) {
    if (TAIL && in_tail(g)) {                          // 1 - sig(g) is 1
        const float dg = sigmoid_tail(g, 1.f, d * u);
        u = sigmoid_tail(g, 0.f, d);
        g = dg;
        return;
    }
    const float s = sigmoid_f(g);
    const float t = d * s;
    const float dg = t * u * (1.f + g * (1.f - s));
    u = t * g;
    g = dg;
}
template <bool F16, bool BIG>
__global__ void __launch_bounds__(kRowThreads) swiglu_grad_kernel(const RowsCall c, const FastDiv f) {
    const int64_t n = c.rows * f.d;
    const uint16_t* gate = static_cast<const uint16_t*>(c.a);
    const uint16_t* up = static_cast<const uint16_t*>(c.b);
    const uint16_t* dh = static_cast<const uint16_t*>(c.dh);
    grid_let_next();
    grid_wait();
    for (int64_t i = blockIdx.x * static_cast<int64_t>(kRowThreads) + threadIdx.x; i < n;
         i += static_cast<int64_t>(gridDim.x) * kRowThreads) {
        int64_t r;
        int col;
        place<BIG>(i, f, r, col);
        const uint4 vg = load16(gate + r * c.in_stride + col), vu = load16(up + r * c.in_stride + col);
        const uint4 vd = load16(dh + r * c.dh_stride + col);
        uint16_t* dg = static_cast<uint16_t*>(c.out) + r * c.out_stride + col;
        uint16_t* du = static_cast<uint16_t*>(c.out2) + r * c.out_stride + col;
        if (any_tail<F16>(vg)) {                       // as in glu8
            uint4 wg = vg, wu = vu, wd = vd;
#pragma unroll 1
            for (int w = 0; w < 4; ++w) {
                float g[2], u[2], d[2];
                unpack2<F16>(wg.x, g);
                unpack2<F16>(wu.x, u);
                unpack2<F16>(wd.x, d);
#pragma unroll
                for (int i = 0; i < 2; ++i) grad_of<true>(g[i], u[i], d[i]);
                turn(wg, F16 ? pack_f16x2(g[0], g[1]) : pack_bf16x2(g[0], g[1]));
                turn(wu, F16 ? pack_f16x2(u[0], u[1]) : pack_bf16x2(u[0], u[1]));
                turn(wd, 0);
            }
            *reinterpret_cast<uint4*>(dg) = wg;
            *reinterpret_cast<uint4*>(du) = wu;
            continue;
        }
        float g[8], u[8], d[8];
        unpack8<F16>(vg, g);
        unpack8<F16>(vu, u);
        unpack8<F16>(vd, d);
#pragma unroll
        for (int j = 0; j < 8; ++j) grad_of<false>(g[j], u[j], d[j]);
        *reinterpret_cast<uint4*>(dg) = pack8<F16>(g);
        *reinterpret_cast<uint4*>(du) = pack8<F16>(u);
    }
}

// Codes of 8 values v: q = rint(v / s), the quotient rounded to nearest first.
// v * (1 / s) is within 127 * 3 * 2^-24 < 2.3e-5 of that quotient (the sum and
// the difference below are rounded once each), so it rounds to the same integer
// unless it lies within 3e-5 of a half; only for such a value is the division
// done.  Adding 1.5 * 2^23 rounds to the nearest integer, ties to even, and
// leaves it in the low byte.
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float s, float inv) {
    constexpr float kMagic = 12582912.f, kNear = 0.49997f;
    uint32_t b[8];
    float off = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float t = fmaf(v[i], inv, kMagic);
        off = fmaxf(off, fabsf(fmaf(v[i], inv, kMagic - t)));
        b[i] = __float_as_uint(t);
    }
    if (off > kNear) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (fabsf(fmaf(v[i], inv, kMagic - __uint_as_float(b[i]))) > kNear)
                b[i] = __float_as_uint(__fdiv_rn(v[i], s) + kMagic);
    }
    return make_uint2(__byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410),
                      __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410));
}

// Codes of a row v (x itself, or SwiGLU of gate and up, in fp32): with
// a = max |v|, s = a / 127 and q = rint(v / s), both divisions rounded to
// nearest (the codes are then those of any fp32 evaluation of the formula).
// a = 0: s = 0 and codes 0.  A row with an infinity or a NaN: s = NaN, codes 0,
// so that the product shows it.  |v| is compared by its bits: a NaN is larger
// than an infinity, and an infinity than every number.
// TPR threads share a row, each keeping up to VPT vectors of it in registers
// between the two passes (as they were loaded; SwiGLU's as computed); what a
// longer row has beyond that is read again.
template <bool F16, bool GLU, int TPR, int VPT>
__global__ void __launch_bounds__(kRowThreads, GLU ? 4 : 5) i8_rows_kernel(const RowsCall c) {
    constexpr int kRows = kRowThreads / TPR;          // rows of a block
    __shared__ uint32_t s_max[kRowThreads / 32];
    grid_let_next();
    grid_wait();
    const int vec = c.cols / 8;
    const int t = threadIdx.x % TPR;
    const int64_t r = blockIdx.x * static_cast<int64_t>(kRows) + threadIdx.x / TPR;
    const bool live = r < c.rows;
    const uint16_t* pa = static_cast<const uint16_t*>(c.a) + (live ? r : 0) * c.in_stride;
    const uint16_t* pb = GLU ? static_cast<const uint16_t*>(c.b) + (live ? r : 0) * c.in_stride : nullptr;

    // |v| of 16-bit values order by their bits, two to an instruction
    uint32_t m = 0, m2 = 0;
    auto widen16 = [&](const uint4& v) {
        m2 = __vmaxu2(m2, v.x & 0x7FFF7FFFu);
        m2 = __vmaxu2(m2, v.y & 0x7FFF7FFFu);
        m2 = __vmaxu2(m2, v.z & 0x7FFF7FFFu);
        m2 = __vmaxu2(m2, v.w & 0x7FFF7FFFu);
    };
    auto widen = [&](const float (&f)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7FFFFFFFu);
    };
    uint4 raw[VPT], raw_b[GLU ? VPT : 1];
    float val[GLU ? VPT : 1][8];
    if (live) {
#pragma unroll
        for (int v = 0; v < VPT; ++v)
            if (t + v * TPR < vec) {
                raw[v] = load16(pa + (t + v * TPR) * 8);
                if constexpr (GLU) raw_b[v] = load16(pb + (t + v * TPR) * 8);
            }
#pragma unroll
        for (int v = 0; v < VPT; ++v)
            if (t + v * TPR < vec) {
                if constexpr (GLU) {
                    glu8<F16>(raw[v], raw_b[v], val[v]);
                    widen(val[v]);
                } else {
                    widen16(raw[v]);
                }
            }
        for (int j = t + VPT * TPR; j < vec; j += TPR) {
            if constexpr (GLU) {
                float f[8];
                glu8<F16>(load16(pa + j * 8), load16(pb + j * 8), f);
                widen(f);
            } else {
                widen16(load16(pa + j * 8));
            }
        }
        if constexpr (!GLU) {
            const unsigned short top = static_cast<unsigned short>(max(m2 & 0xFFFFu, m2 >> 16));
            m = F16 ? __float_as_uint(__half2float(__ushort_as_half(top))) : static_cast<uint32_t>(top) << 16;
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
    // a scale below 2^-100 (its reciprocal and its own rounding are no longer
    // good for the bound above) takes the division for every value
    const bool fast = s > 7.8886091e-31f;
    const float inv = fast ? __fdiv_rn(1.f, s) : 0.f;
    auto store = [&](int j, const float (&f)[8]) {
        uint2 w = make_uint2(0u, 0u);
        if (fast) {
            w = codes8(f, s, inv);
        } else if (finite && s > 0.f) {
            uint32_t b[2] = {0u, 0u};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int code = max(-127, min(127, __float2int_rn(__fdiv_rn(f[i], s))));
                b[i >> 2] |= (static_cast<uint32_t>(code) & 0xFFu) << (8 * (i & 3));
            }
            w = make_uint2(b[0], b[1]);
        }
        *reinterpret_cast<uint2*>(q + j * 8) = w;
    };
#pragma unroll
    for (int v = 0; v < VPT; ++v)
        if (t + v * TPR < vec) {
            if constexpr (GLU) {
                store(t + v * TPR, val[v]);
            } else {
                float f[8];
                unpack8<F16>(raw[v], f);
                store(t + v * TPR, f);
            }
        }
    for (int j = t + VPT * TPR; j < vec; j += TPR) {
        float f[8];
        if constexpr (GLU) glu8<F16>(load16(pa + j * 8), load16(pb + j * 8), f);
        else unpack8<F16>(load16(pa + j * 8), f);
        store(j, f);
    }
}

template <bool F16, bool GLU, int TPR, int VPT>
cudaError_t i8_rows_launch(const RowsCall& c, cudaStream_t stream) {
    const int64_t blocks = (c.rows + kRowThreads / TPR - 1) / (kRowThreads / TPR);
    return launch_chained(i8_rows_kernel<F16, GLU, TPR, VPT>, dim3(static_cast<unsigned>(blocks)), kRowThreads, 0, 1,
                          stream, c);
}

template <bool F16, bool GLU>
cudaError_t i8_rows(const RowsCall& c, cudaStream_t stream) {
    // as few threads to a row as hold it with four vectors each, but no fewer
    // than give the device a block for each SM
    int tpr = 32;
    while (tpr < 256 && (c.cols > tpr * 32 || c.rows * tpr < 148 * kRowThreads)) tpr *= 2;
    switch (tpr) {
        case 32: return i8_rows_launch<F16, GLU, 32, 4>(c, stream);
        case 64: return i8_rows_launch<F16, GLU, 64, 4>(c, stream);
        case 128: return i8_rows_launch<F16, GLU, 128, 4>(c, stream);
        default: return i8_rows_launch<F16, GLU, 256, 4>(c, stream);
    }
}

template <typename K>
cudaError_t flat(K small, K big, const RowsCall& c, cudaStream_t stream) {
    const int64_t n = c.rows * (c.cols / 8);
    const int64_t blocks = (n + kRowThreads - 1) / kRowThreads;
    const unsigned grid = static_cast<unsigned>(blocks < 148 * 64 ? blocks : 148 * 64);
    return launch_chained(n < (int64_t(1) << 31) ? small : big, dim3(grid), kRowThreads, 0, 1, stream, c, FastDiv(c.cols / 8));
}

}  // namespace

cudaError_t launch_swiglu(const RowsCall& c, cudaStream_t stream) {
    return c.dtype == MOE_DTYPE_F16 ? flat(swiglu_kernel<true, false>, swiglu_kernel<true, true>, c, stream)
                                    : flat(swiglu_kernel<false, false>, swiglu_kernel<false, true>, c, stream);
}

cudaError_t launch_swiglu_grad(const RowsCall& c, cudaStream_t stream) {
    return c.dtype == MOE_DTYPE_F16
               ? flat(swiglu_grad_kernel<true, false>, swiglu_grad_kernel<true, true>, c, stream)
               : flat(swiglu_grad_kernel<false, false>, swiglu_grad_kernel<false, true>, c, stream);
}

cudaError_t launch_i8_rows(const RowsCall& c, cudaStream_t stream) {
    if (c.b) return c.dtype == MOE_DTYPE_F16 ? i8_rows<true, true>(c, stream) : i8_rows<false, true>(c, stream);
    return c.dtype == MOE_DTYPE_F16 ? i8_rows<true, false>(c, stream) : i8_rows<false, false>(c, stream);
}

}  // namespace moe
