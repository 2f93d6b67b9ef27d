// grouped_small.cuh -- the grouped product for few rows (single tokens and small
// decode batches), included by grouped.cu.
//
// The work is the weights' bytes: every active expert's matrix once.  A block
// takes 16 output features of one expert at a time, so that even one token's
// eight experts give some hundred pieces, evenly dealt; its eight warps split the
// reduction and stream their shares of the 16 weight rows straight into
// registers, 16 bytes a lane, eight such loads ahead of the ones being multiplied
// and across the pieces' ends.  The products run on mma.sync with the weights as
// the 16-row side and up to 8 of the expert's rows as the other; which k a
// fragment's slots stand for does not matter as long as both sides agree, so a
// lane's 16 consecutive bytes feed two MMAs as they are, and nothing passes
// through shared memory but the eight warps' partial sums (added in order; two
// sets of them, so that a piece costs one barrier).  Over a long reduction a warp
// adds its accumulators to its partial sum, in fp32 rounded to nearest, after each
// segment (of 64 terms a step in each accumulator, as long as a tile's) and starts
// them anew: they lose some of the sum with every MMA, always towards zero (65536
// terms in one sum: 1.1e-5 of the result in bf16, 2.4e-5 in fp16).
//
// Two blocks an SM keep 64 KB of weights in flight (128 bytes a thread): 8 rows
// through 8 experts of 14336 x 2560 take 110 us, 5.3 TB/s; one row through 4096 x 4096
// 10.5 us from HBM, of which the bytes need 5.2.  Loading x ahead as well cost more in
// registers than it hid (16 rows through 8 experts of 14336 x 4096 142 us, 135 without).
#pragma once

constexpr int kSmallThreads = 256;
constexpr int kSmallWarps = kSmallThreads / 32;
constexpr int kSmallRows = 16;                  // weight rows of a block
constexpr int kSmallTok = 8;                    // rows of x at a time
constexpr int kSmallStep = 256;                 // bytes of k that a warp takes at a time

struct SmallArgs {
    const int32_t* offsets;
    const uint8_t* x;
    const uint8_t* w;
    void* out;
    const float* a_scale;
    const float* w_scale;
    int64_t x_bytes;                            // row pitch of x
    int64_t out_stride;
    int64_t rows;
    int E, M, k_bytes;                          // M: output features
    int f16, out_dtype;
    int segment;                                // steps of a segment
};

template <bool I8>
__device__ __forceinline__ void small_mma(uint32_t (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1, bool f16) {
    if constexpr (I8) {
        asm volatile(
            "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    } else {
        float (&f)[4] = reinterpret_cast<float (&)[4]>(c);
        if (f16) mma_f16_16816_acc(f, a0, a1, a2, a3, b0, b1);
        else mma_bf16_16816(f, a0, a1, a2, a3, b0, b1);
    }
}

// 16 bytes by an ordinary load.  x and the weights may be what the kernel before
// this one wrote while this one was already resident (programmatic dependent
// launch), so they are not read-only for as long as this kernel lives and the
// non-coherent path (__ldg, ld.global.nc) is not open to them.
__device__ __forceinline__ uint4 small_load(const uint8_t* p) { return *reinterpret_cast<const uint4*>(p); }

// The piece of work a block is at: 16 output features of an expert and up to 8
// of its rows.
struct SmallUnit {
    int e, f0, tok, hi;
};

template <bool I8>
__global__ void __launch_bounds__(kSmallThreads, 2) grouped_small_kernel(const SmallArgs a) {
    __shared__ uint32_t parts[2][kSmallWarps][kSmallTok][kSmallRows];     // two: one barrier a unit
    __shared__ uint32_t s_has[32];                     // a bit for each expert that has rows
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    bool bad = false;
    grid_let_next();
    grid_wait();
    for (int e0 = warp * 32; e0 < 1024; e0 += kSmallThreads) {
        const int i = e0 + lane;
        const int v = i < a.E ? a.offsets[i] : 0, next = i < a.E ? a.offsets[i + 1] : 0;
        bad |= v < 0 || v > a.rows || next > a.rows || next < v;
        const uint32_t has = __ballot_sync(0xffffffffu, next > v);
        if (lane == 0) s_has[e0 / 32] = has;
    }
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) atomicOr(&g_grouped_err, kErrBadId);
        return;
    }
    const uint32_t has = s_has[lane];
    int before = __popc(has);                          // experts with rows in the words before lane's
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, before, d);
        if (lane >= d) before += o;
    }
    const int tiles = (a.M + kSmallRows - 1) / kSmallRows;
    const int64_t total = static_cast<int64_t>(__shfl_sync(0xffffffffu, before, 31)) * tiles;
    before -= __popc(has);
    int64_t unit = blockIdx.x;
    auto locate = [&](SmallUnit& n) {                  // unit's expert: the unit / tiles-th that has rows
        const int want = static_cast<int>(unit / tiles);
        const int word = 31 - __clz(__ballot_sync(0xffffffffu, before <= want));
        const uint32_t m = __shfl_sync(0xffffffffu, has, word);
        n.e = word * 32 + __fns(m, 0, want - __shfl_sync(0xffffffffu, before, word) + 1);
        n.f0 = static_cast<int>(unit - static_cast<int64_t>(want) * tiles) * kSmallRows;
        // read again: clamped, should the table change under the call
        n.tok = max(0, a.offsets[n.e]);
        n.hi = static_cast<int>(min(static_cast<int64_t>(a.offsets[n.e + 1]), a.rows));
    };
    auto advance = [&](SmallUnit& n) {                 // the next rows, or the next unit
        if (n.tok + kSmallTok < n.hi) {
            n.tok += kSmallTok;
            return true;
        }
        unit += gridDim.x;
        if (unit >= total) return false;
        locate(n);
        return true;
    };
    if (unit >= total) return;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    uint4 al[4], ah[4];
    auto fetch = [&](const SmallUnit& n, int k0) {
        const uint8_t* w = a.w + (static_cast<int64_t>(n.e) * a.M + n.f0 + g) * a.k_bytes;
        const bool ok_lo = n.f0 + g < a.M, ok_hi = n.f0 + 8 + g < a.M;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int k = k0 + u * 64 + t * 16;
            const bool in = k < a.k_bytes;
            al[u] = in && ok_lo ? small_load(w + k) : zero;
            ah[u] = in && ok_hi ? small_load(w + 8 * static_cast<int64_t>(a.k_bytes) + k) : zero;
        }
    };
    SmallUnit cur, next;
    locate(cur);
    const int k_first = warp * kSmallStep;
    fetch(cur, k_first);
    int turn = 0;
    for (bool more = true; more; cur = next, turn ^= 1) {
        uint32_t (&part)[kSmallWarps][kSmallTok][kSmallRows] = parts[turn];
        next = cur;
        more = advance(next);
        const uint8_t* x = a.x + (static_cast<int64_t>(cur.tok) + g) * a.x_bytes;
        const bool ok_x = cur.tok + g < cur.hi;
        uint32_t c[4] = {0, 0, 0, 0}, d[4] = {0, 0, 0, 0};    // two sums: half as many cuts to fp32 in each
        int k0 = k_first;
        bool begun = false;                            // the partial sum holds something
        auto fold = [&] {                              // every thread its own four words
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t& p = part[warp][2 * t + (i & 1)][g + 8 * (i >> 1)];
                if constexpr (I8) {
                    p = c[i] + d[i];
                } else {
                    const float sum = __uint_as_float(c[i]) + __uint_as_float(d[i]);
                    p = __float_as_uint(begun ? __uint_as_float(p) + sum : sum);
                }
                c[i] = d[i] = 0;
            }
            begun = true;
        };
        int left = a.segment;
        do {                                           // the loads of the next step, or unit, go ahead of the MMAs
            uint4 cl[4], ch[4], cb[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {                // x is few rows that the caches hold: no loads ahead
                const int k = k0 + u * 64 + t * 16;
                cl[u] = al[u];
                ch[u] = ah[u];
                cb[u] = k < a.k_bytes && ok_x ? small_load(x + k) : zero;
            }
            k0 += kSmallWarps * kSmallStep;
            if (k0 < a.k_bytes) fetch(cur, k0);
            else if (more) fetch(next, k_first);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                small_mma<I8>(c, cl[u].x, ch[u].x, cl[u].y, ch[u].y, cb[u].x, cb[u].y, a.f16);
                small_mma<I8>(d, cl[u].z, ch[u].z, cl[u].w, ch[u].w, cb[u].z, cb[u].w, a.f16);
            }
            if (!I8 && --left == 0 && k0 < a.k_bytes) {
                fold();
                left = a.segment;
            }
        } while (k0 < a.k_bytes);
        fold();
        __syncthreads();
        const int col = threadIdx.x / kSmallRows, f = cur.f0 + threadIdx.x % kSmallRows;
        if (col < kSmallTok && cur.tok + col < cur.hi && f < a.M) {
            float y;
            if constexpr (I8) {
                int sum = 0;
#pragma unroll
                for (int w = 0; w < kSmallWarps; ++w) sum += static_cast<int>(part[w][col][f - cur.f0]);
                y = static_cast<float>(sum) * a.a_scale[cur.tok + col] *
                    a.w_scale[static_cast<int64_t>(cur.e) * a.M + f];
            } else {
                y = 0.f;
#pragma unroll
                for (int w = 0; w < kSmallWarps; ++w) y += __uint_as_float(part[w][col][f - cur.f0]);
            }
            const int64_t at = (static_cast<int64_t>(cur.tok) + col) * a.out_stride + f;
            if (a.out_dtype == MOE_DTYPE_F32) static_cast<float*>(a.out)[at] = y;
            else if (a.out_dtype == MOE_DTYPE_F16) static_cast<__half*>(a.out)[at] = __float2half_rn(y);
            else static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(y);
        }
    }
}
