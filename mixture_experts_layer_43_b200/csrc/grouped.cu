// grouped.cu -- matrix products grouped by expert on the tcgen05 tensor cores.
//
// Rows o_e .. o_{e+1} - 1 of the row-major sides belong to expert e, whose
// weights are W[e] [d_out][d_in].  Three products and one in 8 bits:
//   gemm   y[r][n]  = sum_k x[r][k] W[e][n][k]
//   dgrad  dx[r][k] = sum_n dy[r][n] W[e][n][k]
//   wgrad  dW[e][n][k] = sum over e's rows of dy[r][n] x[r][k]
//   gemm of 8-bit codes: the sum in int32, times a scale for each row and one
//   for each output channel
//
// Tiles.  A CTA pair (tcgen05.mma.cta_group::2) computes a 256 x <= 256 tile.
// In gemm and dgrad the weights are the 256-row M side and the expert's rows
// the N side: N of an MMA is a run-time field of its instruction descriptor,
// so a ragged segment costs its rows rounded up to 32, not to a 128- or
// 256-row tile.  An expert's rows are split evenly into ceil(n / 256) chunks.
// Rows of a neighbouring expert that a chunk's loads touch only reach MMA
// columns that are not stored.  In wgrad M and N are d_in and d_out (both
// operands are "MN-major": the reduction runs over the rows of shared memory)
// and the rows are the reduction; the rows past the segment's end in its last
// step are overwritten with zeros in shared memory before the MMA reads them,
// since they hold another expert's values (and 0 * NaN would not vanish).
//
// Roles of a CTA: warp 0 loads by TMA into a ring of six 32 KB stages, warp 1
// of the pair's first CTA issues the MMAs, eight warps drain the accumulator
// (two of 256 TMEM columns each, so that they overlap the next tile's MMAs) and
// store it, lanes along the contiguous dimension; wgrad has one more warp that
// zeroes the rows of the last step.
//
// What bounds it.  A stage costs 512 cycles of MMA at 256 columns and takes 32 KB
// into each SM's shared memory, near what an SM can fill (64 B a cycle), so loads
// and MMAs have to overlap without a gap: both warps run their loops converged,
// with one elected lane issuing (a loop run by a single lane took 250 cycles for
// an MMA of any width, the descriptors' moves between register files standing in
// its way; now 138 K cycles for 131 K of MMA in a product of one expert).  On a
// DeepSeek-shaped prompt (24576 rows, 64 experts of 2048 x 2816, Zipf loads) the
// tensor pipe is active in 65% of the cycles and DRAM moves the algorithm's bytes
// once (977 MB): 250 us in a short run, and as long with equal loads.  Over seconds
// the power cap lowers the clock to 1.27 GHz (of 1.965) and the time is 289 us, 980
// TFLOP/s, where a dense product of large matrices keeps 1390 under the same cap.
#include <atomic>
#include <cmath>

#include <cudaTypedefs.h>
#include <string.h>

#include "grouped.cuh"
#include "umma_pair.cuh"

namespace moe {

static __device__ uint32_t g_grouped_err;

namespace {

#include "grouped_small.cuh"

constexpr int kMaxDevices = 64;
constexpr int kTile = 256;                        // tile rows (M), and the most columns (N)
constexpr int kHalf = 128;                        // rows of the tile one CTA holds
constexpr int kKBytes = 128;                      // k-step: 64 16-bit or 128 8-bit elements
constexpr int kStageHalf = kHalf * kKBytes;       // 16 KB, of A and of B
constexpr int kStage = 2 * kStageHalf;
constexpr int kStages = 6;
// An fp32 result is summed in segments of so many k-steps of 64 terms, which the
// epilogue adds up in fp32 rounded to nearest.  The tensor core lines up the 16
// terms of an MMA with the accumulator P, cuts them at 2^-25 P and the sum to fp32,
// always towards zero, which over a long reduction costs more than roundings to
// nearest.  Products of bf16 have 16 significant bits and mostly fit: 512 terms of
// one sign lose 7e-7 of their sum.  Products of fp16 have up to 22, and the cut
// terms add their share: 2.5e-6 in 512 terms, 1.1e-6 in 256, 4.6e-7 in 128.  The
// shorter segments cost a tenth to a fifth: DeepSeek-shaped gemm and dgrad with fp32
// results 277 and 262 us in bf16 (255 and 243 with 16-bit ones), 309 and 317 in fp16.
constexpr int kSegment = 8, kSegmentF16 = 2;
// A 16-bit result shows it only over long reductions: n terms of one sign in one
// sum lose 4.8e-9 n of it in fp16 (measured, 2^17 to 2^22 terms: 2.1e-4 to 6.9e-3)
// and 8e-10 n in bf16 (6.8e-5 to 5.2e-3).  Reductions that may be longer than these
// limits, where that is a third and a fifth of half a step (2^-11, 2^-8), go in
// segments of kSegment steps, too (49152 fp16 rows of 64 experts of 2048 x 2816:
// weight gradient 553 us with them, 523 without).
constexpr int64_t kLongF16 = 1 << 15, kLongBf16 = 1 << 20;

constexpr int kBoxRows = 32;                      // rows of one TMA box of the N side
constexpr int kEpiWarps = 8;                      // two for each quarter of the TMEM lanes
constexpr int kEpiBytes = kEpiWarps * 128;        // 8 bits: 32 scales for each

struct TcArgs {
    CUtensorMap tmA, tmB;
    CUtensorMap tmB128;        // gemm, dgrad: tmB's rows in boxes of 128
    const int32_t* offsets;
    void* out;
    const float* a_scale;
    const float* w_scale;
    int64_t out_stride;
    int64_t rows;
    int E;
    int M, N;              // M: output features (wgrad: d_in).  N: wgrad's columns (d_out)
    int nk;                // k-steps of gemm and dgrad
    int split;             // pairs of a tile (SPLIT)
    int segment;           // k-steps of a segment (SEG)
    int m_block;           // gemm, dgrad: weight tiles of a block (see TileWalk)
    int out_dtype, accumulate;
    uint32_t idesc;        // without the N field
};

// Descriptor of an MN-major 16-bit tile as TMA wrote it with the 128-byte
// swizzle: one box is 64 MN elements (128 B) x 64 k rows; 8-row groups of k
// are 1024 B apart (stride byte offset) and the next 64 MN elements one box
// (8 KB) further (leading byte offset).
__device__ __forceinline__ uint64_t umma_desc_mn_sw128(uint32_t addr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((addr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>(8192u >> 4) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(2u) << 61;
    return d;
}

template <bool I8>
__device__ __forceinline__ void umma_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                          uint32_t idesc, uint32_t accumulate) {
    if constexpr (I8)
        asm volatile(
            "{\n .reg .pred p;\n"
            " setp.ne.b32 p, %4, 0;\n"
            " tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n}\n"
            ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate));
    else
        umma_bf16_pair(d_tmem, a_desc, b_desc, idesc, accumulate);
}

// TMA loads that complete on the mbarrier of either CTA of the pair (`mbar`
// is a shared::cluster address).  No multicast.
__device__ __forceinline__ void tma_pair_2d(uint32_t dst, const CUtensorMap* map, uint32_t mbar,
                                            int32_t c0, int32_t c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];"
        ::"r"(dst), "l"(map), "r"(mbar), "r"(c0), "r"(c1) : "memory");
}
__device__ __forceinline__ void tma_pair_3d(uint32_t dst, const CUtensorMap* map, uint32_t mbar,
                                            int32_t c0, int32_t c1, int32_t c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];"
        ::"r"(dst), "l"(map), "r"(mbar), "r"(c0), "r"(c1), "r"(c2) : "memory");
}
__device__ __forceinline__ void fence_proxy_async() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n"
        " mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
// Arrive on `bar` (the same offset) in the CTAs of the cluster that `ctas` names
// once every MMA this thread issued so far completes.
__device__ __forceinline__ void commit_pair(uint32_t bar, uint16_t ctas) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;" ::"r"(bar), "h"(ctas) : "memory");
}
// Arrive on a barrier of either CTA without waiting for this thread's global
// stores (which a release at cluster scope would): what it hands over is tensor
// memory, ordered by the tcgen05 fences.
__device__ __forceinline__ void mbar_arrive_pair(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// The rest of a wait whose first poll failed: at most kWaitLimitNs, and over at
// once when another wait of this CTA has run out.
__device__ __noinline__ bool mbar_wait_slow(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait_cluster(bar, parity)) {
        if (*abort_flag) return false;
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
            *abort_flag = 1;
            atomicOr(&g_grouped_err, kErrTimeout);
            return false;
        }
    }
    return true;
}
// Bounded wait whose acquire covers the other CTA of the pair; false once a wait
// of this CTA has run out.  The loops below do not leave on that (a vote in each
// step costs a sixth of the MMA warp's rate at small tiles): the waits that
// follow return at once and every role runs to its end, loading and storing
// nothing more.
__device__ __forceinline__ bool mbar_wait_cluster(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
    return mbar_try_wait_cluster(bar, parity) || mbar_wait_slow(bar, parity, abort_flag);
}

// A tile of the product.  gemm and dgrad: features m0.., token rows row0 .. row0 +
// valid - 1 as columns.  wgrad: elements m0.. of the rows n0.. of dW[e], the
// reduction over row0 .. row0 + valid - 1.
struct Tile {
    int e, m0, n0, row0, valid;
    int cols;        // MMA N: valid columns rounded up to 32
    int nk;          // k-steps of the tile
    int k_from, k_to;  // ... and of this pair
};

// Walks the tile numbers first, first + step, ...: expert by expert; within an
// expert of gemm and dgrad by blocks of m_block weight tiles, and within a block
// by row chunks, so that the block's weights stay in L2 while the rows stream by
// once for each block.
template <int OP, bool SPLIT>
struct TileWalk {
    const TcArgs& a;
    const int* off;        // in shared memory (wgrad: the caller's table)
    const int* base;       // gemm, dgrad: row chunks of the experts before e
    int mt, nt;
    int t, total;          // both, and t + step, fit: the launch checks it
    int step, pair, e = 0;

    __device__ TileWalk(const TcArgs& args, const int* s_off, const int* s_base, int first, int n, int of_tile)
        : a(args), off(s_off), base(s_base), t(first), step(n), pair(of_tile) {
        mt = (a.M + kTile - 1) / kTile;
        nt = OP == kOpWgrad ? (a.N + kTile - 1) / kTile : 0;
        total = OP == kOpWgrad ? a.E * mt * nt : base[a.E] * mt;
    }
    __device__ bool next(Tile& g) {
        if (t >= total) return false;
        if constexpr (OP == kOpWgrad) {
            const int per = mt * nt;
            g.e = t / per;
            const int r = t - g.e * per;
            // the shorter side varies fastest: its operand is what L2 keeps
            g.m0 = (mt < nt ? r % mt : r / nt) * kTile;
            g.n0 = (mt < nt ? r / mt : r % nt) * kTile;
            // read again by every role: clamped, should the table change under the call
            g.row0 = max(0, off[g.e]);
            g.valid = max(0, static_cast<int>(min(static_cast<int64_t>(off[g.e + 1]), a.rows)) - g.row0);
            g.cols = (min(kTile, a.N - g.n0) + 31) & ~31;
            g.nk = (g.valid + 63) / 64;
        } else {
            // the last expert whose tiles start at or before t, not far from the last one
            int hi = e + 1;
            for (int leap = 1; hi < a.E && base[hi] * mt <= t; leap *= 2) {
                e = hi;
                hi = min(a.E, hi + leap);
            }
            while (hi - e > 1) {
                const int mid = (e + hi) >> 1;
                if (base[mid] * mt <= t) e = mid; else hi = mid;
            }
            const int c0 = base[e], chunks = base[e + 1] - c0;
            const int n = off[e + 1] - off[e];
            const int r = t - c0 * mt;
            int mi = r, ci = 0, per = (n + 31) & ~31;
            if (chunks > 1) {
                const int per_block = chunks * a.m_block;
                const int block = r / per_block, in_block = r - block * per_block;
                const int mb = min(a.m_block, mt - block * a.m_block);
                ci = in_block / mb;
                mi = block * a.m_block + in_block - ci * mb;
                per = ((n + chunks - 1) / chunks + 31) & ~31;
            }
            g.e = e;
            g.m0 = mi * kTile;
            g.n0 = 0;
            g.row0 = off[e] + ci * per;
            g.valid = min(per, n - ci * per);
            g.cols = (g.valid + 31) & ~31;
            g.nk = a.nk;
        }
        g.k_from = 0;
        g.k_to = g.nk;
        if (SPLIT) {
            const int per = (g.nk + a.split - 1) / a.split;
            g.k_from = min(g.nk, pair * per);
            g.k_to = min(g.nk, g.k_from + per);
        }
        t += step;
        return true;
    }
};

template <int OP>
constexpr int tc_threads() { return (2 + kEpiWarps + (OP == kOpWgrad ? 1 : 0)) * 32; }

// Offsets into shared memory, checked; and the running count of row chunks: each
// thread takes kPer experts in a row, then a scan over the warps.  Returns false
// (for every thread of the block) if the table is not sound.
template <int OP>
__device__ bool load_offsets(const TcArgs& a, int* s_off, int* s_base, int* s_warp) {
    constexpr int kPer = 4;
    static_assert(kPer * tc_threads<OP>() >= kMaxExperts, "every expert has a thread");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int e0 = static_cast<int>(threadIdx.x) * kPer;
    bool bad = false;
    int v[kPer + 1], count[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i <= kPer; ++i) v[i] = e0 + i <= a.E ? a.offsets[e0 + i] : 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        count[i] = 0;
        if (e0 + i < a.E) {
            bad |= v[i] < 0 || v[i] > a.rows || v[i + 1] > a.rows || v[i + 1] < v[i];
            count[i] = (v[i + 1] - v[i] + kTile - 1) / kTile;
        }
        sum += count[i];
    }
    if constexpr (OP == kOpWgrad) {
        bad = __syncthreads_or(bad);
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (e0 + i <= a.E) s_off[e0 + i] = v[i];
        if (a.E == kMaxExperts && e0 + kPer == a.E) s_off[a.E] = v[kPer];
        int upto = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += o;
        }
        if (lane == 31) s_warp[warp] = upto;
        bad = __syncthreads_or(bad);
        int before = upto - sum;
        for (int w = 0; w < warp; ++w) before += s_warp[w];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if (e0 + i < a.E) s_base[e0 + i] = before;
            before += count[i];
            if (e0 + i == a.E - 1) s_base[a.E] = before;
        }
    }
    return !bad;
}


// 32 columns (tokens) of this lane's feature as 16-bit values, `n` of them
// stored: even and odd lanes trade half of their packed pairs of tokens, so
// that each holds two features (4 bytes) of 16 tokens.
template <bool FULL>
__device__ __forceinline__ void store_pairs(uint16_t* out, int64_t stride, const uint32_t (&v)[32], int n, bool f16,
                                            uint32_t lanes) {
    const int odd = threadIdx.x & 1;
    const uint32_t sel_lo = odd ? 0x1054u : 0x5410u, sel_hi = odd ? 0x3276u : 0x7632u;
    const int most = n;                            // the same in every lane
    out += odd * 2 * stride;
    n -= odd * 2;
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
        if (!FULL && i >= most) break;
        uint32_t p[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float x = __uint_as_float(v[i + 2 * j]), y = __uint_as_float(v[i + 2 * j + 1]);
            p[j] = f16 ? pack_f16x2(x, y) : pack_bf16x2(x, y);
        }
        // an even lane keeps tokens i, i + 1 and an odd one i + 2, i + 3, of both features
        const uint32_t got = __shfl_xor_sync(lanes, odd ? p[0] : p[1], 1);
        const uint32_t keep = odd ? p[1] : p[0];
        if (FULL || i < n) *reinterpret_cast<uint32_t*>(out) = __byte_perm(keep, got, sel_lo);
        if (FULL || i + 1 < n) *reinterpret_cast<uint32_t*>(out + stride) = __byte_perm(keep, got, sel_hi);
        out += 4 * stride;
    }
}

// 32 accumulator columns (tokens r0 .. of gemm and dgrad, rows of dW in wgrad),
// n of them if below 32, of this lane's feature f; f0 is lane 0's.  Results of
// 16 bits; in 8 bits of fp32, too.
template <bool I8>
__device__ __forceinline__ void store_columns(const TcArgs& a, uint32_t (&v)[32], int64_t r0, int n, int f, int f0,
                                              float ws, float as, uint32_t own) {
    const int lane = threadIdx.x & 31;
    if constexpr (I8) {
        // the tokens' scales (as: of token r0 + lane), four to a load from shared memory
        __syncwarp();
        asm volatile("st.shared.f32 [%0], %1;" ::"r"(own + lane * 4), "f"(as) : "memory");
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
            if (i >= n) break;
            float k[4];
            asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(k[0]), "=f"(k[1]), "=f"(k[2]), "=f"(k[3]) : "r"(own + i * 4));
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[i + j] = __float_as_uint(static_cast<float>(static_cast<int>(v[i + j])) * k[j] * ws);
        }
    }
    if (I8 && a.out_dtype == MOE_DTYPE_F32) {
        float* o = static_cast<float*>(a.out) + r0 * a.out_stride + f;
#pragma unroll
        for (int i = 0; i < 32; ++i, o += a.out_stride)
            if (i < n && f < a.M) *o = __uint_as_float(v[i]);
    } else if (f < a.M) {                         // M is even: both lanes of a pair or neither
        uint16_t* out = static_cast<uint16_t*>(a.out) + r0 * a.out_stride + (f & ~1);
        const bool f16 = a.out_dtype == MOE_DTYPE_F16;
        const uint32_t lanes = f0 + 32 <= a.M ? 0xffffffffu : (1u << (a.M - f0)) - 1u;
        if (n >= 32) store_pairs<true>(out, a.out_stride, v, n, f16, lanes);
        else store_pairs<false>(out, a.out_stride, v, n, f16, lanes);
    }
}

// 16 consecutive fp32 columns of this thread's TMEM lane (warp-wide).
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// SEG: 16-bit operands summed in segments (see kSegment), for fp32 results and long
// reductions.
// SPLIT: a.split pairs (a cluster of 2 a.split CTAs, one tile each) take parts
// of a tile's reduction and trade their sums through distributed shared memory,
// each adding up (in a fixed order) and storing its share of the columns.
template <int OP, bool I8, bool SEG, bool SPLIT>
__global__ void __launch_bounds__(tc_threads<OP>(), 1)
grouped_tc_kernel(const __grid_constant__ TcArgs a) {
    constexpr int kElem = I8 ? 1 : 2;
    constexpr int kBK = kKBytes / kElem;
    extern __shared__ __align__(1024) uint8_t sm_raw[];
    uint8_t* ring = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(sm_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* epi = ring + kStages * kStage;
    uint64_t* full = reinterpret_cast<uint64_t*>(epi + kEpiBytes);
    uint64_t* empty = full + kStages;
    uint64_t* landed = empty + kStages;              // wgrad: this CTA's loads of a step to pad
    uint64_t* padded = landed + kStages;             // ... and both CTAs' zeros written
    uint64_t* tfull = padded + kStages;
    uint64_t* tempty = tfull + 2;
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(tempty + 2);
    int* s_abort = reinterpret_cast<int*>(s_tmem + 1);
    int* s_warp = s_abort + 1;                       // [16]: sums of the warps
    int* s_off = s_warp + 16;
    int* s_base = s_off + a.E + 1;

    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);      // the same in every lane, and known to be
    const int cta = static_cast<int>(cluster_ctarank());
    const int rank = SPLIT ? cta & 1 : cta;                      // in the pair
    const int pair = SPLIT ? cta >> 1 : 0;
    const int leader = cta - rank;                               // the pair's first CTA
    const int unit = static_cast<int>(blockIdx.x) / (SPLIT ? 2 * a.split : 2);
    const int n_units = static_cast<int>(gridDim.x) / (SPLIT ? 2 * a.split : 2);
    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
            mbar_init(&landed[s], 1);
            mbar_init(&padded[s], 2);
        }
        for (int b = 0; b < 2; ++b) { mbar_init(&tfull[b], 1); mbar_init(&tempty[b], 2 * kEpiWarps); }
        *s_abort = 0;
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc_pair(s_tmem, 512);
    if (warp == 0 && elect_one()) {
        prefetch_tensormap(&a.tmA);
        prefetch_tensormap(&a.tmB);
        if (OP != kOpWgrad) prefetch_tensormap(&a.tmB128);
    }
    grid_let_next();
    tc_fence_before();
    cluster_sync_all();       // the peer's barriers are initialised before any signal
    tc_fence_after();
    grid_wait();
    const bool sound = load_offsets<OP>(a, s_off, s_base, s_warp);   // the same in every CTA
    __syncthreads();
    if (!sound) {
        if (tid == 0) atomicOr(&g_grouped_err, kErrBadId);
        if (warp == 1) tmem_dealloc_pair(*s_tmem, 512);
        return;
    }
    const uint32_t tmem = __shfl_sync(0xffffffffu, *s_tmem, 0);
    const uint32_t ring_base = smem_u32(ring);
    const uint32_t full0 = __shfl_sync(0xffffffffu, mapa_shared(smem_u32(full), leader), 0);   // the first CTA's full[0]
    const uint32_t landed0 = __shfl_sync(0xffffffffu, mapa_shared(smem_u32(landed), cta), 0);
    const uint16_t both = static_cast<uint16_t>(3u << leader);
    volatile int* abort_flag = s_abort;
    auto wait = [&](uint32_t bar, uint32_t parity) { return mbar_wait_cluster(bar, parity, abort_flag); };
    const uint32_t full_u = smem_u32(full), empty_u = smem_u32(empty), landed_u = smem_u32(landed);
    const uint32_t padded_u = smem_u32(padded), tfull_u = smem_u32(tfull), tempty_u = smem_u32(tempty);
    TileWalk<OP, SPLIT> walk(a, OP == kOpWgrad ? a.offsets : s_off, s_base, unit, n_units, pair);
    Tile g;

    if (warp == 0) {
        // ------------------------------------------------------ producer
        int s = 0;
        uint32_t phase = 1;                      // a ring that was never filled is free
        int used = 0;                            // stages filled at least once
        bool stop = false;
        while (walk.next(g)) {
            const int half = g.cols / 2;                  // N rows (columns) of this CTA
            const int m0 = g.m0 + kHalf * rank;
            // boxes of the N side: 64 columns (wgrad), or 32 token rows; more than
            // 96 rows take one box of 128
            const bool big = OP != kOpWgrad && half > 96;
            const int nb = OP == kOpWgrad ? (half + 63) / 64 : big ? 4 : (half + kBoxRows - 1) / kBoxRows;
            const uint32_t bytes = kStageHalf + nb * (OP == kOpWgrad ? 8192u : kBoxRows * kKBytes);
            const int r0 = OP == kOpWgrad ? g.row0 : g.row0 + half * rank;
            for (int kb = g.k_from; kb < g.k_to; ++kb) {
                stop |= !wait(empty_u + s * 8, phase);
                const uint32_t A = ring_base + s * kStage;
                const uint32_t B = A + kStageHalf;
                if (elect_one() && !stop) {
                    if constexpr (OP == kOpWgrad) {
                        // a last step that needs padding lands on this CTA's own
                        // barrier, every other on the first CTA's
                        const bool pad = kb == g.nk - 1 && (g.valid & 15);
                        if (pad) mbar_arrive_expect_tx(&landed[s], bytes);
                        if (rank == 0) {
                            if (pad) mbar_arrive(&full[s]);
                            else mbar_arrive_expect_tx(&full[s], 2 * bytes);
                        }
                        const uint32_t bar = pad ? landed0 + s * 8 : full0 + s * 8;
                        const int r = r0 + kb * 64;
                        tma_pair_2d(A, &a.tmA, bar, m0, r);
                        tma_pair_2d(A + 8192, &a.tmA, bar, m0 + 64, r);
                        tma_pair_2d(B, &a.tmB, bar, g.n0 + half * rank, r);
                        if (nb > 1) tma_pair_2d(B + 8192, &a.tmB, bar, g.n0 + half * rank + 64, r);
                    } else {
                        // the loads of both CTAs complete on the first one's barrier
                        if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * bytes);
                        const uint32_t bar = full0 + s * 8;
                        if constexpr (OP == kOpGemm) {
                            tma_pair_3d(A, &a.tmA, bar, kb * kBK, m0, g.e);
                        } else {
                            tma_pair_3d(A, &a.tmA, bar, m0, kb * kBK, g.e);
                            tma_pair_3d(A + 8192, &a.tmA, bar, m0 + 64, kb * kBK, g.e);
                        }
                        if (big) {
                            tma_pair_2d(B, &a.tmB128, bar, kb * kBK, r0);
                        } else {
                            for (int j = 0; j < nb; ++j)
                                tma_pair_2d(B + j * kBoxRows * kKBytes, &a.tmB, bar, kb * kBK, r0 + kBoxRows * j);
                        }
                    }
                }
                if (used < kStages) ++used;
                if (++s == kStages) { s = 0; phase ^= 1; }
            }
        }
        // every issued stage released by the MMAs: no commit arrives in
        // this CTA's shared memory after it exits
        for (; used > 0; --used) {
            if (s == 0) { s = kStages; phase ^= 1; }
            --s;
            stop |= !wait(empty_u + s * 8, phase ^ 1);
        }
        if (stop) __nanosleep(1000000);          // what was still in flight lands
    } else if (warp == 1) {
        // ---------------------------------------------------------- MMA
        // the whole warp runs the loop, so that the descriptors are computed
        // for the warp and not for a lane; one lane issues
        if (rank == 0) {
            // descriptors of the first stage; a stage or k-slice further is an
            // addition to the address field (no carry: 227 KB / 16 < 2^14)
            const uint64_t a0 = OP == kOpGemm ? umma_desc_sw128(ring_base) : umma_desc_mn_sw128(ring_base);
            const uint64_t b0 = OP == kOpWgrad ? umma_desc_mn_sw128(ring_base + kStageHalf)
                                               : umma_desc_sw128(ring_base + kStageHalf);
            constexpr uint32_t kStepA = (OP == kOpGemm ? 32 : 2048) / 16, kStepB = (OP == kOpWgrad ? 2048 : 32) / 16;
            int s = 0, local = 0;
            uint32_t phase = 0;
            uint32_t pad_phase = 0;                  // a bit for each stage: uses of its padded[]
            while (walk.next(g)) {
                if (OP == kOpWgrad && g.nk == 0) continue;     // no rows: the epilogue stores zeros by itself
                const uint32_t idesc = a.idesc | (static_cast<uint32_t>(g.cols >> 3) << 17);
                // full steps, then (wgrad) a last one of 1 to 4 slices of 16 rows
                const int n_full = OP == kOpWgrad && (g.valid & 63) ? g.nk - 1 : g.nk;
                int kb = g.k_from;
                do {                                 // a segment of the reduction
                    const int b = local & 1;
                    wait(tempty_u + b * 8, ((local >> 1) & 1) ^ 1);
                    tc_fence_after();
                    const uint32_t d_tmem = tmem + b * kTile;
                    const int end = SEG ? min(kb + a.segment, g.k_to) : g.k_to, k0 = kb;
                    for (; kb < min(end, n_full); ++kb) {
                        wait(full_u + s * 8, phase);
                        tc_fence_after();
                        const uint64_t ad = a0 + static_cast<uint32_t>(s * (kStage / 16));
                        const uint64_t bd = b0 + static_cast<uint32_t>(s * (kStage / 16));
                        if (elect_one()) {
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                umma_pair<I8>(d_tmem, ad + kk * kStepA, bd + kk * kStepB, idesc, kk ? 1u : kb != k0);
                            commit_pair(empty_u + s * 8, both);
                        }
                        if (++s == kStages) { s = 0; phase ^= 1; }
                    }
                    if (OP == kOpWgrad && kb < end) {
                        wait(full_u + s * 8, phase);
                        if (g.valid & 15) {
                            wait(padded_u + s * 8, (pad_phase >> s) & 1);
                            pad_phase ^= 1u << s;
                        }
                        tc_fence_after();
                        const uint64_t ad = a0 + static_cast<uint32_t>(s * (kStage / 16));
                        const uint64_t bd = b0 + static_cast<uint32_t>(s * (kStage / 16));
                        const int slices = (((g.valid - 1) & 63) >> 4) + 1;
                        if (elect_one()) {
                            for (int kk = 0; kk < slices; ++kk)
                                umma_pair<I8>(d_tmem, ad + kk * kStepA, bd + kk * kStepB, idesc, kk || kb != k0 ? 1u : 0u);
                            commit_pair(empty_u + s * 8, both);
                        }
                        if (++s == kStages) { s = 0; phase ^= 1; }
                        ++kb;
                    }
                    if (elect_one()) commit_pair(tfull_u + b * 8, both);
                    ++local;
                } while (kb < g.k_to);
            }
        }
    } else if (warp < 2 + kEpiWarps) {
        // ----------------------------------------------------- epilogue
        const int q = warp & 3;                        // TMEM lane quarter of this warp
        const int first_part = (warp - 2) >> 2;        // of the quarter's two warps
        const uint32_t own = smem_u32(epi) + (warp - 2) * 128;       // 8 bits: 32 tokens' scales
        int local = 0;
        while (walk.next(g)) {
            const uint32_t lanes = tmem + (static_cast<uint32_t>(q * 32) << 16);
            const int f0 = g.m0 + kHalf * rank + q * 32;      // this warp's first feature
            const int f = f0 + lane;
            const float ws = I8 && f < a.M ? a.w_scale[static_cast<int64_t>(g.e) * a.M + f] : 1.f;
            // columns: tokens, or (wgrad) rows of the expert's dW
            const int valid = OP == kOpWgrad ? min(kTile, a.N - g.n0) : g.valid;
            const int64_t col0 = OP == kOpWgrad ? static_cast<int64_t>(g.e) * a.N + g.n0 : g.row0;
            const bool empty_expert = OP == kOpWgrad && g.nk == 0;
            bool store = f0 < a.M;
            if (empty_expert) {                               // zeros by 16 bytes, or nothing to add
                store = false;
                const int es = a.out_dtype == MOE_DTYPE_F32 ? 4 : 2;
                const int f_cta = g.m0 + kHalf * rank;
                const int units = min(kHalf, a.M - f_cta) * es / 16;      // of a row of this CTA's
                uint8_t* o = static_cast<uint8_t*>(a.out) + (col0 * a.out_stride + f_cta) * es;
                if (units > 0 && pair == 0 && !a.accumulate)
                    for (int i = (warp - 2) * 32 + lane; i < valid * units; i += kEpiWarps * 32)
                        *reinterpret_cast<uint4*>(o + (i / units) * a.out_stride * es + (i % units) * 16) =
                            make_uint4(0, 0, 0, 0);
            }
            auto scale_of = [&](int c) {                      // 8 bits: of this lane's token of column c ..
                return I8 && c + lane < valid ? a.a_scale[col0 + c + lane] : 0.f;
            };
            if constexpr (SEG || SPLIT) {
                // the segments' sums are added up here, in fp32 rounded to nearest
                // (8 bits: one segment, whose words are int32)
                const int part = first_part;
                float sum[kTile / 64][32];
#pragma unroll
                for (int j = 0; j < kTile / 64; ++j)
#pragma unroll
                    for (int i = 0; i < 32; ++i) sum[j][i] = 0.f;
                const bool none = g.k_from == g.k_to;
                const int segments =
                    empty_expert ? 0 : SEG && !none ? (g.k_to - g.k_from + a.segment - 1) / a.segment : 1;
                for (int seg = 0; seg < segments; ++seg, ++local) {
                    const int b = local & 1;
                    // every decision before the warp-collective tcgen05.ld is warp-uniform
                    if (__any_sync(0xffffffffu, !wait(tfull_u + b * 8, (local >> 1) & 1))) { store = false; continue; }
                    tc_fence_after();
#pragma unroll
                    for (int j = 0; j < kTile / 64; ++j) {
                        const int c = part * 32 + j * 64;
                        if (store && !none && c < valid) {
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                uint32_t v[16];
                                tmem_ld16(lanes + b * kTile + c + h * 16, v);
                                tmem_ld_wait();
#pragma unroll
                                for (int i = 0; i < 16; ++i)
                                    sum[j][h * 16 + i] = SEG ? sum[j][h * 16 + i] + __uint_as_float(v[i]) : __uint_as_float(v[i]);
                            }
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_pair(mapa_shared(tempty_u + b * 8, leader));
                }
                // SPLIT: group k of 32 columns is pair k mod split's, who gets the
                // others' sums of it as [other pair][its group][column][128 rows] in its
                // ring, which no load or MMA of the cluster uses after this barrier
                const int groups = SPLIT ? (g.cols / 32 + a.split - 1) / a.split : 0;      // of a pair, at most
                const int mine = (q * 32 + lane) * 4;
                if constexpr (SPLIT) {
                    cluster_sync_all();
#pragma unroll
                    for (int j = 0; j < kTile / 64; ++j) {
                        const int k = part + 2 * j, owner = k & (a.split - 1);
                        if (!store || k * 32 >= valid) break;
                        if (owner == pair) continue;
                        const int from = pair < owner ? pair : pair - 1;
                        const uint32_t to = mapa_shared(ring_base, owner * 2 + rank) + mine +
                                            (from * groups + k / a.split) * (32 * 512);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + i * 512), "f"(sum[j][i]) : "memory");
                    }
                    cluster_sync_all();
                }
#pragma unroll
                for (int j = 0; j < kTile / 64; ++j) {
                    const int k = part + 2 * j, c = k * 32, n = valid - c;
                    if (!store || n <= 0) break;
                    if constexpr (SPLIT) {
                        if ((k & (a.split - 1)) != pair) continue;
                        for (int from = 0; from < a.split - 1; ++from) {
                            const uint8_t* at = ring + mine + (from * groups + k / a.split) * (32 * 512);
#pragma unroll
                            for (int h = 0; h < 32; h += 16) {          // 16 loads in flight
                                float o[16];
#pragma unroll
                                for (int i = 0; i < 16; ++i) o[i] = *reinterpret_cast<const volatile float*>(at + (h + i) * 512);
#pragma unroll
                                for (int i = 0; i < 16; ++i)
                                    sum[j][h + i] = I8 ? __int_as_float(__float_as_int(sum[j][h + i]) + __float_as_int(o[i]))
                                                       : sum[j][h + i] + o[i];
                            }
                        }
                    }
                    if (SEG && a.out_dtype == MOE_DTYPE_F32) {
                        if (f >= a.M) break;
                        float* o = static_cast<float*>(a.out) + (col0 + c) * a.out_stride + f;
                        if (OP == kOpWgrad && a.accumulate) {
                            // each element has one owner: one addition, in no one's order
#pragma unroll
                            for (int i = 0; i < 32; ++i, o += a.out_stride)
                                if (i < n) red_add_f32(o, sum[j][i]);
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; ++i, o += a.out_stride)
                                if (i < n) *o = sum[j][i];
                        }
                    } else {
                        store_columns<I8>(a, reinterpret_cast<uint32_t (&)[32]>(sum[j]), col0 + c, n, f, f0, ws, scale_of(c), own);
                    }
                }
            } else {
                const int b = local & 1;
                // the two warps of a quarter take turns at the first 32 columns, so that
                // tiles of few rows pass through both
                const int part = first_part ^ b;
                float as = scale_of(part * 32);
                if (!empty_expert) {
                    ++local;
                    if (__any_sync(0xffffffffu, !wait(tfull_u + b * 8, ((local - 1) >> 1) & 1))) continue;
                    tc_fence_after();
                }
                const uint32_t taddr = lanes + b * kTile;
                uint32_t v[2][32];
                if (store && part * 32 < valid) tmem_ld32(taddr + part * 32, v[0]);
#pragma unroll 1
                for (int c0 = part * 32; store && c0 < valid; c0 += 128) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {             // this warp's 32 columns of each 64
                        const int c = c0 + j * 64;
                        if (c >= valid) break;
                        tmem_ld_wait();
                        if (c + 64 < valid) tmem_ld32(taddr + c + 64, v[j ^ 1]);
                        const float next_as = scale_of(c + 64);
                        store_columns<I8>(a, v[j], col0 + c, valid - c, f, f0, ws, as, own);
                        as = next_as;
                    }
                }
                if (!empty_expert) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_pair(mapa_shared(tempty_u + b * 8, leader));
                }
            }
        }
    } else {
        // wgrad: zeros the rows past a segment's end in its last step, up to
        // the next multiple of the MMA's 16, once this CTA's loads have landed
        uint32_t it = 0, phase = 0;
        while (walk.next(g)) {
            it += g.k_to - g.k_from;
            const int pad = -g.valid & 15;
            if (pad == 0 || g.k_to != g.nk || g.k_from == g.k_to) continue;
            const int s = (it - 1) % kStages;
            if (__any_sync(0xffffffffu, !wait(landed_u + s * 8, (phase >> s) & 1))) break;
            phase ^= 1u << s;
            const uint32_t base = ring_base + s * kStage + (g.valid & 63) * 128;
            for (int j = lane; j < pad * 8 * 4; j += 32) {          // four boxes of 64 columns
                const uint32_t at = base + (j / (pad * 8)) * 8192 + (j % (pad * 8)) * 16;
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0) : "memory");
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(mapa_shared(padded_u + s * 8, leader));
        }
    }
    if (SPLIT && !(warp >= 2 && warp < 2 + kEpiWarps && walk.t != unit)) {
        // the epilogue's two barriers, for the warps that have no part in it (and
        // for all where the cluster has no tile)
        __syncwarp();
        cluster_sync_all();
        cluster_sync_all();
    }
    tc_fence_before();
    __syncwarp();
    cluster_sync_all();          // no signal into a CTA that has left
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

template <int OP>
size_t tc_smem_bytes(int E) {
    return 1024 + kStages * kStage + (4 * kStages + 4) * 8 + 8 + 16 * 4 +
           kEpiBytes + (OP == kOpWgrad ? 0 : 2 * (static_cast<size_t>(E) + 1) * 4);
}

// ================================================================= host ===
struct DeviceInfo {
    std::atomic<int> pairs{0};             // CTA pairs the device keeps resident; 0: not asked yet
};
DeviceInfo g_info[kMaxDevices];

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static std::atomic<void*> cached{nullptr};
    void* fn = cached.load(std::memory_order_acquire);
    if (!fn) {
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return nullptr;
        cached.store(fn, std::memory_order_release);
    }
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
}

// dims and box of up to three dimensions (innermost first); pitch in bytes.
bool tile_map(CUtensorMap* m, int elem, const void* base, int nd, const uint64_t* dims,
              const uint64_t* pitch, const uint32_t* box) {
    const PFN_cuTensorMapEncodeTiled_v12000 enc = encoder();
    if (!enc) return false;
    const cuuint32_t es[3] = {1, 1, 1};
    const CUtensorMapDataType t = elem == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    return enc(m, t, nd, const_cast<void*>(base), dims, pitch, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool rows_map(CUtensorMap* m, int elem, const void* base, int64_t cols, int64_t rows, int64_t stride,
              uint32_t box_cols, uint32_t box_rows) {
    const uint64_t dims[2] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows)};
    const uint64_t pitch[1] = {static_cast<uint64_t>(stride) * elem};
    const uint32_t box[2] = {box_cols, box_rows};
    return tile_map(m, elem, base, 2, dims, pitch, box);
}

bool stack_map(CUtensorMap* m, int elem, const void* base, int64_t cols, int64_t rows, int64_t n,
               uint32_t box_cols, uint32_t box_rows) {
    const uint64_t dims[3] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows), static_cast<uint64_t>(n)};
    const uint64_t pitch[2] = {static_cast<uint64_t>(cols) * elem, static_cast<uint64_t>(cols) * rows * elem};
    const uint32_t box[3] = {box_cols, box_rows, 1};
    return tile_map(m, elem, base, 3, dims, pitch, box);
}

// Once per device: raise the kernels' shared-memory limit and ask how many
// pairs fit.
template <int OP, bool I8, bool SEG, bool SPLIT>
bool prepare_kernel(int* pairs) {
    auto* k = grouped_tc_kernel<OP, I8, SEG, SPLIT>;
    const int smem = static_cast<int>(tc_smem_bytes<OP>(kMaxExperts));
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return false;
    // clusters of 8 are within the portable size: nothing more to ask for
    if (SPLIT) return true;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(tc_threads<OP>());
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2; attr[0].val.clusterDim.y = 1; attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, k, &cfg) != cudaSuccess || n < 1) return false;
    *pairs = *pairs == 0 || n < *pairs ? n : *pairs;
    return true;
}

template <int OP, bool I8, bool SEG>
bool prepare_kernels(int* pairs) {
    return prepare_kernel<OP, I8, SEG, false>(pairs) && prepare_kernel<OP, I8, SEG, true>(pairs);
}

int device_pairs() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
    int n = g_info[dev].pairs.load(std::memory_order_acquire);
    if (n) return n;
    if (!prepare_kernels<kOpGemm, false, false>(&n) || !prepare_kernels<kOpGemm, false, true>(&n) ||
        !prepare_kernels<kOpGemm, true, false>(&n) || !prepare_kernels<kOpDgrad, false, false>(&n) ||
        !prepare_kernels<kOpDgrad, false, true>(&n) || !prepare_kernels<kOpWgrad, false, false>(&n) ||
        !prepare_kernels<kOpWgrad, false, true>(&n)) {
        cudaGetLastError();
        return 0;
    }
    g_info[dev].pairs.store(n, std::memory_order_release);
    return n;
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Pairs that share a tile's reduction.  With so few tiles that most SMs would
// idle, two or four pairs to a tile share its loads (an SM fills its shared
// memory at about 100 GB/s) for some 3 us of trading sums.  Measured, 1 / 2 / 4
// pairs: 64 rows through 4096 x 1024 (4 tiles, 64 k-steps) 19.5 / 14.4 / 11.6 us,
// 4096 x 3328 (13 tiles) 19.7 / 14.4 / 12.1, 4096 x 4096 (16) 19.7 / 14.9 / 22.3 (not
// all of its 8-CTA clusters fit at once), 2048 x 8192 (32 tiles, 32 steps) 12.8 / 11.8
// / 27.6, 1024 x 1024 (16 steps) 8.9 / 9.3 / 8.9; with more than 128 columns to
// trade, a weight gradient of 24 steps and 12 tiles 13.9 / 14.0 / 14.4.
int pick_split(int64_t tiles, int nk, int cols) {
    if (nk < (cols > 128 ? 32 : 24)) return 1;
    return tiles <= 13 ? 4 : tiles <= 32 ? 2 : 1;
}

template <int OP, bool I8, bool SEG>
moe_status_t launch_tc(TcArgs& a, int64_t tiles, int nk, int cols, cudaStream_t stream) {
    const int pairs = device_pairs();
    if (!pairs) return MOE_ERR_CUDA;
    a.split = pick_split(tiles, nk, cols);
    const dim3 grid(2 * static_cast<unsigned>(a.split > 1 ? tiles * a.split : tiles < pairs ? tiles : pairs));
    const size_t smem = tc_smem_bytes<OP>(a.E);
    const cudaError_t e =
        a.split > 1 ? launch_chained(grouped_tc_kernel<OP, I8, SEG, true>, grid, tc_threads<OP>(), smem, 2 * a.split, stream, a)
                    : launch_chained(grouped_tc_kernel<OP, I8, SEG, false>, grid, tc_threads<OP>(), smem, 2, stream, a);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// Whether a product goes to grouped_small_kernel, which takes 8 rows of an expert in
// a pass over its weights.  Measured in us, small / tensor cores, twelve sets of
// weights in turn (so from HBM where one is above 10 MB), bf16 (8 bits alike at the
// same bytes):
//  - few tiles, one pass.  8 rows through 512 x 4096 (16 tiles) 3.7 / 5.4, 2048 x 4096
//    6.9 / 10, 8192 x 4096 17 / 21; with 32 tiles 512 x 8192 6 / 6, 2048 x 8192 10.6 /
//    12.1, but 4096 x 8192 18 / 17, 8192 x 8192 29 / 28 and with 24 tiles 8192 x 6144
//    28 / 24, where two pairs share a tile.  One row costs what 8 do;
//  - few tiles, two passes (10 to 16 rows of an expert).  The second reads the weights
//    from L2: 2048 x 2048 (8 tiles) 8.2 / 9.1, 2048 x 4096 9.1 / 10, but 4096 x 4096 14.5 /
//    13.6, 2048 x 8192 15.7 / 12.1, 8192 x 2048 21.6 / 14.6;
//  - one to two waves of tiles, the second of which would leave most pairs idle.
//    80 tiles: 4096 x 2560 38 / 42, 8192 x 2560 66 / 81, 14336 x 2560 110 / 131; 96 (six
//    experts of 4096): 4096 45 / 43, 8192 79 / 81, 14336 131 / 135; but 112: 8192 90 / 82,
//    14336 151 / 137; 128: 2048 30 / 24, 8192 95 / 88, 14336 158 / 148.  The call does not
//    know how many experts have rows: the rule takes what even routing reaches.
bool few_rows(const GroupedCall& c) {
    const int64_t slots = c.rows < c.E ? c.rows : c.E;      // experts with rows, at most
    const int64_t per_expert = ceil_div(c.d_out, kTile), tiles = slots * per_expert;
    const int64_t k_bytes = static_cast<int64_t>(c.d_in) * (c.dtype == MOE_DTYPE_I8 ? 1 : 2);
    if (tiles <= 16) return c.rows <= (k_bytes <= 4096 ? 16 : 8) * slots;
    if (tiles <= 37) return k_bytes <= 4096 && c.rows <= 8 * slots;
    if (tiles <= 74 || c.rows > 2 * slots || k_bytes < 8192) return false;
    const double reached = c.E * (1 - std::pow(1 - 1.0 / c.E, static_cast<double>(c.rows))) * per_expert;
    return reached > 74 && reached <= 100;
}

}  // namespace

moe_status_t launch_grouped(GroupedOp op, const GroupedCall& c, cudaStream_t stream) {
    const bool i8 = c.dtype == MOE_DTYPE_I8;
    const int elem = i8 ? 1 : 2;
    const int bk = kKBytes / elem;
    if (c.rows == 0) {
        if (op != kOpWgrad || c.accumulate) return MOE_OK;
        const size_t n = static_cast<size_t>(c.E) * c.d_out * c.d_in * (c.out_dtype == MOE_DTYPE_F32 ? 4 : 2);
        return cudaMemsetAsync(c.out, 0, n, stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
    }
    const int segment = c.dtype == MOE_DTYPE_F16 && c.out_dtype == MOE_DTYPE_F32 ? kSegmentF16 : kSegment;
    if (op == kOpGemm && few_rows(c)) {
        SmallArgs m{};
        m.offsets = c.offsets;
        m.x = static_cast<const uint8_t*>(c.a);
        m.w = static_cast<const uint8_t*>(c.w);
        m.out = c.out;
        m.a_scale = c.a_scale;
        m.w_scale = c.w_scale;
        m.x_bytes = c.x_stride * elem;
        m.out_stride = c.y_stride;
        m.rows = c.rows;
        m.E = c.E;
        m.M = c.d_out;
        m.k_bytes = c.d_in * elem;
        m.f16 = c.dtype == MOE_DTYPE_F16;
        m.out_dtype = c.out_dtype;
        m.segment = segment;
        const int64_t units = ceil_div(c.d_out, kSmallRows) * (c.rows < c.E ? c.rows : c.E);    // at most
        const unsigned grid = static_cast<unsigned>(units < 2 * 148 ? units : 2 * 148);
        const cudaError_t e = launch_chained(i8 ? grouped_small_kernel<true> : grouped_small_kernel<false>, dim3(grid),
                                             kSmallThreads, 0, 1, stream, m);
        return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
    }
    TcArgs a;
    memset(&a, 0, sizeof(a));
    a.offsets = c.offsets;
    a.out = c.out;
    a.a_scale = c.a_scale;
    a.w_scale = c.w_scale;
    a.rows = c.rows;
    a.E = c.E;
    a.out_dtype = c.out_dtype;
    a.accumulate = c.accumulate;
    a.segment = segment;
    // D fp32 (int32), A and B bf16 (signed 8-bit; fp16 is 0), M 256 over the pair
    a.idesc = (i8 ? 2u << 4 : 1u << 4) | (16u << 24);
    if (c.dtype != MOE_DTYPE_F16) a.idesc |= (1u << 7) | (1u << 10);
    bool ok = true;
    int64_t tiles = 0;
    if (op != kOpWgrad) {
        // weight tiles that take 32 MB, a quarter of L2
        const int64_t k_bytes = static_cast<int64_t>(op == kOpGemm ? c.d_in : c.d_out) * elem;
        const int64_t mb = (32 << 20) / (kTile * k_bytes);
        a.m_block = static_cast<int>(mb < 1 ? 1 : mb > 64 ? 64 : mb);
    }
    // at most so many row chunks: each expert with rows adds at most 255 of padding
    const int64_t chunks = (c.rows + 255 * (c.rows < c.E ? c.rows : c.E)) / kTile;
    int nk, cols = c.rows < kTile ? static_cast<int>(c.rows) : kTile;      // of a tile, at most
    if (op == kOpGemm) {
        a.M = c.d_out;
        a.nk = static_cast<int>(ceil_div(c.d_in, bk));
        a.out_stride = c.y_stride;
        ok &= stack_map(&a.tmA, elem, c.w, c.d_in, c.d_out, c.E, bk, kHalf);
        ok &= rows_map(&a.tmB, elem, c.a, c.d_in, c.rows, c.x_stride, bk, kBoxRows);
        ok &= rows_map(&a.tmB128, elem, c.a, c.d_in, c.rows, c.x_stride, bk, 128);
        tiles = chunks * ceil_div(a.M, kTile);
        nk = a.nk;
    } else if (op == kOpDgrad) {
        a.M = c.d_in;
        a.nk = static_cast<int>(ceil_div(c.d_out, bk));
        a.out_stride = c.x_stride;
        a.idesc |= 1u << 15;                               // A MN-major
        ok &= stack_map(&a.tmA, elem, c.w, c.d_in, c.d_out, c.E, 64, 64);
        ok &= rows_map(&a.tmB, elem, c.a, c.d_out, c.rows, c.y_stride, bk, kBoxRows);
        ok &= rows_map(&a.tmB128, elem, c.a, c.d_out, c.rows, c.y_stride, bk, 128);
        tiles = chunks * ceil_div(a.M, kTile);
        nk = a.nk;
    } else {
        a.M = c.d_in;
        a.N = c.d_out;
        a.out_stride = c.d_in;
        a.idesc |= (1u << 15) | (1u << 16);                // A and B MN-major
        ok &= rows_map(&a.tmA, elem, c.w, c.d_in, c.rows, c.x_stride, 64, 64);
        ok &= rows_map(&a.tmB, elem, c.a, c.d_out, c.rows, c.y_stride, 64, 64);
        tiles = static_cast<int64_t>(c.E) * ceil_div(a.M, kTile) * ceil_div(a.N, kTile);
        nk = static_cast<int>(ceil_div(c.rows, 64 * static_cast<int64_t>(c.E)));            // on average
        cols = a.N < kTile ? a.N : kTile;
    }
    if (!ok || tiles > 0x7FFF0000) return MOE_ERR_INVALID_ARG;
    if (i8) return launch_tc<kOpGemm, true, false>(a, tiles, nk, cols, stream);
    const int64_t terms = op == kOpGemm ? c.d_in : op == kOpDgrad ? c.d_out : c.rows;        // of a sum, at most
    if (c.out_dtype == MOE_DTYPE_F32 || terms > (c.dtype == MOE_DTYPE_F16 ? kLongF16 : kLongBf16)) {
        if (op == kOpGemm) return launch_tc<kOpGemm, false, true>(a, tiles, nk, cols, stream);
        if (op == kOpDgrad) return launch_tc<kOpDgrad, false, true>(a, tiles, nk, cols, stream);
        return launch_tc<kOpWgrad, false, true>(a, tiles, nk, cols, stream);
    }
    if (op == kOpGemm) return launch_tc<kOpGemm, false, false>(a, tiles, nk, cols, stream);
    if (op == kOpDgrad) return launch_tc<kOpDgrad, false, false>(a, tiles, nk, cols, stream);
    return launch_tc<kOpWgrad, false, false>(a, tiles, nk, cols, stream);
}

moe_status_t grouped_status_read() {
    uint32_t v = 0;
    const uint32_t zero = 0;
    if (cudaDeviceSynchronize() != cudaSuccess) return MOE_ERR_CUDA;
    if (cudaMemcpyFromSymbol(&v, g_grouped_err, 4) != cudaSuccess) return MOE_ERR_CUDA;
    if (v && cudaMemcpyToSymbol(g_grouped_err, &zero, 4) != cudaSuccess) return MOE_ERR_CUDA;
    if (v & kErrTimeout) return MOE_ERR_TIMEOUT;
    return v ? MOE_ERR_DEVICE_FLAG : MOE_OK;
}

}  // namespace moe
