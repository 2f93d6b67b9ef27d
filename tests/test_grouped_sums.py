"""How exact the sums of the experts' products are, with operands of one sign.

There the sum of the absolute values is the result itself, so a bias towards
zero cannot hide behind terms that cancel.  Operands lie in [1, 1.25]: products
in [1, 25/16], and a partial sum of i MMAs of 16 terms is at most 25 i.

What a tensor core loses (its alignment, seen by adding 15 equal terms to one
2^k times as large: whole down to 2^-25 of it, partly or wholly gone from 2^-26 on): each MMA
lines its addends up with the largest partial sum P and cuts each at or below
2^-25 P, 16 of them 4 * 2^-23 P together, and then cuts the sum to fp32, 2^-23 P,
all towards zero.  In bf16 the products are multiples of 2^-14 and no segment of
512 terms reaches 2^10, whose addends are cut at 2^-16: only the sum's cut is
left.  So an MMA loses at most c 2^-23 P with c = 1 (bf16) or 5 (fp16), a segment of
m MMAs at most c 2^-23 25 m (m + 1) / 2, and n terms in segments of m MMAs at most
c 2^-23 (25 / 32) (m + 1) n.

Adding the segments up rounds to nearest, each time at most 2^-24 of what has
been added so far: J in a row cost at most 2^-24 (25 / 16) (J + 1) / 2 of the sum,
and a few more for the parts of a block, a pair or a pair of accumulators.
"""
import numpy as np
import pytest
import torch

from mixture_experts_layer_43_b200 import binding as B

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
MOE = {"bf16": B.MOE_DTYPE_BF16, "f16": B.MOE_DTYPE_F16, "f32": B.MOE_DTYPE_F32}
CUTS = {"bf16": 1, "f16": 5}                      # c above
MMAS = 32                                         # MMAs of a segment, at most


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def _above_one(shape, dtype, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return (1 + torch.rand(shape, generator=gen, device="cuda") / 4).to(T[dtype])


def _offsets(counts):
    return torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda")


def _done():
    torch.cuda.synchronize()
    assert B.moe_grouped_status() == B.MOE_OK


def _product64(a, b):
    """a [m][n] times b [o][n], transposed, in 64 bits."""
    out = torch.zeros((a.shape[0], b.shape[0]), dtype=torch.float64, device="cuda")
    for i in range(0, a.shape[1], 1 << 16):
        out += a[:, i:i + (1 << 16)].double() @ b[:, i:i + (1 << 16)].double().T
    return out


def _bound(n, ref, dtype, joins, more):
    return CUTS[dtype] * 2.0 ** -23 * (25 / 32) * (MMAS + 1) * n + ref * 2.0 ** -24 * ((25 / 16) * (joins + 1) / 2 + more)


def gemm(counts, d_in, d_out, dtype, out, seed=1, scale=1.0):
    E, R = len(counts), sum(counts)
    off = _offsets(counts)
    x, w = _above_one((R, d_in), dtype, seed) * scale, _above_one((E, d_out, d_in), dtype, seed + 1) * scale
    y = torch.empty((R, d_out), dtype=T[out], device="cuda")
    B.moe_grouped_gemm(B.moe_grouped_t(R, E, d_in, d_out, MOE[dtype], MOE[out], 0, off.data_ptr(), d_in, d_out),
                       x.data_ptr(), w.data_ptr(), y.data_ptr(), torch.cuda.current_stream().cuda_stream)
    _done()
    ends = off.tolist()
    ref = torch.cat([_product64(x[a:b], w[e]) for e, (a, b) in enumerate(zip(ends[:-1], ends[1:]))])
    return y, ref


# few rows: a block's eight warps share the reduction, each adding its two accumulators to its part of the sum after
# every segment: a join for each 8 steps of 1024 terms, the accumulators' own and the warps' 8
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("counts,d_in,d_out", [([1], 1024, 64), ([2, 0, 1], 8192 + 8, 24), ([3, 1], 65536, 40),
                                               ([0, 2], (1 << 18) - 8, 16), ([1, 1], 1 << 20, 8)], ids=str)
def test_few_rows_of_any_length(counts, d_in, d_out, dtype):
    y, ref = gemm(counts, d_in, d_out, dtype, "f32")
    tol = _bound(d_in, ref, dtype, joins=-(-d_in // 8192), more=1 + 8 + 1)
    err = (y.double() - ref).abs()
    assert bool((err <= tol).all()), f"{(err / ref).max().item():.3g} of the sum, {(tol / ref).max().item():.3g} allowed"


# In earnest: segments of 512 terms in bf16 and of 128 in fp16.  A cut loses half of its most on average, and 2^-23 P
# stands for one unit of fp32, which is 0.72 of that on average over P's significand: 0.36 2^-23 P for the sum and, where
# every bit of the terms is at stake, 1.44 2^-23 P for the 16 of them.  Segments of m MMAs of even terms then lose
# (m + 1) / 2 times as much of their sum: 16.5 * 0.36 * 2^-23 = 7.1e-7 in bf16 and 4.5 * 1.8 * 2^-23 = 9.7e-7 in fp16,
# on average over the elements.
def _average(y, ref):
    return ((y.double() - ref) / ref).mean().abs().item()


# one pair a tile; two and four pairs that share a reduction; few rows; ends inside a k-step
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("counts,d_in,d_out", [([300], 1024, 4104), ([300], 8192 + 8, 4104), ([64], 8192, 4096 + 8),
                                               ([40, 0, 30], 65536, 264), ([2, 1], 1024, 264), ([1, 3], 65536, 40)], ids=str)
def test_gemm_in_32_bits(counts, d_in, d_out, dtype):
    y, ref = gemm(counts, d_in, d_out, dtype, "f32", seed=5)
    err, tol = (y.double() - ref).abs(), _bound(d_in, ref, dtype, joins=-(-d_in // 128), more=10)
    assert bool((err <= tol).all()), f"{(err / ref).max().item():.3g} of the sum"
    assert _average(y, ref) <= 1e-6


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("counts,d_in,d_out", [([300, 21], 4104, 1024), ([64], 264, 65536)], ids=str)
def test_dgrad_in_32_bits(counts, d_in, d_out, dtype):
    E, R, off = len(counts), sum(counts), _offsets(counts)
    dy, w = _above_one((R, d_out), dtype, 7), _above_one((E, d_out, d_in), dtype, 8)
    dx = torch.empty((R, d_in), device="cuda")
    B.moe_grouped_dgrad(B.moe_grouped_t(R, E, d_in, d_out, MOE[dtype], 2, 0, off.data_ptr(), d_in, d_out),
                        dy.data_ptr(), w.data_ptr(), dx.data_ptr(), torch.cuda.current_stream().cuda_stream)
    _done()
    ends = off.tolist()
    ref = torch.cat([_product64(dy[a:b], w[e].T) for e, (a, b) in enumerate(zip(ends[:-1], ends[1:]))])
    err, tol = (dx.double() - ref).abs(), _bound(d_out, ref, dtype, joins=-(-d_out // 128), more=10)
    assert bool((err <= tol).all()), f"{(err / ref).max().item():.3g} of the sum"
    assert _average(dx, ref) <= 1e-6


def wgrad(counts, d_in, d_out, dtype, out, accumulate=0, scale=1.0):
    E, R, off = len(counts), sum(counts), _offsets(counts)
    dy, x = _above_one((R, d_out), dtype, 9) * scale, _above_one((R, d_in), dtype, 10) * scale
    dw = torch.zeros((E, d_out, d_in), dtype=T[out], device="cuda")
    B.moe_grouped_wgrad(B.moe_grouped_t(R, E, d_in, d_out, MOE[dtype], MOE[out], accumulate, off.data_ptr(), d_in, d_out),
                        dy.data_ptr(), x.data_ptr(), dw.data_ptr(), torch.cuda.current_stream().cuda_stream)
    _done()
    ends = off.tolist()
    return dw, torch.stack([_product64(dy[a:b].T, x[a:b].T) for a, b in zip(ends[:-1], ends[1:])])


# many tiles; a few that pairs share; accumulated
@pytest.mark.parametrize("acc", [0, 1])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("counts,d_in,d_out", [([1000, 8200], 1032, 2056), ([8200], 264, 72), ([70001], 64, 264)], ids=str)
def test_wgrad_in_32_bits(counts, d_in, d_out, dtype, acc):
    dw, ref = wgrad(counts, d_in, d_out, dtype, "f32", acc)
    for e, n in enumerate(counts):
        err, tol = (dw[e].double() - ref[e]).abs(), _bound(n, ref[e], dtype, joins=-(-n // 128), more=10)
        assert bool((err <= tol).all()), f"{(err / ref[e]).max().item():.3g} of the sum"
        assert _average(dw[e], ref[e]) <= 1e-6


# Results of 16 bits: a reduction long enough for the cuts to show in half a step of the result goes in segments, too
def _close16(got, ref, n, dtype, joins):
    info = torch.finfo(T[dtype])
    tol = _bound(n, ref, dtype, joins, more=10)
    tol = tol + (ref + tol) * (info.eps / 2) + info.smallest_normal * info.eps / 2
    err = (got.double() - ref).abs()
    assert bool((err <= tol).all()), f"{(err / ref).max().item():.3g} of the sum, half a step is {info.eps / 2:.3g}"


@pytest.mark.parametrize("counts,d_in,d_out,dtype", [([1 << 18], 40, 24, "f16"), ([70001, 0, 5, 200000], 264, 136, "f16"),
                                                     ([(1 << 22) + 3], 16, 8, "bf16")], ids=str)
def test_wgrad_of_millions_of_rows_in_16_bits(counts, d_in, d_out, dtype):
    # by 2^-8 each, exact: sums of 2^18 products stay in fp16's range
    dw, ref = wgrad(counts, d_in, d_out, dtype, dtype, scale=2.0 ** -8)
    for e, n in enumerate(counts):
        _close16(dw[e], ref[e], n * 2.0 ** -16, dtype, joins=-(-n // 512))


@pytest.mark.parametrize("counts,d_in,d_out", [([64], (1 << 20) - 8, 16), ([20, 0, 44], 1 << 19, 264), ([2], 1 << 20, 8)], ids=str)
def test_long_products_in_fp16(counts, d_in, d_out):
    y, ref = gemm(counts, d_in, d_out, "f16", "f16", scale=2.0 ** -8)
    _close16(y, ref, d_in * 2.0 ** -16, "f16", joins=-(-d_in // 512))


def test_long_dgrad_in_fp16():
    R, d_in, d_out, off = 50, 24, 1 << 20, _offsets([50])
    dy, w = _above_one((R, d_out), "f16", 11) * 2.0 ** -8, _above_one((1, d_out, d_in), "f16", 12) * 2.0 ** -8
    dx = torch.empty((R, d_in), dtype=torch.float16, device="cuda")
    B.moe_grouped_dgrad(B.moe_grouped_t(R, 1, d_in, d_out, 1, 1, 0, off.data_ptr(), d_in, d_out),
                        dy.data_ptr(), w.data_ptr(), dx.data_ptr(), torch.cuda.current_stream().cuda_stream)
    _done()
    _close16(dx, _product64(dy, w[0].T), d_out * 2.0 ** -16, "f16", joins=-(-d_out // 512))


# The product of few rows by each of its rules, against 64 bits; random signs, so that the sums cancel: bounds as
# in the tests of the tensor-core products, (n / 16 + 13) 2^-23 of the terms' absolute sum
FEW = [
    ([1], 4096, 4096),                               # a row, 16 tiles
    ([8, 8], 8200, 2048),                            # one full pass, long
    ([9, 16, 0, 1], 2048, 1032),                     # a second pass, full and of one row, short
    ([21, 1, 0, 3, 0, 0, 1, 2], 264, 520),           # three passes of one expert, 24 tiles
    ([2, 0, 1, 1, 0, 4, 0, 0], 8200, 4104),          # long tiles that would make two waves (8 rows, 136 tiles at most)
    ([1] * 18 + [0] * 46, 8192, 1536),               # the same of many experts (108 tiles at most)
]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "i8"])
@pytest.mark.parametrize("counts,d_in,d_out", FEW, ids=lambda v: str(v)[:24])
def test_few_rows_by_every_rule(counts, d_in, d_out, dtype):
    E, R, off = len(counts), sum(counts), _offsets(counts)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(d_in + d_out)
    st = torch.cuda.current_stream().cuda_stream
    y = torch.full((R, d_out + 8), -77.0, device="cuda")
    if dtype == "i8":
        d_in = d_in // 16 * 16
        x, w = (torch.randint(-127, 128, s, generator=gen, device="cuda", dtype=torch.int32).to(torch.int8)
                for s in ((R, d_in), (E, d_out, d_in)))
        xs, ws = torch.rand(R, generator=gen, device="cuda") + 0.5, torch.rand((E, d_out), generator=gen, device="cuda") + 0.5
        B.moe_i8_grouped_gemm(B.moe_grouped_t(R, E, d_in, d_out, B.MOE_DTYPE_I8, 2, 0, off.data_ptr(), d_in, d_out + 8),
                              x.data_ptr(), xs.data_ptr(), w.data_ptr(), ws.data_ptr(), y.data_ptr(), st)
    else:
        x = torch.randn((R, d_in), generator=gen, device="cuda").to(T[dtype])
        w = (torch.randn((E, d_out, d_in), generator=gen, device="cuda") * 0.05).to(T[dtype])
        B.moe_grouped_gemm(B.moe_grouped_t(R, E, d_in, d_out, MOE[dtype], 2, 0, off.data_ptr(), d_in, d_out + 8),
                           x.data_ptr(), w.data_ptr(), y.data_ptr(), st)
    _done()
    assert bool((y[:, d_out:] == -77.0).all())
    for e, (a, b) in enumerate(zip(off.tolist()[:-1], off.tolist()[1:])):
        xe, we = x[a:b].double(), w[e].double()
        ref = xe @ we.T
        if dtype == "i8":
            ref = ref * xs[a:b, None].double() * ws[e].double()
            tol = ref.abs() * (4.5 * 2.0 ** -24)
        else:
            tol = (d_in / 16 + 13) * 2.0 ** -23 * (xe.abs() @ we.abs().T) + ref.abs() * 2.0 ** -24
        assert bool(((y[a:b, :d_out].double() - ref).abs() <= tol).all()), f"expert {e}"
