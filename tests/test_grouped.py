"""The experts' operators on the GPU against plain evaluations in 64 bits.

Tolerances, derived element by element:
  * a result rounded to type t is off by at most half a step,
    finfo(t).eps / 2 of its value (below the smallest normal number: half of
    the smallest subnormal);
  * a product's sum: the products of two 16-bit numbers are exact in fp32 (at
    most 22 significant bits); a tensor core adds 16 of them at a time to the
    accumulator, with the addends cut at or below 2^-23 of the largest and one
    cut of the sum to fp32.  Over n terms whose absolute values add up to S the
    error is at most (n / 16 + 9) 2^-23 S; further roundings to nearest of the
    partial sums (splits of the reduction, sums kept in registers) add one
    2^-24 S for each, counted as 8 more;
  * 8-bit products: the integer sum is exact; its conversion and the two
    scalings round three times, 2^-24 each (4 counted);
  * SwiGLU: the power of two within 2^-22, its correction's sum and product and
    the sum 1 + e^-g half a step each, the reciprocal one step (2^-23), two
    products half a step each: at most (4 + 1 + 1 + 1 + 2 + 2) 2^-24 = 11 * 2^-24
    relative, the sigmoid alone 9 * 2^-24.
"""
import ctypes

import numpy as np
import pytest
import torch

from mixture_experts_layer_43_b200 import binding as B
from mixture_experts_layer_43_b200 import device as D
from mixture_experts_layer_43_b200 import synth

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
MOE = {"bf16": B.MOE_DTYPE_BF16, "f16": B.MOE_DTYPE_F16, "f32": B.MOE_DTYPE_F32, "i8": B.MOE_DTYPE_I8}
U24 = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _ok():
    torch.cuda.synchronize()
    assert B.moe_grouped_status() == B.MOE_OK


def _within(got, ref, tol, what):
    d = (got.double() - ref).abs()
    # a value half a step or more above the largest number of its type rounds to infinity
    info = torch.finfo(got.dtype)
    over = got.isinf() & (ref.abs() >= info.max * (1 + info.eps / 4)) & (torch.sign(got).double() == torch.sign(ref))
    d = torch.where(over, 0.0, d)
    worst = (d - tol).max().item() if d.numel() else 0.0
    assert d.numel() == 0 or bool((d <= tol).all()), \
        f"{what}: {int((~(d <= tol)).sum())} of {d.numel()} outside, worst by {worst:.3g}"


def _rounding(ref, dtype):
    t = torch.finfo(T[dtype])
    return ref.abs() * (t.eps / 2) + t.smallest_normal * t.eps / 2


def _sum_tol(n, s):
    return (n / 16 + 9 + 4) * 2 * U24 * s


class Group:
    """A ragged grouping with poisoned rows before and behind the segments, padded row strides
    and guard values around the outputs."""

    def __init__(self, counts, d_in, d_out, dtype, before=0, behind=0, pad_x=0, pad_y=0, seed=0):
        self.counts, self.d_in, self.d_out, self.dtype = counts, d_in, d_out, dtype
        self.E, self.before = len(counts), before
        self.rows = before + sum(counts) + behind
        off = before + np.concatenate([[0], np.cumsum(counts)])
        self.off = [int(v) for v in off]
        self.offsets = torch.tensor(self.off, dtype=torch.int32, device="cuda")
        self.gen = torch.Generator(device="cuda")
        self.gen.manual_seed(seed + 17)
        self.pad = {"x": pad_x, "y": pad_y}

    def spans(self):
        return [(e, a, b) for e, (a, b) in enumerate(zip(self.off[:-1], self.off[1:])) if b > a]

    def sides(self, side):
        return self.d_in if side == "x" else self.d_out

    def normal(self, shape, scale):
        return torch.randn(shape, generator=self.gen, device="cuda") * scale

    def rows_in(self, side, scale, dtype=None):
        """[rows][d] inside a buffer of wider rows; everything that belongs to nobody is NaN."""
        d = self.sides(side)
        buf = torch.full((self.rows, d + self.pad[side]), float("nan"), device="cuda")
        lo, hi = self.off[0], self.off[-1]
        buf[lo:hi, :d] = self.normal((hi - lo, d), scale)
        return buf.to(T[dtype or self.dtype])

    def rows_out(self, side, dtype):
        return torch.full((self.rows, self.sides(side) + self.pad[side]), -77.0, device="cuda").to(T[dtype])

    def untouched(self, out, side):
        d = self.sides(side)
        lo, hi = self.off[0], self.off[-1]
        assert bool((out[:lo] == -77.0).all()) and bool((out[hi:] == -77.0).all())
        assert bool((out[lo:hi, d:] == -77.0).all())
        return out[:, :d]

    def weights(self):
        return self.normal((self.E, self.d_out, self.d_in), 0.05).to(T[self.dtype])

    def g(self, out, accumulate=0, dtype=None):
        return B.moe_grouped_t(self.rows, self.E, self.d_in, self.d_out, MOE[dtype or self.dtype], MOE[out],
                               accumulate, self.offsets.data_ptr(), self.d_in + self.pad["x"],
                               self.d_out + self.pad["y"])


def check_gemm(G, out):
    x, w, y = G.rows_in("x", 1.0), G.weights(), G.rows_out("y", out)
    B.moe_grouped_gemm(G.g(out), x.data_ptr(), w.data_ptr(), y.data_ptr(), _stream())
    _ok()
    got = G.untouched(y, "y")
    for e, a, b in G.spans():
        xe, we = x[a:b, :G.d_in].double(), w[e].double()
        ref = xe @ we.T
        tol = _sum_tol(G.d_in, xe.abs() @ we.abs().T) + _rounding(ref, out)
        _within(got[a:b], ref, tol * (1 + 1e-6), f"expert {e}")


def check_dgrad(G, out):
    dy, w, dx = G.rows_in("y", 1.0), G.weights(), G.rows_out("x", out)
    B.moe_grouped_dgrad(G.g(out), dy.data_ptr(), w.data_ptr(), dx.data_ptr(), _stream())
    _ok()
    got = G.untouched(dx, "x")
    for e, a, b in G.spans():
        de, we = dy[a:b, :G.d_out].double(), w[e].double()
        ref = de @ we
        tol = _sum_tol(G.d_out, de.abs() @ we.abs()) + _rounding(ref, out)
        _within(got[a:b], ref, tol * (1 + 1e-6), f"expert {e}")


def check_wgrad(G, out, accumulate=False):
    dy, x = G.rows_in("y", 1.0), G.rows_in("x", 1.0)
    n = G.E * G.d_out * G.d_in
    buf = torch.full((n + 64,), -77.0, device="cuda").to(T[out])
    if accumulate:
        buf[:n] = G.normal((n,), 3.0)
    old = buf[:n].clone().view(G.E, G.d_out, G.d_in)
    B.moe_grouped_wgrad(G.g(out, int(accumulate)), dy.data_ptr(), x.data_ptr(), buf.data_ptr(), _stream())
    _ok()
    assert bool((buf[n:] == -77.0).all())
    got = buf[:n].view(G.E, G.d_out, G.d_in)
    for e in range(G.E):
        a, b = G.off[e], G.off[e + 1]
        if a == b:
            assert torch.equal(got[e], old[e] if accumulate else torch.zeros_like(got[e]))
            continue
        de, xe = dy[a:b, :G.d_out].double(), x[a:b, :G.d_in].double()
        ref = de.T @ xe
        tol = _sum_tol(b - a, de.abs().T @ xe.abs()) + _rounding(ref, out)
        if accumulate:
            ref = ref + old[e].double()
            tol = tol + _rounding(ref, out)
        _within(got[e], ref, tol * (1 + 1e-6), f"expert {e}")


# lengths of none, one, around the 32-row boxes and the 256-row chunks; experts without rows first, last and
# between; sizes below a tile, at its edges and over it
CASES = [
    ([1], 8, 8, {}),
    ([0, 1, 0], 64, 8, dict(before=3, behind=2)),
    ([0, 0, 0], 64, 64, dict(before=1, behind=1)),
    ([1] * 8 + [0] * 24, 2048, 1024, {}),
    ([3, 0, 1, 2, 0, 0, 2], 72, 136, dict(behind=5, pad_x=8, pad_y=24)),
    ([7, 8, 9, 15, 16, 17], 264, 520, dict(before=1)),
    ([31, 32, 33, 63, 64, 65], 136, 248, dict(pad_x=16)),
    ([127, 128, 129], 200, 256, dict(pad_y=8)),
    ([255, 0, 256, 257], 320, 264, dict(before=130, behind=1)),
    ([300, 513, 1, 90], 1064, 712, {}),
    ([1500], 128, 384, {}),
    ([5] * 300, 96, 72, {}),
    ([2] * 512 + [0] * 511 + [9], 64, 40, {}),
    (([0] * 7 + [50] + [0, 3]) * 20, 328, 264, dict(behind=3)),
]


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f16", "f32")])
@pytest.mark.parametrize("counts,d_in,d_out,kw", CASES, ids=lambda v: str(v)[:24])
def test_gemm(counts, d_in, d_out, kw, dtype, out):
    check_gemm(Group(counts, d_in, d_out, dtype, **kw), out)


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f16", "f32")])
@pytest.mark.parametrize("counts,d_in,d_out,kw", CASES, ids=lambda v: str(v)[:24])
def test_dgrad(counts, d_in, d_out, kw, dtype, out):
    check_dgrad(Group(counts, d_in, d_out, dtype, **kw), out)


@pytest.mark.parametrize("dtype,out,acc", [("bf16", "bf16", False), ("f16", "f16", False), ("bf16", "f32", False),
                                           ("f16", "f32", False), ("bf16", "f32", True), ("f16", "f32", True)])
@pytest.mark.parametrize("counts,d_in,d_out,kw", CASES, ids=lambda v: str(v)[:24])
def test_wgrad(counts, d_in, d_out, kw, dtype, out, acc):
    check_wgrad(Group(counts, d_in, d_out, dtype, **kw), out, acc)


# few weight tiles and a long reduction: several CTA pairs share a tile (1 to 8 groups of 32 columns, one and two
# tiles, ends inside a k-step), beside the same sizes with a row or two, which go another way
LONG = [
    ([40], 4096, 520, dict(behind=3, pad_x=8, pad_y=8)),
    ([130, 0, 70], 2056, 264, dict(before=2)),
    ([256], 3080, 1032, {}),
    ([1, 300], 1544, 8, {}),
    ([17], 2048, 3336, {}),
    ([3], 4104, 24, {}),
    ([2, 0, 9, 1, 0, 4, 0, 0], 8200, 4104, dict(before=1, pad_x=8)),
]


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f16", "f32")])
@pytest.mark.parametrize("counts,d_in,d_out,kw", LONG, ids=lambda v: str(v)[:24])
def test_long_reductions_over_few_tiles(counts, d_in, d_out, kw, dtype, out):
    check_gemm(Group(counts, d_in, d_out, dtype, **kw), out)
    swapped = {**kw, "pad_x": kw.get("pad_y", 0), "pad_y": kw.get("pad_x", 0)}
    check_dgrad(Group(counts, d_out, d_in, dtype, **swapped), out)


@pytest.mark.parametrize("dtype,out,acc", [("bf16", "bf16", False), ("f16", "f32", False), ("bf16", "f32", True)])
@pytest.mark.parametrize("counts,d_in,d_out", [([2100], 64, 40), ([4099, 0], 264, 520), ([5, 0, 6001], 136, 248),
                                               ([2500, 2500], 512, 256)], ids=str)
def test_wgrad_of_many_rows_over_few_tiles(counts, d_in, d_out, dtype, out, acc):
    check_wgrad(Group(counts, d_in, d_out, dtype, before=1, behind=70), out, acc)


def _codes(G, shape):
    return torch.randint(-128, 128, shape, generator=G.gen, device="cuda", dtype=torch.int32).to(torch.int8)


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("counts,d_in,d_out,kw", [(c, max(16, d_in // 16 * 16), o, {**k, **({"pad_x": 16} if "pad_x" in k else {})})
                                                  for c, d_in, o, k in CASES + LONG], ids=lambda v: str(v)[:24])
def test_i8_gemm(counts, d_in, d_out, kw, out):
    G = Group(counts, d_in, d_out, "bf16", **kw)
    q = _codes(G, (G.rows, d_in + G.pad["x"]))
    w = _codes(G, (G.E, d_out, d_in))
    scale = torch.rand(G.rows, generator=G.gen, device="cuda") * 1e-3 + 1e-4
    ws = torch.rand((G.E, d_out), generator=G.gen, device="cuda") * 1e-3 + 1e-4
    y = G.rows_out("y", out)
    B.moe_i8_grouped_gemm(G.g(out, dtype="i8"), q.data_ptr(), scale.data_ptr(), w.data_ptr(), ws.data_ptr(),
                          y.data_ptr(), _stream())
    _ok()
    got = G.untouched(y, "y")
    for e, a, b in G.spans():
        ref = (q[a:b, :d_in].double() @ w[e].double().T) * scale[a:b, None].double() * ws[e].double()
        _within(got[a:b], ref, _rounding(ref, out) + ref.abs() * (4.5 * U24), f"expert {e}")


def test_i8_gemm_longest_sum_is_exact():
    """The largest int32 sum: every code -128 over the longest reduction allowed."""
    k = 131056
    G = Group([1, 2], k, 8, "bf16")
    q = torch.full((3, k), -128, dtype=torch.int8, device="cuda")
    w = torch.full((2, 8, k), -128, dtype=torch.int8, device="cuda")
    one, ws = torch.ones(3, device="cuda"), torch.ones((2, 8), device="cuda")
    y = G.rows_out("y", "f32")
    B.moe_i8_grouped_gemm(G.g("f32", dtype="i8"), q.data_ptr(), one.data_ptr(), w.data_ptr(), ws.data_ptr(),
                          y.data_ptr(), _stream())
    _ok()
    assert bool((y == float(np.float32(128 * 128 * k))).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("counts", [[40, 70, 3, 50], [1, 2, 1, 1], [300, 40, 290, 17]], ids=str)
def test_another_experts_nan_stays_there(counts, dtype):
    """One expert's rows (and weights) are NaN and infinities: no other expert's result changes."""
    G = Group(counts, 136, 264, dtype)
    x, dy, w = G.rows_in("x", 1.0), G.rows_in("y", 1.0), G.weights()

    def three(x, dy, w):
        y, dx = G.rows_out("y", dtype), G.rows_out("x", dtype)
        dw = torch.empty_like(w)
        B.moe_grouped_gemm(G.g(dtype), x.data_ptr(), w.data_ptr(), y.data_ptr(), _stream())
        B.moe_grouped_dgrad(G.g(dtype), dy.data_ptr(), w.data_ptr(), dx.data_ptr(), _stream())
        B.moe_grouped_wgrad(G.g(dtype), dy.data_ptr(), x.data_ptr(), dw.data_ptr(), _stream())
        _ok()
        return y, dx, dw

    y0, dx0, dw0 = three(x, dy, w)
    for bad in (1, 2):
        xb, db, wb = x.clone(), dy.clone(), w.clone()
        a, b = G.off[bad], G.off[bad + 1]
        xb[a:b], db[a:b], wb[bad] = float("nan"), float("inf"), float("nan")
        y1, dx1, dw1 = three(xb, db, wb)
        keep = torch.ones(G.rows, dtype=torch.bool, device="cuda")
        keep[a:b] = False
        assert torch.equal(y0[keep], y1[keep]) and torch.equal(dx0[keep], dx1[keep])
        others = [e for e in range(G.E) if e != bad]
        assert torch.equal(dw0[others], dw1[others])
        assert bool(y1[a:b].isnan().all()) and bool(dx1[a:b].isnan().all()) and bool(dw1[bad].isnan().all())


@pytest.mark.parametrize("table", [[0, 4, 3, 8], [-1, 2, 4, 8], [0, 2, 4, 9], [5, 2, 7, 8], [0, 0, 0, 1 << 30]],
                         ids=str)
def test_unsound_offsets_write_nothing(table):
    """A table that does not ascend within the rows: nothing is written, and the status says so once."""
    G = Group([2, 2, 4], 64, 64, "bf16")
    x, w = G.rows_in("x", 1.0), G.weights()
    G.offsets.copy_(torch.tensor(table, dtype=torch.int32))
    codes, ones = _codes(G, (8, 64)), torch.ones(8 * 64, device="cuda")
    for call in ("gemm", "dgrad", "wgrad", "i8"):
        out = torch.full((64 * 64 * 3,), -77.0, dtype=torch.bfloat16, device="cuda")
        if call == "i8":
            B.moe_i8_grouped_gemm(G.g("bf16", dtype="i8"), codes.data_ptr(), ones.data_ptr(), w.data_ptr(),
                                  ones.data_ptr(), out.data_ptr(), _stream())
        else:
            second = x if call == "wgrad" else w
            getattr(B, "moe_grouped_" + call)(G.g("bf16"), x.data_ptr(), second.data_ptr(), out.data_ptr(), _stream())
        assert B.moe_grouped_status() == B.MOE_ERR_DEVICE_FLAG
        assert B.moe_grouped_status() == B.MOE_OK
        assert bool((out == -77.0).all())


def test_wgrad_without_rows_writes_zeros():
    w = torch.full((3, 8, 16), 5.0, device="cuda")
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    g = B.moe_grouped_t(0, 3, 16, 8, B.MOE_DTYPE_BF16, B.MOE_DTYPE_F32, 1, off.data_ptr(), 16, 8)
    B.moe_grouped_wgrad(g, None, None, w.data_ptr(), _stream())
    _ok()
    assert bool((w == 5.0).all())
    g.accumulate = 0
    B.moe_grouped_wgrad(g, None, None, w.data_ptr(), _stream())
    _ok()
    assert bool((w == 0.0).all())


def test_host_memory_is_refused():
    G = Group([2, 2], 64, 64, "bf16")
    x, w, y = G.rows_in("x", 1.0), G.weights(), G.rows_out("y", "bf16")
    host = torch.empty(4096, dtype=torch.bfloat16)
    address = (host.data_ptr() + 15) // 16 * 16
    L = B.lib()
    for ptrs in ((address, w.data_ptr(), y.data_ptr()), (x.data_ptr(), address, y.data_ptr()),
                 (x.data_ptr(), w.data_ptr(), address)):
        assert L.moe_grouped_gemm(ctypes.byref(G.g("bf16")), *ptrs, None) == B.MOE_ERR_INVALID_ARG
    assert L.moe_swiglu(4, 64, 0, address, x.data_ptr(), 64, y.data_ptr(), 64, None) == B.MOE_ERR_INVALID_ARG
    _ok()


# ---------------------------------------------------------------- rows
ROWS = [(1, 8), (3, 72), (9, 1024), (5, 1032), (2, 8192), (3, 14336), (700, 264), (1, 65536)]


def _swiglu64(g, u):
    g, u = g.double(), u.double()
    return g * torch.sigmoid(g) * u


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,cols", ROWS)
def test_swiglu_and_its_gradient(rows, cols, dtype):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(rows + cols)
    gu = (torch.randn((rows, 2 * cols + 16), generator=gen, device="cuda") * 4).to(T[dtype])
    gu[0, :4] = torch.tensor([-100.0, 100.0, 0.0, -1.28], device="cuda").to(T[dtype])
    gu[0, 4:8] = torch.tensor([-60.0, 60.0, -20.0, 1e4], device="cuda").to(T[dtype])
    gate, up = gu[:, :cols], gu[:, cols:2 * cols]
    dh = torch.randn((rows, cols + 8), generator=gen, device="cuda").to(T[dtype])
    h = torch.full((rows, cols + 8), -77.0, device="cuda").to(T[dtype])
    p, st = gu.data_ptr(), 2 * cols + 16
    B.moe_swiglu(rows, cols, MOE[dtype], p, p + 2 * cols, st, h.data_ptr(), cols + 8, _stream())
    ref = _swiglu64(gate, up)
    _within(h[:, :cols], ref, _rounding(ref, dtype) + ref.abs() * (11 * U24), "h")
    assert bool((h[:, cols:] == -77.0).all())

    d = torch.full((rows, 2 * cols + 8), -77.0, device="cuda").to(T[dtype])
    B.moe_swiglu_grad(rows, cols, MOE[dtype], dh.data_ptr(), cols + 8, p, p + 2 * cols, st, d.data_ptr(),
                      d.data_ptr() + 2 * cols, 2 * cols + 8, _stream())
    g64 = gate.double().requires_grad_()
    u64 = up.double().requires_grad_()
    (g64 * torch.sigmoid(g64) * u64).backward(dh[:, :cols].double())
    dg, du, s = g64.grad, u64.grad, torch.sigmoid(g64.detach())
    # 1 - s is off by s's 9 half steps and its own, 1 + g (1 - s) by |g| times that, the product g (1 - s) and
    # itself (at most 1 + |g|); dh s u by 9 and 2 more
    slack = (dh[:, :cols].double() * u64.detach()).abs() * s * ((g64.detach().abs() * 12 + 1) + (9 + 4) * (1 + g64.detach().abs() * (1 - s))) * U24
    _within(d[:, :cols], dg, _rounding(dg, dtype) + slack, "dgate")
    _within(d[:, cols:2 * cols], du, _rounding(du, dtype) + du.abs() * (12 * U24), "dup")
    assert bool((d[:, 2 * cols:] == -77.0).all())
    # in place: the gradients over gate and up, h over up
    over = gu.clone()
    B.moe_swiglu_grad(rows, cols, MOE[dtype], dh.data_ptr(), cols + 8, over.data_ptr(), over.data_ptr() + 2 * cols,
                      st, over.data_ptr(), over.data_ptr() + 2 * cols, st, _stream())
    assert torch.equal(over[:, :2 * cols], d[:, :2 * cols])
    over = gu.clone()
    B.moe_swiglu(rows, cols, MOE[dtype], over.data_ptr(), over.data_ptr() + 2 * cols, st,
                 over.data_ptr() + 2 * cols, st, _stream())
    assert torch.equal(over[:, cols:2 * cols], h[:, :cols])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_swiglu_of_infinities_and_nan(dtype):
    """As the formula in fp32 has it: silu(inf) = inf, silu(-inf) = -inf * 0 = NaN, NaN stays NaN; the neighbours of
    such values are not touched."""
    inf, nan = float("inf"), float("nan")
    g = torch.tensor([inf, -inf, nan, 1.0, 0.0, 2.0, inf, -3.0], device="cuda").to(T[dtype])[None].contiguous()
    u = torch.tensor([2.0, 2.0, 2.0, inf, inf, nan, -1.0, 0.5], device="cuda").to(T[dtype])[None].contiguous()
    h = torch.empty_like(g)
    B.moe_swiglu(1, 8, MOE[dtype], g.data_ptr(), u.data_ptr(), 8, h.data_ptr(), 8, _stream())
    want = g.float() / (1 + torch.exp(-g.float())) * u.float()
    assert torch.equal(h.isnan(), want.isnan()) and torch.equal(h.isinf(), want.isinf())
    assert torch.equal(torch.sign(h[h.isinf()]), torch.sign(want[want.isinf()]).to(T[dtype]))
    ref = _swiglu64(g, u)[0, 7]
    _within(h[0, 7:], ref[None], _rounding(ref[None], dtype) + ref.abs() * (11 * U24), "h")


def test_swiglu_gradient_against_differences():
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    g, u, dh = (torch.randn((6, 64), generator=gen, device="cuda").half() for _ in range(3))
    dg, du = torch.empty_like(g), torch.empty_like(g)
    B.moe_swiglu_grad(6, 64, MOE["f16"], dh.data_ptr(), 64, g.data_ptr(), u.data_ptr(), 64, dg.data_ptr(),
                      du.data_ptr(), 64, _stream())
    step = 1e-5
    for got, plus, minus in ((dg, _swiglu64(g.double() + step, u), _swiglu64(g.double() - step, u)),
                             (du, _swiglu64(g, u.double() + step), _swiglu64(g, u.double() - step))):
        ref = dh.double() * (plus - minus) / (2 * step)
        # central differences: step^2 / 6 times the third derivative (below 1 for these) and 1e-16 / step
        _within(got, ref, _rounding(ref, "f16") + 1e-6, "difference")


def _check_codes(q, scale, v64, rel):
    """v64: the rows in 64 bits, known to the kernel within a relative error `rel`."""
    top = v64.abs().amax(1)
    assert bool(((scale.double() - top / 127).abs() <= top / 127 * (rel + 1.01 * U24)).all())
    # the quotient v / s is off by rel of it twice (v and s) and its own rounding
    quot = v64 / torch.where(top > 0, top / 127, 1.0)[:, None]
    off = (q.double() - quot).abs()
    assert bool((off <= 0.5 + 127 * (2 * rel + 3 * U24)).all())
    assert int(q.to(torch.int32).abs().max()) <= 127


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,cols", ROWS)
def test_i8_rows(rows, cols, dtype):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(rows * 3 + cols)
    x = torch.randn((rows, 2 * cols + 8), generator=gen, device="cuda").to(T[dtype])
    if rows > 2:
        x[1] = 0
        x[2, 5] = 1e-7 if dtype == "f16" else 1e-38
        x[2, :5] = 0
        x[2, 6:] = 0
    q = torch.full((rows, cols + 8), 99, dtype=torch.int8, device="cuda")
    scale = torch.full((rows + 1,), -77.0, device="cuda")
    p = x.data_ptr()
    B.moe_i8_quantize(rows, cols, MOE[dtype], p, 2 * cols + 8, q.data_ptr(), cols + 8, scale.data_ptr(), _stream())
    torch.cuda.synchronize()
    assert bool((q[:, cols:] == 99).all()) and scale[rows].item() == -77.0
    # the same formula in fp32 on the host, whose divisions round to nearest: exactly these codes
    v = x[:, :cols].float().cpu().numpy()
    s = np.abs(v).max(1) / np.float32(127)
    want = np.where(s[:, None] > 0, np.rint(v / np.where(s > 0, s, 1).astype(np.float32)[:, None]), 0)
    assert np.array_equal(scale[:rows].cpu().numpy(), s)
    assert np.array_equal(q[:, :cols].cpu().numpy(), np.clip(want, -127, 127).astype(np.int8))
    normal = [r for r in range(rows) if r not in (1, 2)] if rows > 2 else list(range(rows))
    _check_codes(q[normal, :cols], scale[:rows][normal], x[normal, :cols].double(), 0.0)
    # SwiGLU on the way (the rows of zeros and of one tiny value among them)
    B.moe_swiglu_i8(rows, cols, MOE[dtype], p, p + 2 * cols, 2 * cols + 8, q.data_ptr(), cols + 8, scale.data_ptr(),
                    _stream())
    torch.cuda.synchronize()
    assert bool((q[:, cols:] == 99).all()) and scale[rows].item() == -77.0
    v64 = _swiglu64(x[:, :cols], x[:, cols:2 * cols])
    _check_codes(q[normal, :cols], scale[:rows][normal], v64[normal], 11 * U24)
    if rows > 2:
        assert scale[1].item() == 0.0 and bool((q[1, :cols] == 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_i8_ties_go_to_even(dtype):
    """Quotients that lie exactly on a half, for scales of 1, of a large and of a tiny power of two, and quotients next
    to a half (a scale of 1/127 of a power of two: v 127 / 2^k rounds to either side)."""
    half = torch.arange(128, device="cuda", dtype=torch.float32) - 63.5          # exact in bf16 too
    for k in ([0, 8, -9] if dtype == "f16" else [0, 60, -60]):
        x = torch.cat([half, torch.tensor([127.0], device="cuda").expand(8)]) * 2.0 ** k
        x = x.to(T[dtype]).repeat(3, 1)
        q, s = torch.empty((3, 136), dtype=torch.int8, device="cuda"), torch.empty(3, device="cuda")
        B.moe_i8_quantize(3, 136, MOE[dtype], x.data_ptr(), 136, q.data_ptr(), 136, s.data_ptr(), _stream())
        assert bool((s == 2.0 ** k).all())
        assert torch.equal(q[1].float(), torch.round(x[1].float() / 2.0 ** k))
    v = torch.arange(1, 1025, device="cuda", dtype=torch.float32).to(T[dtype]).view(8, 128)
    v[:, 0] = 1024.0
    q, s = torch.empty((8, 128), dtype=torch.int8, device="cuda"), torch.empty(8, device="cuda")
    B.moe_i8_quantize(8, 128, MOE[dtype], v.data_ptr(), 128, q.data_ptr(), 128, s.data_ptr(), _stream())
    host = v.float().cpu().numpy()
    scale = np.abs(host).max(1) / np.float32(127)
    assert np.array_equal(q.cpu().numpy(), np.rint(host / scale[:, None]).astype(np.int8))


@pytest.mark.parametrize("cols", [64, 4096, 16384])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_i8_rows_that_are_not_finite_say_so(cols, bad):
    x = torch.randn((4, cols), device="cuda").to(torch.bfloat16)
    x[1, cols - 3] = bad
    q = torch.empty((4, cols), dtype=torch.int8, device="cuda")
    scale = torch.empty(4, device="cuda")
    B.moe_i8_quantize(4, cols, 0, x.data_ptr(), cols, q.data_ptr(), cols, scale.data_ptr(), _stream())
    assert scale[1].isnan() and bool((q[1] == 0).all())
    assert bool(scale[[0, 2, 3]].isfinite().all())
    w, ws = torch.ones((1, 8, cols), dtype=torch.int8, device="cuda"), torch.ones((1, 8), device="cuda")
    off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    y = torch.empty((4, 8), device="cuda")
    g = B.moe_grouped_t(4, 1, cols, 8, MOE["i8"], MOE["f32"], 0, off.data_ptr(), cols, 8)
    B.moe_i8_grouped_gemm(g, q.data_ptr(), scale.data_ptr(), w.data_ptr(), ws.data_ptr(), y.data_ptr(), _stream())
    _ok()
    assert bool(y[1].isnan().all()) and bool(y[[0, 2, 3]].isfinite().all())


# ------------------------------------------------- as a program uses them
def _route(sh, seed):
    """The layer's inputs, moe_forward's output and its routing tables."""
    inp = synth.make_inputs(sh, seed=seed)
    layer = D.DeviceLayer(inp)
    plan = B.moe_plan_create(layer.config(sh.T))
    x = D.upload_x(inp.x, "cuda")
    out = torch.empty((sh.T, sh.d), device="cuda")
    r = D.Routing(sh.T, sh.k, sh.E, "cuda")
    B.moe_forward(plan, layer.weights, x.data_ptr(), sh.T, sh.k, sh.wfmt, out.data_ptr(), r.struct, _stream())
    torch.cuda.synchronize()
    assert B.moe_get_device_status(plan) == B.MOE_OK
    B.moe_plan_destroy(plan)
    bits = lambda a: torch.from_numpy(a.view(np.int16)).cuda().view(torch.bfloat16)  # noqa: E731
    return bits(inp.x), bits(inp.gate), bits(inp.up), bits(inp.down), out, r


@pytest.mark.parametrize("T_", [1, 8, 200])
def test_the_layer_from_its_operators(T_):
    """Route, gather, gate and up in one product, SwiGLU, down, weighted sum: the layer that moe_forward computes
    in one call; then in 8 bits."""
    sh = synth.MoEShape("ops", T=T_, d=256, E=16, k=3, F=192)
    x, gate, up, down, want, r = _route(sh, seed=5)
    R, F, d, E = sh.T * sh.k, sh.F, sh.d, sh.E
    pair = r.slot_pair.long()
    token, weight = pair // sh.k, r.weights.reshape(-1)[pair]
    xp = x[token].contiguous()
    wgu = torch.cat([gate.view(E, F, d), up.view(E, F, d)], 1).contiguous()
    wd = down.view(E, d, F).contiguous()
    y1 = torch.empty((R, 2 * F), dtype=torch.bfloat16, device="cuda")
    h = torch.empty((R, F), dtype=torch.bfloat16, device="cuda")
    y2 = torch.empty((R, d), device="cuda")
    off = r.offsets.data_ptr()
    up_g = B.moe_grouped_t(R, E, d, 2 * F, 0, 0, 0, off, d, 2 * F)
    down_g = B.moe_grouped_t(R, E, F, d, 0, B.MOE_DTYPE_F32, 0, off, F, d)
    B.moe_grouped_gemm(up_g, xp.data_ptr(), wgu.data_ptr(), y1.data_ptr(), _stream())
    B.moe_swiglu(R, F, 0, y1.data_ptr(), y1.data_ptr() + 2 * F, 2 * F, h.data_ptr(), F, _stream())
    B.moe_grouped_gemm(down_g, h.data_ptr(), wd.data_ptr(), y2.data_ptr(), _stream())
    _ok()
    got = torch.zeros((sh.T, d), device="cuda").index_add_(0, token, y2 * weight[:, None])
    # h and its two factors are rounded to bf16 (half a step is 2^-9 each), independent over F = 192 terms;
    # moe_forward rounds h at most once: relative L2 below 3 * 2^-9
    assert ((got - want).norm() / want.norm()).item() < 3 * 2.0 ** -9

    q1, s1 = torch.empty((R, d), dtype=torch.int8, device="cuda"), torch.empty(R, device="cuda")
    q2, s2 = torch.empty((R, F), dtype=torch.int8, device="cuda"), torch.empty(R, device="cuda")

    def codes(w, rows, cols):
        q = torch.empty((rows, cols), dtype=torch.int8, device="cuda")
        s = torch.empty(rows, device="cuda")
        B.moe_i8_quantize(rows, cols, 0, w.data_ptr(), cols, q.data_ptr(), cols, s.data_ptr(), _stream())
        return q, s

    wgu8, wgu_s = codes(wgu, E * 2 * F, d)
    wd8, wd_s = codes(wd, E * d, F)
    up_g.dtype = down_g.dtype = B.MOE_DTYPE_I8
    B.moe_i8_quantize(R, d, 0, xp.data_ptr(), d, q1.data_ptr(), d, s1.data_ptr(), _stream())
    B.moe_i8_grouped_gemm(up_g, q1.data_ptr(), s1.data_ptr(), wgu8.data_ptr(), wgu_s.data_ptr(), y1.data_ptr(), _stream())
    B.moe_swiglu_i8(R, F, 0, y1.data_ptr(), y1.data_ptr() + 2 * F, 2 * F, q2.data_ptr(), F, s2.data_ptr(), _stream())
    B.moe_i8_grouped_gemm(down_g, q2.data_ptr(), s2.data_ptr(), wd8.data_ptr(), wd_s.data_ptr(), y2.data_ptr(), _stream())
    _ok()
    got8 = torch.zeros((sh.T, d), device="cuda").index_add_(0, token, y2 * weight[:, None])
    # a code is off by half a step of max / 127, uniform: rms max / (127 sqrt 12) = max / 440 over an rms of
    # at least max / 6 for these rows: below 1.4 % for each of the four roundings (and gate and up each enter
    # once), 2.8 % together when independent; twice that bounds the sample
    assert ((got8 - want).norm() / want.norm()).item() < 0.06


def test_a_training_step_of_the_experts():
    """Forward and backward of the experts' FFN through the operators, against autograd in 64 bits on the same
    rounded intermediates' formulas, with the weight gradients added up over two batches."""
    torch.manual_seed(3)
    counts, d, F = [20, 0, 133, 1, 47], 136, 200
    R, E = sum(counts), len(counts)
    off = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda")
    wgu = (torch.randn((E, 2 * F, d), device="cuda") * 0.1).half()
    wd = (torch.randn((E, d, F), device="cuda") * 0.1).half()
    dwgu, dwd = torch.zeros(wgu.shape, device="cuda"), torch.zeros(wd.shape, device="cuda")
    ref_dwgu, ref_dwd = torch.zeros(wgu.shape, dtype=torch.float64, device="cuda"), \
        torch.zeros(wd.shape, dtype=torch.float64, device="cuda")
    f16, f32 = B.MOE_DTYPE_F16, B.MOE_DTYPE_F32
    gu_g = B.moe_grouped_t(R, E, d, 2 * F, f16, f16, 0, off.data_ptr(), d, 2 * F)
    dn_g = B.moe_grouped_t(R, E, F, d, f16, f16, 0, off.data_ptr(), F, d)
    gu_w = B.moe_grouped_t(R, E, d, 2 * F, f16, f32, 1, off.data_ptr(), d, 2 * F)
    dn_w = B.moe_grouped_t(R, E, F, d, f16, f32, 1, off.data_ptr(), F, d)
    for batch in range(2):
        x, dy = torch.randn((R, d), device="cuda").half(), torch.randn((R, d), device="cuda").half()
        y1, h = torch.empty((R, 2 * F), device="cuda").half(), torch.empty((R, F), device="cuda").half()
        y, dh, dx = torch.empty_like(x), torch.empty_like(h), torch.empty_like(x)
        d1 = torch.empty_like(y1)
        s = _stream()
        B.moe_grouped_gemm(gu_g, x.data_ptr(), wgu.data_ptr(), y1.data_ptr(), s)
        B.moe_swiglu(R, F, f16, y1.data_ptr(), y1.data_ptr() + 2 * F, 2 * F, h.data_ptr(), F, s)
        B.moe_grouped_gemm(dn_g, h.data_ptr(), wd.data_ptr(), y.data_ptr(), s)
        B.moe_grouped_dgrad(dn_g, dy.data_ptr(), wd.data_ptr(), dh.data_ptr(), s)
        B.moe_grouped_wgrad(dn_w, dy.data_ptr(), h.data_ptr(), dwd.data_ptr(), s)
        B.moe_swiglu_grad(R, F, f16, dh.data_ptr(), F, y1.data_ptr(), y1.data_ptr() + 2 * F, 2 * F, d1.data_ptr(),
                          d1.data_ptr() + 2 * F, 2 * F, s)
        B.moe_grouped_dgrad(gu_g, d1.data_ptr(), wgu.data_ptr(), dx.data_ptr(), s)
        B.moe_grouped_wgrad(gu_w, d1.data_ptr(), x.data_ptr(), dwgu.data_ptr(), s)
        _ok()
        xr = x.double().requires_grad_()
        wr, vr = wgu.double().requires_grad_(), wd.double().requires_grad_()
        owner = torch.repeat_interleave(torch.arange(E, device="cuda"), off.diff().long())
        t = torch.einsum("rk,rnk->rn", xr, wr[owner])
        hr = t[:, :F] * torch.sigmoid(t[:, :F]) * t[:, F:]
        yr = torch.einsum("rk,rnk->rn", hr, vr[owner])
        yr.backward(dy.double())
        ref_dwgu += wr.grad
        ref_dwd += vr.grad
        # relative L2: y1, h, (dh, d1,) and the result rounded to fp16, 2^-11 at most each and averaged over the
        # sums: below 6 * 2^-11
        for got, ref in ((y, yr.detach()), (dx, xr.grad)):
            assert ((got.double() - ref).norm() / ref.norm()).item() < 6 * 2.0 ** -11
    for got, ref in ((dwgu, ref_dwgu), (dwd, ref_dwd)):
        assert ((got.double() - ref).norm() / ref.norm()).item() < 6 * 2.0 ** -11
    assert not dwgu[1].any() and not dwd[1].any()


def test_gradients_against_differences():
    """<dy, y(x + t v) - y(x - t v)> / 2t = <dx, v>, and the same for the weights: y is linear in both, so the
    difference quotient is exact but for the roundings of its two outputs."""
    G = Group([30, 0, 45, 5], 64, 72, "f16")
    w, x, dy = G.weights(), G.rows_in("x", 1.0), G.rows_in("y", 1.0)
    v, u = G.rows_in("x", 1.0), G.weights() * 20
    dx, dw = G.rows_out("x", "f32"), torch.empty(w.shape, device="cuda")
    B.moe_grouped_dgrad(G.g("f32"), dy.data_ptr(), w.data_ptr(), dx.data_ptr(), _stream())
    B.moe_grouped_wgrad(G.g("f32"), dy.data_ptr(), x.data_ptr(), dw.data_ptr(), _stream())

    def y(x, w):
        out = G.rows_out("y", "f32")
        B.moe_grouped_gemm(G.g("f32"), x.data_ptr(), w.data_ptr(), out.data_ptr(), _stream())
        return out.double()

    _ok()
    xp, xm = (x.float() + v.float()).half(), (x.float() - v.float()).half()
    lhs = (dy.double() * (y(xp, w) - y(xm, w))).sum()
    rhs = (dx.double() * (xp.double() - xm.double())).sum()
    scale = (dx.double() * (xp.double() - xm.double())).abs().sum()
    assert abs(lhs - rhs) <= scale * 64 * U24
    wp, wm = (w.float() + u.float()).half(), (w.float() - u.float()).half()
    lhs = (dy.double() * (y(x, wp) - y(x, wm))).sum()
    diff = wp.double() - wm.double()
    rhs, scale = (dw.double() * diff).sum(), (dw.double() * diff).abs().sum()
    assert abs(lhs - rhs) <= scale * 64 * U24


# ------------------------------------------------- streams, graphs, order
def test_calls_on_two_streams_at_once():
    """No state is shared: the same and other products running side by side give what they give alone."""
    Ga, Gb = Group([200, 30, 500], 512, 768, "bf16"), Group([1, 0, 6, 3], 1024, 512, "f16", seed=9)
    xa, wa, xb, wb = Ga.rows_in("x", 1.0), Ga.weights(), Gb.rows_in("x", 1.0), Gb.weights()
    ya, yb = Ga.rows_out("y", "bf16"), Gb.rows_out("y", "f16")
    B.moe_grouped_gemm(Ga.g("bf16"), xa.data_ptr(), wa.data_ptr(), ya.data_ptr(), _stream())
    B.moe_grouped_gemm(Gb.g("f16"), xb.data_ptr(), wb.data_ptr(), yb.data_ptr(), _stream())
    _ok()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for i in range(8):
        o1, o2 = Ga.rows_out("y", "bf16"), Gb.rows_out("y", "f16")
        outs.append((o1, o2))
    torch.cuda.synchronize()
    for o1, o2 in outs:
        B.moe_grouped_gemm(Ga.g("bf16"), xa.data_ptr(), wa.data_ptr(), o1.data_ptr(), s1.cuda_stream)
        B.moe_grouped_gemm(Gb.g("f16"), xb.data_ptr(), wb.data_ptr(), o2.data_ptr(), s2.cuda_stream)
    _ok()
    assert all(torch.equal(o1, ya) and torch.equal(o2, yb) for o1, o2 in outs)


def test_captured_calls_replay_with_new_offsets():
    """One graph holds all three products and the row operators; a replay reads the offsets and rows of that time."""
    G = Group([40, 10, 14], 128, 256, "bf16")
    x, dy, w = G.rows_in("x", 1.0), G.rows_in("y", 1.0), G.weights()
    y, dx, dw = G.rows_out("y", "bf16"), G.rows_out("x", "bf16"), torch.empty_like(w)
    h = torch.empty((64, 128), dtype=torch.bfloat16, device="cuda")
    q, s = torch.empty((64, 128), dtype=torch.int8, device="cuda"), torch.empty(64, device="cuda")

    def calls(st):
        B.moe_grouped_gemm(G.g("bf16"), x.data_ptr(), w.data_ptr(), y.data_ptr(), st)
        B.moe_swiglu(64, 128, 0, y.data_ptr(), y.data_ptr() + 256, 256, h.data_ptr(), 128, st)
        B.moe_i8_quantize(64, 128, 0, h.data_ptr(), 128, q.data_ptr(), 128, s.data_ptr(), st)
        B.moe_grouped_dgrad(G.g("bf16"), dy.data_ptr(), w.data_ptr(), dx.data_ptr(), st)
        B.moe_grouped_wgrad(G.g("bf16"), dy.data_ptr(), x.data_ptr(), dw.data_ptr(), st)

    calls(_stream())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls(_stream())
    for table in ([0, 0, 1, 64], [0, 64, 64, 64], [0, 20, 30, 64]):
        G.offsets.copy_(torch.tensor(table, dtype=torch.int32))
        x.copy_(torch.randn(x.shape, device="cuda"))
        outs = (y, h, q, s, dx, dw)
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        replayed = [o.clone() for o in outs]
        for o in outs:
            o.zero_()
        calls(_stream())
        _ok()
        assert all(torch.equal(a, b) for a, b in zip(replayed, outs))


def _chain(st, between=lambda: None):
    """Rounding, product, SwiGLU with rounding, product, gradient of SwiGLU, both gradients: every call reads what the
    one before wrote.  `between` runs after each."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(8)
    counts, d, F = [70, 0, 9, 121], 256, 192
    R, E = sum(counts), len(counts)
    off = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda")
    x = torch.randn((R, d), generator=gen, device="cuda").to(torch.bfloat16)
    w8 = torch.randint(-127, 128, (E, 2 * F, d), generator=gen, device="cuda", dtype=torch.int32).to(torch.int8)
    v8 = torch.randint(-127, 128, (E, d, F), generator=gen, device="cuda", dtype=torch.int32).to(torch.int8)
    w = (w8.float() / 1000).to(torch.bfloat16)
    ws, vs = torch.full((E, 2 * F), 1e-3, device="cuda"), torch.full((E, d), 1e-3, device="cuda")
    q, s = torch.empty((R, d), dtype=torch.int8, device="cuda"), torch.empty(R, device="cuda")
    h, hs = torch.empty((R, F), dtype=torch.int8, device="cuda"), torch.empty(R, device="cuda")
    y = torch.empty((R, 2 * F), dtype=torch.bfloat16, device="cuda")
    z, dx = torch.empty_like(x), torch.empty_like(x)
    dw = torch.empty(w.shape, device="cuda")
    up = B.moe_grouped_t(R, E, d, 2 * F, 3, 0, 0, off.data_ptr(), d, 2 * F)
    dn = B.moe_grouped_t(R, E, F, d, 3, 0, 0, off.data_ptr(), F, d)
    up16 = B.moe_grouped_t(R, E, d, 2 * F, 0, 0, 0, off.data_ptr(), d, 2 * F)
    up32 = B.moe_grouped_t(R, E, d, 2 * F, 0, 2, 0, off.data_ptr(), d, 2 * F)
    torch.cuda.synchronize()
    calls = [
        lambda: B.moe_i8_quantize(R, d, 0, x.data_ptr(), d, q.data_ptr(), d, s.data_ptr(), st),
        lambda: B.moe_i8_grouped_gemm(up, q.data_ptr(), s.data_ptr(), w8.data_ptr(), ws.data_ptr(), y.data_ptr(), st),
        lambda: B.moe_swiglu_i8(R, F, 0, y.data_ptr(), y.data_ptr() + 2 * F, 2 * F, h.data_ptr(), F, hs.data_ptr(), st),
        lambda: B.moe_i8_grouped_gemm(dn, h.data_ptr(), hs.data_ptr(), v8.data_ptr(), vs.data_ptr(), z.data_ptr(), st),
        lambda: B.moe_swiglu_grad(R, F, 0, z.data_ptr(), d, y.data_ptr(), y.data_ptr() + 2 * F, 2 * F, y.data_ptr(),
                                  y.data_ptr() + 2 * F, 2 * F, st),
        lambda: B.moe_grouped_dgrad(up16, y.data_ptr(), w.data_ptr(), dx.data_ptr(), st),
        lambda: B.moe_grouped_wgrad(up32, y.data_ptr(), x.data_ptr(), dw.data_ptr(), st),
        lambda: B.moe_swiglu(R, F, 0, dx.data_ptr(), dx.data_ptr() + 128, d, x.data_ptr(), d, st),
    ]

    def step():
        for c in calls:
            c()
            between()

    step.offsets = off                             # the descriptions hold its address alone
    return step, (x, q, s, h, hs, y, z, dx, dw)


def test_a_chain_of_calls_needs_no_synchronisation():
    """Kernels of the chain start while their predecessors still run: five rounds without a wait between any two calls
    give what rounds with one after every call give; the last call overwrites what the first of the next round reads."""
    step, outs = _chain(_stream(), torch.cuda.synchronize)
    for _ in range(5):
        step()
    _ok()
    want = [o.clone() for o in outs]
    for _ in range(6):
        step, outs = _chain(_stream())
        for _ in range(5):
            step()
        _ok()
        for a, b in zip(outs, want):
            assert torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b.float()))


def test_two_captured_graphs_at_once():
    """Two graphs of the chain, each with its own tensors, replayed side by side on two streams."""
    graphs, outs = [], []
    for _ in range(2):
        _chain(_stream())[0]()                      # a first call outside the capture
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            step, o = _chain(s.cuda_stream)
            start = [v.clone() for v in o]
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                step()
        graphs.append((graph, s, start, step))
        outs.append(o)
    torch.cuda.synchronize()
    for (_graph, _s, start, _step), o in zip(graphs, outs):
        for v, to in zip(start, o):
            to.copy_(v)
    torch.cuda.synchronize()
    for _ in range(3):
        for graph, s, _start, _step in graphs:
            with torch.cuda.stream(s):
                graph.replay()
    _ok()
    step, want = _chain(_stream())
    for _ in range(3):
        step()
    _ok()
    for o in outs:
        for a, b in zip(o, want):
            assert torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b.float()))


def test_captured_behind_copies_and_joined_streams():
    """A call captured behind a memset, a device copy, and two branches that another stream runs: it still waits for
    all of them."""
    G = Group([40, 10, 14], 128, 256, "bf16")
    src = [G.rows_in("x", 1.0) for _ in range(3)]
    x, w, y, z = G.rows_in("x", 1.0), G.weights(), G.rows_out("y", "bf16"), G.rows_out("y", "bf16")
    big = torch.randn((4096, 4096), device="cuda")
    side, main = torch.cuda.Stream(), torch.cuda.Stream()

    def gemm(a, out):
        B.moe_grouped_gemm(G.g("bf16"), a.data_ptr(), w.data_ptr(), out.data_ptr(), _stream())

    gemm(x, y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        y.zero_()
        x.copy_(src[0])
        gemm(x, y)                                  # behind a copy
        side.wait_stream(main)
        with torch.cuda.stream(side):
            slow = big.sin().cos().exp().sin()      # the branch that takes longer
            src[2].copy_(torch.where(slow.sum() > float("inf"), src[0], src[1]))
        x.copy_(src[0] + src[0])
        main.wait_stream(side)
        gemm(src[2], z)                             # behind both branches
        gemm(x, y)                                  # behind a kernel of its own kind
    for _ in range(3):
        src[0].normal_()
        src[1].normal_()
        src[2].zero_()
        graph.replay()
        torch.cuda.synchronize()
        got_y, got_z = y.clone(), z.clone()
        gemm(src[1], z)
        torch.cuda.synchronize()
        gemm(src[0] + src[0], y)
        _ok()
        assert torch.equal(got_z, z) and torch.equal(got_y, y)


@pytest.mark.parametrize("counts", [[30, 2, 70], [1, 1]], ids=str)
def test_pointers_on_any_16_byte_boundary(counts):
    """Every tensor 16 bytes past a 256-byte boundary."""
    G = Group(counts, 72, 136, "bf16")

    def off16(t):
        buf = torch.empty(t.numel() * t.element_size() + 16, dtype=torch.uint8, device="cuda")
        v = buf[16:].view(t.dtype).view(t.shape)
        v.copy_(t)
        return v

    x, w, dy = off16(G.rows_in("x", 1.0)), off16(G.weights()), off16(G.rows_in("y", 1.0))
    y, dx, dw = off16(G.rows_out("y", "bf16")), off16(G.rows_out("x", "bf16")), off16(torch.zeros_like(w))
    assert x.data_ptr() % 256 == 16
    B.moe_grouped_gemm(G.g("bf16"), x.data_ptr(), w.data_ptr(), y.data_ptr(), _stream())
    B.moe_grouped_dgrad(G.g("bf16"), dy.data_ptr(), w.data_ptr(), dx.data_ptr(), _stream())
    B.moe_grouped_wgrad(G.g("bf16"), dy.data_ptr(), x.data_ptr(), dw.data_ptr(), _stream())
    _ok()
    a, b, c = torch.empty_like(y), torch.empty_like(dx), torch.empty_like(dw)
    x, w, dy = x.clone(), w.clone(), dy.clone()
    B.moe_grouped_gemm(G.g("bf16"), x.data_ptr(), w.data_ptr(), a.data_ptr(), _stream())
    B.moe_grouped_dgrad(G.g("bf16"), dy.data_ptr(), w.data_ptr(), b.data_ptr(), _stream())
    B.moe_grouped_wgrad(G.g("bf16"), dy.data_ptr(), x.data_ptr(), c.data_ptr(), _stream())
    _ok()
    assert torch.equal(a, y) and torch.equal(b, dx) and torch.equal(c, dw)


@pytest.mark.parametrize("acc", [0, 1])
def test_the_same_call_gives_the_same_bits(acc):
    G = Group([700, 3, 0, 260], 264, 520, "bf16")
    x, dy, w = G.rows_in("x", 1.0), G.rows_in("y", 1.0), G.weights()
    got = []
    for _ in range(4):
        y, dx = G.rows_out("y", "bf16"), G.rows_out("x", "bf16")
        dw = torch.ones(w.shape, device="cuda")
        B.moe_grouped_gemm(G.g("bf16"), x.data_ptr(), w.data_ptr(), y.data_ptr(), _stream())
        B.moe_grouped_dgrad(G.g("bf16"), dy.data_ptr(), w.data_ptr(), dx.data_ptr(), _stream())
        B.moe_grouped_wgrad(G.g("f32", acc), dy.data_ptr(), x.data_ptr(), dw.data_ptr(), _stream())
        _ok()
        got.append((y, dx, dw))
    assert all(torch.equal(a, b) for o in got[1:] for a, b in zip(o, got[0]))


def test_rows_past_4_gi_bytes():
    """Rows whose elements lie past 2^32 bytes and 2^31 elements of their buffers: 64-bit offsets throughout."""
    rows, d_in, d_out, stride = 70000, 16, 16, 1 << 15
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB free")
    off = torch.tensor([0, 5, rows - 40, rows], dtype=torch.int32, device="cuda")
    x = torch.empty((rows, stride), dtype=torch.bfloat16, device="cuda")
    x[:, :d_in] = torch.randn((rows, d_in), device="cuda")
    y = torch.empty((rows, stride), dtype=torch.bfloat16, device="cuda")
    w = torch.randn((3, d_out, d_in), device="cuda").to(torch.bfloat16)
    g = B.moe_grouped_t(rows, 3, d_in, d_out, 0, 0, 0, off.data_ptr(), stride, stride)
    B.moe_grouped_gemm(g, x.data_ptr(), w.data_ptr(), y.data_ptr(), _stream())
    _ok()
    for e, a, b in ((0, 0, 5), (1, rows - 300, rows - 40), (2, rows - 40, rows)):
        xe, we = x[a:b, :d_in].double(), w[e].double()
        ref = xe @ we.T
        _within(y[a:b, :d_out], ref, _sum_tol(d_in, xe.abs() @ we.abs().T) + _rounding(ref, "bf16"), f"expert {e}")
    h = torch.empty((rows, 8), dtype=torch.bfloat16, device="cuda")
    B.moe_swiglu(rows, 8, 0, x.data_ptr(), x.data_ptr() + 16, stride, h.data_ptr(), 8, _stream())
    ref = _swiglu64(x[-50:, :8], x[-50:, 8:16])
    _within(h[-50:], ref, _rounding(ref, "bf16") + ref.abs() * (11 * U24), "h")
