"""SwiGLU where the gate's sigmoid is below the smallest normal number of fp32
while its products are not: bf16 has the range of fp32, so silu(-88) = -5.3e-37
is an ordinary number there, and silu(-150) times 1e30 is one, too.

Tolerances: as for other gates, 11 * 2^-24 relative for h and dup (the power of
two 4, its correction 2, g times it, b and one more product 1 each), and for
dgate the rounding of dh up and of 1 + gate more, 13 * 2^-24; half a step of the
result's type; and where the product is itself below 2^-126 up to four roundings
to multiples of 2^-149.
"""
import pytest
import torch

from mixture_experts_layer_43_b200 import binding as B

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f16": torch.float16}
MOE = {"bf16": B.MOE_DTYPE_BF16, "f16": B.MOE_DTYPE_F16}
U24 = 2.0 ** -24
GATES = [-86.5, -87.0, -87.5, -88.0, -88.5, -89.0, -90.0, -91.5, -92.0, -95.0, -100.0, -103.0, -104.0, -120.0, -150.0,
         -174.0, -176.0, -200.0, -260.0, -290.0, -298.0, -300.0, -302.0, -1000.0, -60000.0, 1.0, -1.0, 0.0, 90.0]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def _st():
    return torch.cuda.current_stream().cuda_stream


def _grid(dtype):
    """Every gate beside every factor, shuffled, so that vectors of 8 hold some of these gates, all and none."""
    factors = [1.0, -3.0, 1e-3, 2e4] + ([1e10, -1e25, 3e38, 1e-30] if dtype == "bf16" else [])
    g, u = torch.meshgrid(torch.tensor(GATES), torch.tensor(factors), indexing="ij")
    g, u = g.flatten(), u.flatten()
    gen = torch.Generator()
    gen.manual_seed(2)
    order = torch.cat([torch.arange(g.numel()), torch.randperm(g.numel(), generator=gen)])
    n = order.numel() // 8 * 8
    return g[order[:n]].to(T[dtype]).cuda()[None], u[order[:n]].to(T[dtype]).cuda()[None]


def _within(got, ref, rel, what):
    info = torch.finfo(got.dtype)
    tol = ref.abs() * (rel + info.eps / 2) + info.smallest_normal * info.eps / 2 + 4 * 2.0 ** -149
    over = got.isinf() & (ref.abs() >= info.max * (1 + info.eps / 4)) & (torch.sign(got).double() == torch.sign(ref))
    bad = ((got.double() - ref).abs() > tol) & ~over | got.isnan()
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} outside, first {got[bad][0].item()} for {ref[bad][0].item()}"


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_gates_far_below_zero(dtype):
    g, u = _grid(dtype)
    n = g.shape[1]
    h = torch.empty_like(g)
    B.moe_swiglu(1, n, MOE[dtype], g.data_ptr(), u.data_ptr(), n, h.data_ptr(), n, _st())
    torch.cuda.synchronize()
    _within(h, g.double() * torch.sigmoid(g.double()) * u.double(), 11 * U24, "h")
    if dtype == "bf16":
        at = (g == -88.0) & (u == 1.0)
        assert bool(at.any()) and bool((h[at] != 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("up", [1.0, -700.0])
def test_gradients_of_gates_far_below_zero(dtype, up):
    g, d = _grid(dtype)
    g, d = g[d.abs() < 1e30][None], d[d.abs() < 1e30][None]           # dh times up stays a number
    n = g.shape[1] // 8 * 8
    g, d = g[:, :n].contiguous(), d[:, :n].contiguous()
    u = torch.full_like(g, up)
    dg, du = torch.empty_like(g), torch.empty_like(g)
    B.moe_swiglu_grad(1, n, MOE[dtype], d.data_ptr(), n, g.data_ptr(), u.data_ptr(), n, dg.data_ptr(), du.data_ptr(), n,
                      _st())
    torch.cuda.synchronize()
    g64, u64, d64 = g.double(), u.double(), d.double()
    s = torch.sigmoid(g64)
    _within(du, d64 * g64 * s, 12 * U24, "dup")
    far = g64 < -80                                    # 1 - s is 1 there; the others have tests of their own
    _within(dg[far], (d64 * u64 * s * (1 + g64 * (1 - s)))[far], 13 * U24, "dgate")
    # in place
    over = torch.cat([g, u], 1)
    B.moe_swiglu_grad(1, n, MOE[dtype], d.data_ptr(), n, over.data_ptr(), over.data_ptr() + 2 * n, 2 * n, over.data_ptr(),
                      over.data_ptr() + 2 * n, 2 * n, _st())
    torch.cuda.synchronize()
    assert torch.equal(over[:, :n], dg) and torch.equal(over[:, n:], du)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("cols", [8, 264, 2048, 14336])
def test_codes_of_rows_of_such_gates(cols, dtype):
    """A row whose every gate is there has a scale and codes like any other."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(cols)
    g = (torch.rand((5, cols), generator=gen, device="cuda") * -6 - 87.5).to(T[dtype])
    u = (torch.rand((5, cols), generator=gen, device="cuda") * 2000 - 1000).to(T[dtype])
    g[3, ::3] = -400.0
    q, s = torch.empty((5, cols), dtype=torch.int8, device="cuda"), torch.empty(5, device="cuda")
    B.moe_swiglu_i8(5, cols, MOE[dtype], g.data_ptr(), u.data_ptr(), cols, q.data_ptr(), cols, s.data_ptr(), _st())
    torch.cuda.synchronize()
    v = g.double() * torch.sigmoid(g.double()) * u.double()
    top = v.abs().amax(1)
    # v and s are known to 11 * 2^-24 and to four multiples of 2^-149, s to its own rounding, too
    rel = 11 * U24 + 4 * 2.0 ** -149 / top
    assert bool((top > 0).all())
    assert bool(((s.double() - top / 127).abs() <= top / 127 * (rel + U24 * 1.01) + 2.0 ** -149).all())
    off = (q.double() - v / (top / 127)[:, None]).abs()
    slack = 127 * (2 * rel + 3 * U24 + 2.0 ** -149 * 127 / top)
    assert bool((off <= 0.5 + slack[:, None]).all()) and int(q.int().abs().max()) == 127
    assert bool((q[3, ::3] == 0).all())


def test_not_a_number_among_them():
    """-inf and NaN beside such gates: NaN as ever, and the neighbours keep their values."""
    inf, nan = float("inf"), float("nan")
    g = torch.tensor([[-inf, -90.0, nan, -88.0, -500.0, 2.0, -87.5, 0.0]], device="cuda").bfloat16()
    neg_nan = torch.tensor([[-64]], dtype=torch.int16, device="cuda").view(torch.bfloat16)       # 0xFFC0
    g = torch.cat([g, torch.cat([neg_nan, g[:, 1:]], 1)], 1)
    u = torch.ones_like(g)
    h, dg, du = torch.empty_like(g), torch.empty_like(g), torch.empty_like(g)
    B.moe_swiglu(1, 16, 0, g.data_ptr(), u.data_ptr(), 16, h.data_ptr(), 16, _st())
    B.moe_swiglu_grad(1, 16, 0, u.data_ptr(), 16, g.data_ptr(), u.data_ptr(), 16, dg.data_ptr(), du.data_ptr(), 16, _st())
    torch.cuda.synchronize()
    bad = g.isnan() | g.isinf()
    assert torch.equal(h.isnan(), bad) and torch.equal(du.isnan(), bad) and torch.equal(dg.isnan(), bad)
    ref = (g.double() * torch.sigmoid(g.double()))[~bad]
    _within(h[~bad], ref, 11 * U24, "h")
    _within(du[~bad], ref, 12 * U24, "dup")
