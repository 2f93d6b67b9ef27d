"""Calls that follow one another without a wait, through the product of few
rows: a kernel of the experts' operators may be resident while the one before
it still writes what it will read."""
import glob
import os
import re

import pytest
import torch

from mixture_experts_layer_43_b200 import binding as B
from mixture_experts_layer_43_b200 import build as build_mod


def _code(path):
    """A source file without its comments."""
    text = open(path).read()
    return re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", text, flags=re.S))


def test_chained_kernels_load_coherently():
    """ld.global.nc (and __ldg, and what a compiler makes of __restrict__) is for data that nobody writes for as long
    as the kernel lives.  A kernel launched as a programmatic dependent is alive while its predecessor writes: no source
    of such kernels, nor a header it takes, uses that path."""
    chained = [p for p in glob.glob(os.path.join(build_mod.CSRC, "*.cu")) if "launch_chained" in _code(p)]
    assert {os.path.basename(p) for p in chained} >= {"grouped.cu", "rows.cu"}
    seen, todo = set(), list(chained)
    while todo:
        p = todo.pop()
        if p in seen:
            continue
        seen.add(p)
        todo += [q for q in (os.path.join(build_mod.CSRC, n) for n in re.findall(r'#include "([^"]+)"', _code(p)))
                 if os.path.exists(q)]
    assert os.path.join(build_mod.CSRC, "grouped_small.cuh") in seen
    for p in sorted(seen):
        found = re.findall(r"__ldg|ld\.global\.nc|\.nc\.|__restrict__|__ldcv_nc", _code(p))
        assert not found, f"{os.path.basename(p)}: {found}"


ROUNDS = 24


def _few_rows_chain(dtype, st, between=lambda: None, run=lambda rounds: rounds()):
    """Rounds in which one buffer of x, one of its codes, one of the weights and one of their codes are written anew by
    row operators (from three sources in turn) and read by products of few rows; every round's products are kept.
    `run` is handed the rounds and may run them in its own way."""
    counts, d, o = [1, 0, 2, 1, 0, 0, 1, 1], 512, 256            # 6 rows, at most 6 tiles: the few-row kernel
    R, E = sum(counts), len(counts)
    t = {"bf16": torch.bfloat16, "f16": torch.float16}[dtype]
    code = {"bf16": B.MOE_DTYPE_BF16, "f16": B.MOE_DTYPE_F16}[dtype]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(21)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda").to(t)

    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[1:] = torch.tensor(counts, device="cuda").cumsum(0)
    xs = [(normal(R, d), normal(R, d)) for _ in range(3)]
    ws = [(normal(E * o, d), normal(E * o, d)) for _ in range(3)]
    x, w = torch.empty((R, d), dtype=t, device="cuda"), torch.empty((E * o, d), dtype=t, device="cuda")
    xq, wq = torch.empty((R, d), dtype=torch.int8, device="cuda"), torch.empty((E * o, d), dtype=torch.int8, device="cuda")
    x_s, w_s = torch.empty(R, device="cuda"), torch.empty(E * o, device="cuda")
    y = torch.zeros((ROUNDS, R, o), dtype=t, device="cuda")
    y32, y8 = torch.zeros((ROUNDS, R, o), device="cuda"), torch.zeros((ROUNDS, R, o), device="cuda")

    def g(dt, out):
        return B.moe_grouped_t(R, E, d, o, dt, out, 0, off.data_ptr(), d, o)

    torch.cuda.synchronize()

    def rounds():
        for i in range(ROUNDS):
            (xg, xu), (wg, wu) = xs[i % 3], ws[i // 2 % 3]
            calls = [
                lambda: B.moe_swiglu(R, d, code, xg.data_ptr(), xu.data_ptr(), d, x.data_ptr(), d, st),
                lambda: B.moe_grouped_gemm(g(code, code), x.data_ptr(), w.data_ptr(), y[i].data_ptr(), st),
                lambda: B.moe_swiglu(E * o, d, code, wg.data_ptr(), wu.data_ptr(), d, w.data_ptr(), d, st),
                lambda: B.moe_grouped_gemm(g(code, B.MOE_DTYPE_F32), x.data_ptr(), w.data_ptr(), y32[i].data_ptr(), st),
                lambda: B.moe_i8_quantize(E * o, d, code, w.data_ptr(), d, wq.data_ptr(), d, w_s.data_ptr(), st),
                lambda: B.moe_swiglu_i8(R, d, code, xu.data_ptr(), xg.data_ptr(), d, xq.data_ptr(), d, x_s.data_ptr(), st),
                lambda: B.moe_i8_grouped_gemm(g(B.MOE_DTYPE_I8, B.MOE_DTYPE_F32), xq.data_ptr(), x_s.data_ptr(),
                                              wq.data_ptr(), w_s.data_ptr(), y8[i].data_ptr(), st),
            ]
            if i == 0:
                calls.insert(0, calls[2])                     # the first product's weights
            for c in calls:
                c()
                between()

    run(rounds)
    torch.cuda.synchronize()
    assert B.moe_grouped_status() == B.MOE_OK
    return y, y32, y8


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_products_of_few_rows_read_what_was_just_written(dtype):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    st = torch.cuda.current_stream().cuda_stream
    want = _few_rows_chain(dtype, st, torch.cuda.synchronize)
    assert all(bool(v.isfinite().all()) and bool((v[1:] != v[:-1]).any(-1).any(-1).all()) for v in want)
    for _ in range(4):
        for got, ref in zip(_few_rows_chain(dtype, st), want):
            assert torch.equal(got, ref)


@pytest.mark.gpu
def test_a_captured_chain_of_few_rows():
    """The same rounds as one graph, replayed three times with nothing between."""
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    want = _few_rows_chain("bf16", torch.cuda.current_stream().cuda_stream, torch.cuda.synchronize)
    side = torch.cuda.Stream()

    def captured(rounds):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            rounds()
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()

    for got, ref in zip(_few_rows_chain("bf16", side.cuda_stream, run=captured), want):
        assert torch.equal(got, ref)


@pytest.mark.gpu
def test_chains_of_few_rows_on_two_streams():
    """Two chains side by side, each with its own tensors, issued from one thread."""
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    st = torch.cuda.current_stream().cuda_stream
    want = {d: _few_rows_chain(d, st, torch.cuda.synchronize) for d in ("bf16", "f16")}
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    got = {}

    def beside(rounds):
        got["f16"] = _few_rows_chain("f16", b.cuda_stream, run=lambda other: (rounds(), other()))

    got["bf16"] = _few_rows_chain("bf16", a.cuda_stream, run=beside)
    for d in want:
        for x, ref in zip(got[d], want[d]):
            assert torch.equal(x, ref)
