"""The experts' operators, measured one pass at a time.

Rows of tokens are sorted by expert: rows offsets[e] .. offsets[e + 1] - 1
belong to expert e, whose weights are w[e] of shape [d_out, d_in].

  gemm         y[r] = w[e] x[r]
  dgrad        dx[r] = w[e]^T dy[r]
  wgrad        dw[e] = sum over e's rows of dy[r] x[r]^T
  i8_up        x quantised to 8 bits by token, then the product with weights
               held in 8 bits with a scale for each output channel
  i8_down      SwiGLU of gate and up, quantised by token, then the product
  swiglu       h = silu(gate) * up
  swiglu_grad  its gradients

`run` computes them in elementary torch operations in 32 bits, or, where `own`
is true, by the library's entry points.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _case(name, op, tokens, top_k, experts, d_in, d_out, dtype, out, skew):
    return {"name": name, "op": op, "tokens": tokens, "top_k": top_k, "experts": experts,
            "d_in": d_in, "d_out": d_out, "dtype": dtype, "out": out, "skew": skew}


def listed():
    return [
        # one token of the 35B-A3B-shaped layer: gate and up of its 8 experts, where latency counts
        _case("gemm_a3b_T1", "gemm", 1, 8, 256, 2048, 1024, "bf16", "bf16", 0.0),
        # a decode batch of the Mixtral-shaped layer: the down product, bound by the weights' bytes
        _case("gemm_mixtral_T8", "gemm", 8, 2, 8, 14336, 4096, "f16", "f16", 0.0),
        # a prompt through the DeepSeek-MoE-shaped layer: gate and up of 64 experts with Zipf loads
        _case("gemm_deepseek_T4096", "gemm", 4096, 6, 64, 2048, 2816, "bf16", "bf16", 1.1),
        # the gradient of that product's input
        _case("dgrad_deepseek_T4096", "dgrad", 4096, 6, 64, 2048, 2816, "bf16", "bf16", 1.1),
        # a small layer with odd sizes and few, ragged rows
        _case("dgrad_odd_T509", "dgrad", 509, 3, 13, 1064, 712, "f16", "f16", 0.7),
        # the gradient of the weights, added up in 32 bits as an optimiser wants it
        _case("wgrad_mixtral_T4096", "wgrad", 4096, 2, 8, 4096, 14336, "bf16", "f32", 0.0),
        # ... and of the small odd layer, rounded to the weights' own type
        _case("wgrad_odd_T509", "wgrad", 509, 3, 13, 1064, 712, "f16", "f16", 0.7),
        # a decode batch in 8 bits: gate and up of about 58 active experts
        _case("i8_up_a3b_T8", "i8_up", 8, 8, 256, 2048, 1024, "bf16", "bf16", 0.0),
        # a prompt in 8 bits: gate and up, then SwiGLU and down
        _case("i8_up_deepseek_T4096", "i8_up", 4096, 6, 64, 2048, 2816, "bf16", "bf16", 1.1),
        _case("i8_down_deepseek_T4096", "i8_down", 4096, 6, 64, 1408, 2048, "bf16", "bf16", 1.1),
        # between the two products of a prompt, and backwards
        _case("swiglu_deepseek_T4096", "swiglu", 4096, 6, 64, 1408, 1408, "bf16", "bf16", 1.1),
        _case("swiglu_grad_odd_T2047", "swiglu_grad", 2047, 3, 13, 1416, 1416, "f16", "f16", 0.7),
    ]


def draw(rng):
    op = rng.choice(["gemm", "gemm", "dgrad", "wgrad", "i8_up", "i8_down", "swiglu", "swiglu_grad"])

    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    experts = log_int(1, 256)
    top_k = rng.randint(1, min(8, experts))
    step = 16 if op.startswith("i8") else 8
    d_in = step * log_int(max(1, 64 // step), 4096 // step)
    # the weights of all experts stay below 0.8 G values
    d_out = 8 * log_int(8, max(8, min(14336, 800_000_000 // (experts * d_in)) // 8))
    if op.startswith("swiglu"):
        d_out = d_in
    tokens = log_int(1, max(1, min(8192, 900_000_000_000 // (2 * top_k * d_in * d_out))))
    dtype = rng.choice(["bf16", "bf16", "f16"])
    out = dtype
    if op in ("gemm", "dgrad", "wgrad") and rng.random() < 0.2:
        out = "f32"
    case = _case("", op, tokens, top_k, experts, d_in, d_out, dtype, out, rng.choice([0.0, 0.7, 1.1]))
    del case["name"]
    return case


def _offsets(case, g):
    """Row offsets by expert of `tokens` tokens that choose top_k different experts each, the
    experts' popularity falling as a power of their rank."""
    e, t, k = case["experts"], case["tokens"], case["top_k"]
    logit = -case["skew"] * torch.log(torch.arange(1, e + 1, device="cuda", dtype=torch.float32))
    u = torch.rand((t, e), generator=g, device="cuda").clamp_(1e-20, 1.0)
    chosen = (logit - torch.log(-torch.log(u) + 1e-20)).topk(k, dim=1).indices.reshape(-1)
    offsets = torch.zeros(e + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.bincount(chosen, minlength=e).cumsum(0)
    return offsets


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    r, e = case["tokens"] * case["top_k"], case["experts"]
    i, o, t = case["d_in"], case["d_out"], _TYPES[case["dtype"]]

    def normal(shape, scale):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(scale).to(t)

    s = {"case": case, "offsets": _offsets(case, g)}
    s["ends"] = s["offsets"].tolist()
    op = case["op"]
    if op in ("gemm", "wgrad", "i8_up"):
        s["x"] = normal((r, i), 1.0)
    if op in ("dgrad", "wgrad"):
        s["dy"] = normal((r, o), 0.05)
    if op in ("gemm", "dgrad"):
        s["w"] = torch.empty((e, o, i), dtype=t, device="cuda")
        for k in range(e):
            s["w"][k] = normal((o, i), 0.02)
    if op in ("i8_up", "i8_down"):
        # weights in 8 bits, as they are kept: codes, and a scale for each output channel
        s["wq"] = torch.empty((e, o, i), dtype=torch.int8, device="cuda")
        s["ws"] = torch.empty((e, o), dtype=torch.float32, device="cuda")
        for k in range(e):
            w = torch.randn((o, i), generator=g, device="cuda") * 0.02
            s["ws"][k] = w.abs().amax(1) / 127
            s["wq"][k] = torch.round(w / s["ws"][k][:, None]).to(torch.int8)
    if op in ("i8_down", "swiglu", "swiglu_grad"):
        # the product of gate and up side by side, as one product of both leaves them
        s["gu"] = normal((r, 2 * i), 1.0)
    if op == "swiglu_grad":
        s["dh"] = normal((r, i), 0.05)
    return s


def _quantised(v):
    """Codes (as 32-bit values) and scales of the rows of v."""
    scale = v.abs().amax(1, keepdim=True) / 127
    return torch.where(scale > 0, torch.round(v / scale), 0.0).clamp(-127, 127), scale


def _plain_swiglu(gu, i):
    gate, up = gu[:, :i].float(), gu[:, i:].float()
    return gate / (1 + torch.exp(-gate)) * up


def _plain(s):
    case, ends = s["case"], s["ends"]
    op, i, o, t = case["op"], case["d_in"], case["d_out"], _TYPES[case["out"]]
    r, e = ends[-1], case["experts"]
    spans = [(k, a, b) for k, (a, b) in enumerate(zip(ends[:-1], ends[1:])) if b > a]
    if op == "gemm":
        y = torch.empty((r, o), dtype=t, device="cuda")
        for k, a, b in spans:
            y[a:b] = s["x"][a:b].float() @ s["w"][k].float().T
        return {"y": y}
    if op == "dgrad":
        dx = torch.empty((r, i), dtype=t, device="cuda")
        for k, a, b in spans:
            dx[a:b] = s["dy"][a:b].float() @ s["w"][k].float()
        return {"dx": dx}
    if op == "wgrad":
        dw = torch.zeros((e, o, i), dtype=t, device="cuda")
        for k, a, b in spans:
            dw[k] = s["dy"][a:b].float().T @ s["x"][a:b].float()
        return {"dw": dw}
    if op in ("i8_up", "i8_down"):
        q, scale = _quantised(s["x"].float() if op == "i8_up" else _plain_swiglu(s["gu"], i))
        y = torch.empty((r, o), dtype=t, device="cuda")
        for k, a, b in spans:
            y[a:b] = (q[a:b] @ s["wq"][k].float().T) * scale[a:b] * s["ws"][k]
        return {"y": y}
    if op == "swiglu":
        return {"h": _plain_swiglu(s["gu"], i).to(t)}
    gate, up, dh = s["gu"][:, :i].float(), s["gu"][:, i:].float(), s["dh"].float()
    sig = 1 / (1 + torch.exp(-gate))
    return {"dgu": torch.cat([dh * up * sig * (1 + gate * (1 - sig)), dh * gate * sig], 1).to(t)}


def _own(s):
    from mixture_experts_layer_43_b200 import binding as B

    case, stream = s["case"], torch.cuda.current_stream().cuda_stream
    op, i, o, e = case["op"], case["d_in"], case["d_out"], case["experts"]
    t, r = _TYPES[case["out"]], s["ends"][-1]
    types = {"bf16": B.MOE_DTYPE_BF16, "f16": B.MOE_DTYPE_F16, "f32": B.MOE_DTYPE_F32}
    dtype, out = types[case["dtype"]], types[case["out"]]
    if op == "swiglu":
        h = torch.empty((r, i), dtype=t, device="cuda")
        gu = s["gu"].data_ptr()
        B.moe_swiglu(r, i, dtype, gu, gu + 2 * i, 2 * i, h.data_ptr(), i, stream)
        return {"h": h}
    if op == "swiglu_grad":
        dgu = torch.empty((r, 2 * i), dtype=t, device="cuda")
        gu, d = s["gu"].data_ptr(), dgu.data_ptr()
        B.moe_swiglu_grad(r, i, dtype, s["dh"].data_ptr(), i, gu, gu + 2 * i, 2 * i, d, d + 2 * i, 2 * i, stream)
        return {"dgu": dgu}
    i8 = op in ("i8_up", "i8_down")
    g = B.moe_grouped_t(r, e, i, o, B.MOE_DTYPE_I8 if i8 else dtype, out, 0, s["offsets"].data_ptr(), i, o)
    if op == "gemm":
        y = torch.empty((r, o), dtype=t, device="cuda")
        B.moe_grouped_gemm(g, s["x"].data_ptr(), s["w"].data_ptr(), y.data_ptr(), stream)
        return {"y": y}
    if op == "dgrad":
        dx = torch.empty((r, i), dtype=t, device="cuda")
        B.moe_grouped_dgrad(g, s["dy"].data_ptr(), s["w"].data_ptr(), dx.data_ptr(), stream)
        return {"dx": dx}
    if op == "wgrad":
        dw = torch.empty((e, o, i), dtype=t, device="cuda")
        B.moe_grouped_wgrad(g, s["dy"].data_ptr(), s["x"].data_ptr(), dw.data_ptr(), stream)
        return {"dw": dw}
    q = torch.empty((r, i), dtype=torch.int8, device="cuda")
    scale = torch.empty(r, dtype=torch.float32, device="cuda")
    if op == "i8_up":
        B.moe_i8_quantize(r, i, dtype, s["x"].data_ptr(), i, q.data_ptr(), i, scale.data_ptr(), stream)
    else:
        gu = s["gu"].data_ptr()
        B.moe_swiglu_i8(r, i, dtype, gu, gu + 2 * i, 2 * i, q.data_ptr(), i, scale.data_ptr(), stream)
    y = torch.empty((r, o), dtype=t, device="cuda")
    B.moe_i8_grouped_gemm(g, q.data_ptr(), scale.data_ptr(), s["wq"].data_ptr(), s["ws"].data_ptr(),
                          y.data_ptr(), stream)
    return {"y": y}


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    r, e, i, o = case["tokens"] * case["top_k"], case["experts"], case["d_in"], case["d_out"]
    b, bo = (4 if case[k] == "f32" else 2 for k in ("dtype", "out"))
    # experts that the tokens are expected to reach: each expert is missed by all rows with
    # probability (1 - p)^rows
    p = [(k + 1.0) ** -case["skew"] for k in range(e)]
    reached = min(r, e, sum(1 - (1 - v / sum(p)) ** r for v in p))
    if case["top_k"] == e or case["tokens"] == 1:
        reached = min(r, e)
    op, flops = case["op"], 2.0 * r * i * o
    if op == "gemm":
        moved = r * i * b + reached * o * i * b + r * o * bo
    elif op == "dgrad":
        moved = r * o * b + reached * o * i * b + r * i * bo
    elif op == "wgrad":
        moved = r * (i + o) * b + e * o * i * bo
    elif op == "i8_up":
        moved = r * i * b + reached * o * (i + 4) + r * o * bo
    elif op == "i8_down":
        moved = 2 * r * i * b + reached * o * (i + 4) + r * o * bo
    elif op == "swiglu":
        moved, flops = 2 * r * i * b + r * i * bo, 5.0 * r * i
    else:
        moved, flops = 3 * r * i * b + 2 * r * i * bo, 12.0 * r * i
    return {"bytes": float(moved + 4 * (e + 1)), "flops": flops}


def exact(case, seed):
    s = prepare(case, seed)
    op, i = case["op"], case["d_in"]
    owner = torch.repeat_interleave(torch.arange(case["experts"], device="cuda"),
                                    s["offsets"].diff().long())
    if op in ("i8_down", "swiglu", "swiglu_grad"):
        gate, up = s["gu"].double().split(i, dim=1)
        silu = gate * torch.sigmoid(gate)
    if op == "swiglu":
        return {"h": silu * up}
    if op == "swiglu_grad":
        sig, dh = torch.sigmoid(gate), s["dh"].double()
        return {"dgu": torch.cat([dh * up * (sig + silu * (1 - sig)), dh * silu], 1)}
    if op == "wgrad":
        dw = torch.zeros((case["experts"], case["d_out"], i), dtype=torch.float64, device="cuda")
        for k in owner.unique().tolist():
            rows = (owner == k).nonzero()[:, 0]
            dw[k] = torch.einsum("rn,rk->nk", s["dy"][rows].double(), s["x"][rows].double())
        return {"dw": dw}
    if op == "i8_up":
        left = s["x"].double()
    elif op == "i8_down":
        left = silu * up
    else:
        left = s["x" if op == "gemm" else "dy"].double()
    if op in ("i8_up", "i8_down"):
        scale = left.abs().max(dim=1).values / 127
        left = torch.round(left / scale[:, None]).nan_to_num(0.0)
        weights = s["wq"]
    else:
        weights = s["w"]
    wide = case["d_in" if op == "dgrad" else "d_out"]
    out = torch.zeros((left.shape[0], wide), dtype=torch.float64, device="cuda")
    for k in owner.unique().tolist():
        rows = (owner == k).nonzero()[:, 0]
        form = "rn,nk->rk" if op == "dgrad" else "rk,nk->rn"
        out[rows] = torch.einsum(form, left[rows], weights[k].double())
        if op in ("i8_up", "i8_down"):
            out[rows] *= scale[rows][:, None] * s["ws"][k].double()
    return {"dx" if op == "dgrad" else "y": out}
