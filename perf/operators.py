"""The 8-bit activation operators as measured calls.

Four operators around a transformer block's projections whose activations and
weights are both held in 8 bits: ``quantize`` (one scale a token),
``addnorm`` (residual addition and root-mean-square norm into 8 bits),
``gate`` (gated SiLU into 8 bits) and ``gemm`` (the 8-bit product with token
and channel scales).  The 8-bit formats are those of the framework's weights:
8 is int8 with scale max/127, 3 is FP8 E4M3 with scale max/448.
"""
import math

import torch

own = False

Q8, E4M3 = 8, 3
TOP = {Q8: 127.0, E4M3: 448.0}
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-6


def listed():
    return [
        # one token's attention output on its way to the output projection
        {"name": "quantize m1", "op": "quantize", "M": 1, "K": 512, "dtype": "f32", "fmt": E4M3},
        # the same at the block benchmark's 4096 rows
        {"name": "quantize m4096", "op": "quantize", "M": 4096, "K": 512, "dtype": "f32", "fmt": Q8},
        # a golden batch of 5 x 16 rows before the qkvg or w1/w3 projection
        {"name": "addnorm m80", "op": "addnorm", "M": 80, "K": 512, "dtype": "bf16", "residual": True, "fmt": Q8},
        # odd sizes, the first norm of a model: no residual yet
        {"name": "addnorm m1001 k528", "op": "addnorm", "M": 1001, "K": 528, "dtype": "f16", "residual": False, "fmt": E4M3},
        # the largest batch of contexts the framework is measured at
        {"name": "addnorm m65536", "op": "addnorm", "M": 65536, "K": 512, "dtype": "f32", "residual": True, "fmt": E4M3},
        # between w1/w3 and w2 at 80 rows
        {"name": "gate m80", "op": "gate", "M": 80, "K": 2048, "dtype": "f32", "fmt": Q8},
        # the same at the largest batch, halves in 16 bits
        {"name": "gate m65536", "op": "gate", "M": 65536, "K": 2048, "dtype": "bf16", "fmt": E4M3},
        # one token through w1/w3: weight latency
        {"name": "gemm m1", "op": "gemm", "M": 1, "N": 4096, "K": 512, "dtype": "f32", "fmt": Q8, "bias": False},
        # 80 rows through w2, the long-K projection
        {"name": "gemm m80 w2", "op": "gemm", "M": 80, "N": 512, "K": 2048, "dtype": "f32", "fmt": E4M3, "bias": True},
        # w1/w3 at the block benchmark's 4096 rows, results in 32 bits as the weight-only path gives them
        {"name": "gemm m4096 w13", "op": "gemm", "M": 4096, "N": 4096, "K": 512, "dtype": "f32", "fmt": Q8, "bias": False},
        # ragged in every size, results in 16 bits
        {"name": "gemm m20001", "op": "gemm", "M": 20001, "N": 2003, "K": 1040, "dtype": "bf16", "fmt": Q8, "bias": True},
        # a wide model's projection, bound by the tensor cores
        {"name": "gemm 8192", "op": "gemm", "M": 8192, "N": 8192, "K": 8192, "dtype": "bf16", "fmt": E4M3, "bias": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "addnorm", "gate", "gemm", "gemm"])
    case = {"op": op, "dtype": rng.choice(["f32", "f16", "bf16"]), "fmt": rng.choice([Q8, E4M3])}
    if op == "gemm":
        K = 16 * _log(rng, 4, 512)
        N = _log(rng, 64, 8192)
        most = min(65536, (1 << 39) // (N * K), (1 << 28) // N)
        case.update(M=_log(rng, 1, most), N=N, K=K, bias=rng.random() < 0.5)
    else:
        K = 16 * _log(rng, 8, 512)
        case.update(M=_log(rng, 1, min(65536, (1 << 26) // K)), K=K)
        if op == "addnorm":
            case["residual"] = rng.random() < 0.7
    return case


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _codes(g, rows, K, fmt):
    """Codes as quantized normal rows have them (largest value at the end of the range)."""
    x = torch.randn(rows, K, generator=g, device="cuda")
    x *= TOP[fmt] / x.abs().amax(dim=1, keepdim=True)
    if fmt == Q8:
        return x.round().to(torch.int8)
    return x.to(torch.float8_e4m3fn).view(torch.uint8)


def prepare(case, seed):
    g, M, K, fmt = _gen(seed), case["M"], case["K"], case["fmt"]
    dt = DTYPES[case["dtype"]]
    s = {"op": case["op"], "fmt": fmt, "dtype": dt}
    if case["op"] == "gemm":
        N = case["N"]
        s["Xq"], s["Wq"] = _codes(g, M, K, fmt), _codes(g, N, K, fmt)
        s["xs"] = (0.5 + torch.rand(M, generator=g, device="cuda")) * (4.0 / TOP[fmt])
        s["ws"] = (0.5 + torch.rand(N, generator=g, device="cuda")) * (4.0 / TOP[fmt] / math.sqrt(K))
        s["bias"] = torch.randn(N, generator=g, device="cuda") if case["bias"] else None
        s["Y"] = torch.empty(M, N, dtype=dt, device="cuda")
        return s
    width = 2 * K if case["op"] == "gate" else K
    x = torch.randn(M, width, generator=g, device="cuda")
    # a few channels far above the others, as activations have them
    hot = torch.rand(width, generator=g, device="cuda") < 0.01
    x *= torch.where(hot, 8.0, 1.0)
    s["X"] = x.to(dt)
    if case["op"] == "addnorm":
        s["gain"] = 1.0 + 0.2 * torch.randn(K, generator=g, device="cuda")
        s["R"] = (2.0 * torch.randn(M, K, generator=g, device="cuda")).to(dt) if case["residual"] else None
        s["H"] = torch.empty(M, K, dtype=dt, device="cuda") if case["residual"] else None
    s["codes"] = torch.empty(M, K, dtype=torch.int8 if fmt == Q8 else torch.uint8, device="cuda")
    s["scales"] = torch.empty(M, dtype=torch.float32, device="cuda")
    if fmt == Q8:
        s["values"] = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    return s


def _quantized(y, fmt):
    """(values, scale) of the rows of y.  E4M3 codes are returned as FP8 values before
    the scale, int8 codes as their values in 16 bits."""
    scale = y.abs().amax(dim=1) / TOP[fmt]
    inv = torch.where(scale > 0, 1.0 / scale, torch.zeros_like(scale))
    t = y * inv[:, None]
    if fmt == Q8:
        return (t.round().clamp(-127, 127) * scale[:, None]).to(torch.bfloat16), scale
    return t.clamp(-448, 448).to(torch.float8_e4m3fn), scale


def _plain(s):
    fmt, dt = s["fmt"], s["dtype"]
    if s["op"] == "gemm":
        if fmt == Q8:
            x, w = s["Xq"].float(), s["Wq"].float()
        else:
            x, w = (s[k].view(torch.float8_e4m3fn).float() for k in ("Xq", "Wq"))
        y = (x @ w.t()) * s["xs"][:, None] * s["ws"][None, :]
        if s["bias"] is not None:
            y = y + s["bias"]
        return y.to(dt)
    x = s["X"].float()
    if s["op"] == "quantize":
        values, scale = _quantized(x, fmt)
        return {"values": values, "scales": scale}
    if s["op"] == "gate":
        a, b = x.chunk(2, dim=1)
        values, scale = _quantized(a / (1.0 + torch.exp(-a)) * b, fmt)
        return {"values": values, "scales": scale}
    h = x if s["R"] is None else x + s["R"].float()
    y = h / torch.sqrt(h.square().mean(dim=1, keepdim=True) + EPS) * s["gain"]
    values, scale = _quantized(y, fmt)
    out = {"values": values, "scales": scale}
    if s["R"] is not None:
        out["H"] = h.to(dt)
    return out


def _own(s):
    import int8_dequant_gemm_b200 as rtq

    fmt = s["fmt"]
    if s["op"] == "gemm":
        return rtq.qgemm_a8(fmt, s["Xq"], s["xs"], s["Wq"], s["ws"], bias=s["bias"], Y=s["Y"])
    out = {}
    if s["op"] == "quantize":
        codes, scales = rtq.quantize_a8(s["X"], fmt, codes=s["codes"], scales=s["scales"])
    elif s["op"] == "gate":
        codes, scales = rtq.gate_a8(s["X"], fmt, codes=s["codes"], scales=s["scales"])
    else:
        codes, scales, H = rtq.addnorm_a8(s["X"], s["gain"], fmt, residual=s["R"], eps=EPS, H=s["H"],
                                          codes=s["codes"], scales=s["scales"])
        if s["R"] is not None:
            out["H"] = H
    out["scales"] = scales
    if fmt == Q8:
        out["values"] = rtq.dequant_a8(fmt, codes, scales, out=s["values"])
    else:
        out["values"] = codes.view(torch.float8_e4m3fn)
    return out


def run(state):
    return _own(state) if own else _plain(state)


def exact(case, seed):
    s = prepare(case, seed)
    fmt = s["fmt"]
    if s["op"] == "gemm":
        wide = [(s[k] if fmt == Q8 else s[k].view(torch.float8_e4m3fn)).double() for k in ("Xq", "Wq")]
        y = torch.einsum("mk,nk->mn", *wide)
        y *= torch.outer(s["xs"].double(), s["ws"].double())
        return y if s["bias"] is None else y + s["bias"].double()
    x = s["X"].double()
    out = {}
    if s["op"] == "gate":
        F = case["K"]
        x = torch.sigmoid(x[:, :F]) * x[:, :F] * x[:, F:]
    elif s["op"] == "addnorm":
        if s["R"] is not None:
            x = x + s["R"].double()
            out["H"] = x
        x = x * torch.rsqrt((x * x).sum(1, keepdim=True) / case["K"] + EPS) * s["gain"].double()
    scale = x.abs().max(dim=1).values / TOP[fmt]
    code = x / scale[:, None]
    if fmt == Q8:
        out["values"] = torch.round(code) * scale[:, None]
    else:
        # the nearest of 8 steps a binade, the smallest binade from 2^-6 on
        step = torch.exp2(torch.floor(torch.log2(code.abs().clamp(min=2.0 ** -6))) - 3)
        out["values"] = torch.round(code / step) * step
    out["scales"] = scale
    return out


def work(case):
    M, K = case["M"], case["K"]
    es = SIZE[case["dtype"]]
    if case["op"] == "gemm":
        N = case["N"]
        return {"bytes": (M + N) * K + 4 * (M + N) + (4 * N if case["bias"] else 0) + M * N * es, "flops": 2 * M * N * K}
    held = M * K * (2 if case["fmt"] == Q8 else 1) + 4 * M  # the values as they come back, and the scales
    if case["op"] == "quantize":
        return {"bytes": M * K * es + held, "flops": 3 * M * K}
    if case["op"] == "gate":
        return {"bytes": 2 * M * K * es + held, "flops": 8 * M * K}
    streams = 3 if case["residual"] else 1  # x, the residual, and their sum
    return {"bytes": streams * M * K * es + 4 * K + held, "flops": 8 * M * K}
