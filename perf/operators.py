"""Cases that time the operators of the 8-bit linear layer, in plain form or with the library's kernels.

The operators (rows are tokens, columns are channels):
  norm       h = x + r, y = h * rstd * w, and y's rows in 8 bits with one scale each
  norm_grad  its backward pass: dx (with the residual's gradient added) and dw,
             the norm's input kept in 16 bits or as an 8-bit checkpoint
  rows       an 8-bit checkpoint of an activation, written and read back
  grad       D = A . diag(s) . Q with Q an 8-bit tensor whose rows carry a scale:
             a linear layer's weight gradient from the checkpoint of its input
             (A is dY transposed), or its input gradient from 8-bit weights
  scaled     the int8 matrix product with a scale for each token and channel
Codes are returned as the values they stand for, in the activations' type.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-5
WORKSPACE = 96 << 20  # bytes a program keeps for all of its calls


def listed():
    return [
        # one token through a wide norm: the latency of a decoding step
        {"name": "norm_1x8192", "op": "norm", "M": 1, "N": 8192, "dtype": "bf16", "residual": True, "pad": 0},
        # a long prompt's residual stream
        {"name": "norm_8192x8192", "op": "norm", "M": 8192, "N": 8192, "dtype": "bf16", "residual": True, "pad": 0},
        # a training step's backward pass over the stored residual stream
        {"name": "norm_grad_8192x4096", "op": "norm_grad", "M": 8192, "N": 4096, "dtype": "bf16", "x8": False,
         "residual": True, "pad": 0},
        # a short ragged batch, its input kept in 8 bits
        {"name": "norm_grad_777x1990_x8", "op": "norm_grad", "M": 777, "N": 1990, "dtype": "f16", "x8": True,
         "residual": False, "pad": 6},
        # a long prompt's hidden layer, whose rows are written to a checkpoint and read back
        {"name": "rows_8192x8192", "op": "rows", "M": 8192, "N": 8192, "dtype": "bf16", "pad": 0},
        # a short ragged batch of odd rows
        {"name": "rows_333x2047", "op": "rows", "M": 333, "N": 2047, "dtype": "f16", "pad": 3},
        # the weight gradient of a square layer over a batch of 8192 tokens
        {"name": "grad_w_8192", "op": "grad", "M": 8192, "N": 8192, "K": 8192, "dtype": "bf16", "dtypeD": "bf16",
         "layoutA": "mn_contig", "add": False, "pad": 0},
        # the input gradient of a ragged batch, from the 8-bit weights
        {"name": "grad_x_1000x2048x4000", "op": "grad", "M": 1000, "N": 2048, "K": 4000, "dtype": "f16",
         "dtypeD": "f16", "layoutA": "k_contig", "add": False, "pad": 0},
        # one token's product: bound by reading the weights
        {"name": "scaled_1x8192x8192", "op": "scaled", "M": 1, "N": 8192, "K": 8192, "dtypeD": "bf16",
         "layoutB": "k_contig", "bias": False, "pad": 0},
        # a decoding batch over a rectangular layer
        {"name": "scaled_24x4096x16384", "op": "scaled", "M": 24, "N": 4096, "K": 16384, "dtypeD": "bf16",
         "layoutB": "k_contig", "bias": False, "pad": 0},
        # a ragged prompt with a bias
        {"name": "scaled_500x4096x4096", "op": "scaled", "M": 500, "N": 4096, "K": 4096, "dtypeD": "f16",
         "layoutB": "k_contig", "bias": True, "pad": 0},
        # the large product of training and of long prompts
        {"name": "scaled_8192", "op": "scaled", "M": 8192, "N": 8192, "K": 8192, "dtypeD": "bf16",
         "layoutB": "k_contig", "bias": False, "pad": 0},
    ]


def _size(rng, low, high, odd):
    """A size spread over its logarithm; a multiple of 64 (the usual widths of layers) or any."""
    n = math.exp(rng.uniform(math.log(low), math.log(high)))
    return max(low, min(high, int(n) if odd else 64 * max(1, round(n / 64))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "rows", "grad", "scaled", "scaled"])
    odd = rng.random() < 0.3
    pad = rng.randrange(1, 9) if odd else rng.choice([0, 0, 64])
    case = {"op": op, "M": _size(rng, 1, 8192, True), "N": _size(rng, 64, 8192, odd), "pad": pad}
    if op in ("norm", "norm_grad"):
        case |= {"dtype": rng.choice(["bf16", "f16"]), "residual": rng.random() < 0.6}
        if op == "norm_grad":
            case |= {"x8": rng.random() < 0.4}
    elif op == "rows":
        case |= {"dtype": rng.choice(["bf16", "f16"])}
    elif op == "grad":
        dtype = rng.choice(["bf16", "f16"])
        case |= {"K": _size(rng, 64, 8192, odd), "dtype": dtype, "layoutA": rng.choice(["k_contig", "mn_contig"]),
                 "add": rng.random() < 0.3, "dtypeD": rng.choice([dtype, dtype, "f32"])}
        # a binary32 result (a gradient that is summed over steps) costs more than a 16-bit one
        if case["dtypeD"] == "f32":
            case["M"] = min(case["M"], 4096)
    else:
        case |= {"K": _size(rng, 64, 8192, odd), "dtypeD": rng.choice(["bf16", "f16", "f32"]),
                 "layoutB": rng.choice(["k_contig", "k_contig", "mn_contig"]), "bias": rng.random() < 0.4}
    return case


def _matrix(rows, cols, pad, dtype, fill=None):
    """A rows x cols view of a buffer whose rows lie cols + pad elements apart."""
    t = torch.zeros((rows, cols + pad), dtype=dtype, device="cuda")
    if fill is not None:
        t[:, :cols] = fill.to(dtype)
    return t[:, :cols]


def _codes(g, rows, cols, pad):
    """8-bit codes of normal rows, the largest of each near the end of the range."""
    x = torch.randn((rows, cols), generator=g, device="cuda") * 32.0
    return _matrix(rows, cols, pad, torch.int8, x.round_().clamp_(-127, 127))


def _scales(g, n, around):
    return around * torch.exp(0.3 * torch.randn(n, generator=g, device="cuda"))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    M, N, pad, op = case["M"], case["N"], case["pad"], case["op"]
    s = {"case": case}

    def normal(rows, cols, dtype, gain=1.0):
        return _matrix(rows, cols, pad, DTYPES[dtype], torch.randn((rows, cols), generator=g, device="cuda") * gain)

    if op in ("norm", "norm_grad", "rows"):
        dt = case["dtype"]
        # a few channels of a residual stream are much larger than the others
        gain = torch.exp(0.5 * torch.randn(N, generator=g, device="cuda"))
        weight = (1.0 + 0.2 * torch.randn(N, generator=g, device="cuda")).to(DTYPES[dt])
        s["values"] = _matrix(M, N, pad, DTYPES[dt])
        s["q"] = _matrix(M, N, pad, torch.int8)
        s["scale"] = torch.zeros(M, device="cuda")
    if op == "norm":
        s |= {"x": normal(M, N, dt, gain), "w": weight, "rstd": torch.zeros(M, device="cuda")}
        s["r"] = normal(M, N, dt, gain) if case["residual"] else None
        s["h"] = _matrix(M, N, pad, DTYPES[dt]) if case["residual"] else None
    elif op == "norm_grad":
        x = torch.randn((M, N), generator=g, device="cuda") * gain
        if case["x8"]:
            s["scale"] = x.abs().amax(1) / 127.0
            s["q"] = _matrix(M, N, pad, torch.int8, (x / s["scale"][:, None]).round_().clamp_(-127, 127))
            x = s["q"].float() * s["scale"][:, None]
        else:
            s["x"] = _matrix(M, N, pad, DTYPES[dt], x)
            x = s["x"].float()
        s |= {"w": weight, "rstd": torch.rsqrt(x.square().mean(1) + EPS), "dy": normal(M, N, dt, 0.1),
              "dx": _matrix(M, N, pad, DTYPES[dt]), "dw": torch.zeros(N, device="cuda")}
        s["dr"] = normal(M, N, dt, 0.1) if case["residual"] else None
        s["workspace"] = torch.empty(WORKSPACE, dtype=torch.uint8, device="cuda")
    elif op == "rows":
        s["x"] = normal(M, N, dt, gain)
    elif op == "grad":
        K = case["K"]
        rows, cols = (M, K) if case["layoutA"] == "k_contig" else (K, M)
        s["a"] = normal(rows, cols, case["dtype"], 0.1)
        s["q"] = _codes(g, K, N, pad)
        s["s"] = _scales(g, K, 0.02)
        s["c"] = normal(M, N, case["dtypeD"]) if case["add"] else None
        s["d"] = _matrix(M, N, pad, DTYPES[case["dtypeD"]])
        s["workspace"] = torch.empty(WORKSPACE, dtype=torch.uint8, device="cuda")
    else:
        K = case["K"]
        s["a"] = _codes(g, M, K, pad)
        s["b"] = _codes(g, N, K, pad) if case["layoutB"] == "k_contig" else _codes(g, K, N, pad)
        s["sa"], s["sb"] = _scales(g, M, 0.02), _scales(g, N, 0.001)
        s["bias"] = torch.randn(N, generator=g, device="cuda") if case["bias"] else None
        s["d"] = _matrix(M, N, pad, DTYPES[case["dtypeD"]])
        s["workspace"] = torch.empty(WORKSPACE, dtype=torch.uint8, device="cuda")
    return s


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _quantized(y, dtype):
    """The rows of y in 8 bits: the values that the codes stand for, and the scales."""
    scale = y.abs().amax(1) / 127.0
    step = scale.clamp_min(torch.finfo(torch.float32).tiny)[:, None]
    q = (y / step).round_().clamp_(-127, 127).to(torch.int8)
    return (q * scale[:, None]).to(dtype), scale


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "norm":
        dt = DTYPES[c["dtype"]]
        h = s["x"].float()
        if s["r"] is not None:
            h = h + s["r"].float()
        rstd = torch.rsqrt(h.square().mean(1) + EPS)
        values, scale = _quantized(h * rstd[:, None] * s["w"].float(), dt)
        out = {"values": values, "scale": scale, "rstd": rstd}
        return out if s["r"] is None else out | {"h": h.to(dt)}
    if op == "norm_grad":
        x = s["q"] * s["scale"][:, None] if c["x8"] else s["x"].float()
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        g = dy * s["w"].float()
        xn = x * rstd
        dx = rstd * (g - xn * (g * xn).mean(1, keepdim=True))
        if s["dr"] is not None:
            dx = dx + s["dr"].float()
        return {"dx": dx.to(DTYPES[c["dtype"]]), "dw": (dy * xn).sum(0)}
    if op == "rows":
        values, scale = _quantized(s["x"].float(), DTYPES[c["dtype"]])
        return {"values": values, "scale": scale}
    if op == "grad":
        a = s["a"].float()
        d = (a if c["layoutA"] == "k_contig" else a.T) @ (s["q"] * s["s"][:, None])
        if s["c"] is not None:
            d = d + s["c"].float()
        return {"d": d.to(DTYPES[c["dtypeD"]])}
    b = s["b"].float()
    d = s["a"].float() @ (b.T if c["layoutB"] == "k_contig" else b) * s["sa"][:, None] * s["sb"]
    if s["bias"] is not None:
        d = d + s["bias"]
    return {"d": d.to(DTYPES[c["dtypeD"]])}


def _ld(t):
    return 0 if t is None else t.stride(0)


def _run_own(s):
    import matrix_core_gemm_amd as mcg
    c = s["case"]
    op, M, N = c["op"], c["M"], c["N"]
    if op == "norm":
        mcg.rmsnorm_quant(c["dtype"], M, N, s["x"], _ld(s["x"]), s["r"], _ld(s["r"]), s["w"], EPS, s["h"], _ld(s["h"]),
                          s["q"], _ld(s["q"]), s["scale"], s["rstd"])
        mcg.dequantize_rows(c["dtype"], M, N, s["q"], _ld(s["q"]), s["scale"], s["values"], _ld(s["values"]))
        out = {"values": s["values"], "scale": s["scale"], "rstd": s["rstd"]}
        return out if s["r"] is None else out | {"h": s["h"]}
    if op == "norm_grad":
        x, scale = (s["q"], s["scale"]) if c["x8"] else (s["x"], None)
        mcg.rmsnorm_backward(c["dtype"], "i8" if c["x8"] else c["dtype"], M, N, s["dy"], _ld(s["dy"]), x, _ld(x), scale,
                             s["w"], s["rstd"], s["dr"], _ld(s["dr"]), s["dx"], _ld(s["dx"]), s["dw"], s["workspace"])
        return {"dx": s["dx"], "dw": s["dw"]}
    if op == "rows":
        mcg.quantize_rows(c["dtype"], M, N, s["x"], _ld(s["x"]), s["q"], _ld(s["q"]), s["scale"])
        mcg.dequantize_rows(c["dtype"], M, N, s["q"], _ld(s["q"]), s["scale"], s["values"], _ld(s["values"]))
        return {"values": s["values"], "scale": s["scale"]}
    if op == "grad":
        mcg.gemm_grad_i8(c["dtype"], c["layoutA"], M, N, c["K"], s["a"], _ld(s["a"]), s["q"], _ld(s["q"]), s["s"],
                         s["c"], s["d"], _ld(s["d"]), c["dtypeD"], 0.0 if s["c"] is None else 1.0, s["workspace"])
        return {"d": s["d"]}
    mcg.gemm_i8_scaled(c["layoutB"], M, N, c["K"], s["a"], _ld(s["a"]), s["sa"], s["b"], _ld(s["b"]), s["sb"],
                       s["bias"], s["d"], _ld(s["d"]), c["dtypeD"], s["workspace"])
    return {"d": s["d"]}


def work(case):
    M, N, op = case["M"], case["N"], case["op"]
    if op == "norm":
        # x and r read, h and the codes written; scale and rstd; the weights
        return {"bytes": M * N * (7 if case["residual"] else 3) + 8 * M + 2 * N, "flops": 9 * M * N}
    if op == "norm_grad":
        read = 2 + (1 if case["x8"] else 2) + (2 if case["residual"] else 0)
        return {"bytes": M * N * (read + 2) + (8 if case["x8"] else 4) * M + 6 * N, "flops": 11 * M * N}
    if op == "rows":
        # x read, the codes written and read, the values written
        return {"bytes": M * N * 6 + 8 * M, "flops": 4 * M * N}
    K = case["K"]
    out = 4 if case["dtypeD"] == "f32" else 2
    if op == "grad":
        return {"bytes": 2 * M * K + K * N + 4 * K + M * N * out * (2 if case["add"] else 1), "flops": 2 * M * N * K}
    return {"bytes": M * K + N * K + 4 * M + (8 if case["bias"] else 4) * N + M * N * out, "flops": 2 * M * N * K}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]

    def codes_of(y):
        top = y.abs().max(dim=1, keepdim=True).values
        q = torch.where(top > 0, y * 127.0 / top, torch.zeros_like(y)).round()
        return q * top / 127.0, (top / 127.0).squeeze(1)

    if op == "norm":
        h = s["x"].double() + (s["r"].double() if case["residual"] else 0.0)
        var = torch.linalg.vector_norm(h, dim=1) ** 2 / case["N"] + EPS
        values, scale = codes_of(s["w"].double() * h / var.sqrt()[:, None])
        out = {"values": values, "scale": scale, "rstd": 1.0 / var.sqrt()}
        return out | {"h": h} if case["residual"] else out
    if op == "norm_grad":
        x = torch.diag_embed(s["scale"].double()) @ s["q"].double() if case["x8"] else s["x"].double()
        r, dy = s["rstd"].double().unsqueeze(1), s["dy"].double()
        g = dy * s["w"].double()
        dot = torch.linalg.vecdot(g, x).unsqueeze(1)
        dx = r * g - r ** 3 / case["N"] * dot * x
        if case["residual"]:
            dx += s["dr"].double()
        return {"dx": dx, "dw": torch.mv((dy * x).T.contiguous(), r.squeeze(1))}
    if op == "rows":
        values, scale = codes_of(s["x"].double())
        return {"values": values, "scale": scale}
    if op == "grad":
        a = s["a"].double()
        a = a if case["layoutA"] == "k_contig" else a.T
        d = (a * s["s"].double()) @ s["q"].double()
        return {"d": d + s["c"].double() if case["add"] else d}
    a, b = s["a"].double() * s["sa"].double()[:, None], s["b"].double()
    d = a @ (b.T if case["layoutB"] == "k_contig" else b)
    d = d * s["sb"].double()
    return {"d": d + s["bias"].double() if case["bias"] else d}
