"""Cases that time the products of expert layers and of block-scaled 8-bit floats, in plain form or with the library's kernels.

The operators (rows are tokens, columns are channels):
  blocks        a matrix in 8-bit floats with a scale for each block of 128 (of a row, of a
                column, or 128 x 128), written and read back
  f8            the product of two such matrices: a linear layer's output, its input gradient
                (B stored the other way), its weight gradient (both operands scaled along the tokens)
  grouped       a product by expert: the rows of each group by the group's own weights
  grouped_grad  its weight gradients: one product per group, over the group's rows
  grouped_f8    the product by expert on block-scaled 8-bit floats
Groups are runs of rows, given by their offsets; rows behind the last one belong to none and their
outputs stay as they were.  Codes are returned as the values they stand for, in the activations' type.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32,
          "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}  # of the 8-bit floats
BLOCK = 128


def listed():
    return [
        # an odd short batch scaled along its tokens, for a weight gradient
        {"name": "blocks_333x2047", "op": "blocks", "M": 333, "N": 2047, "dtype": "f16", "to": "e4m3", "block": "128x1",
         "pad": 3},
        # a long prompt's hidden layer on its way to a product
        {"name": "blocks_8192x8192", "op": "blocks", "M": 8192, "N": 8192, "dtype": "bf16", "to": "e4m3",
         "block": "1x128", "pad": 0},
        # one token's product: bound by reading the weights
        {"name": "f8_1x8192x8192", "op": "f8", "M": 1, "N": 8192, "K": 8192, "dtypeA": "e4m3", "layoutA": "k_contig",
         "layoutB": "k_contig", "blockB": 128, "dtypeD": "bf16", "add": False, "pad": 0},
        # the input gradient of a ragged prompt, from the weights as the forward pass has them
        {"name": "f8_x_500x4096x4096", "op": "f8", "M": 500, "N": 4096, "K": 4096, "dtypeA": "e5m2",
         "layoutA": "k_contig", "layoutB": "mn_contig", "blockB": 128, "dtypeD": "bf16", "add": False, "pad": 0},
        # the large product of training and of long prompts
        {"name": "f8_8192", "op": "f8", "M": 8192, "N": 8192, "K": 8192, "dtypeA": "e4m3", "layoutA": "k_contig",
         "layoutB": "k_contig", "blockB": 128, "dtypeD": "bf16", "add": False, "pad": 0},
        # a weight gradient over 8192 tokens, added to the binary32 gradient of earlier batches
        {"name": "f8_w_4096x4096x8192", "op": "f8", "M": 4096, "N": 4096, "K": 8192, "dtypeA": "e4m3",
         "layoutA": "mn_contig", "layoutB": "mn_contig", "blockB": 1, "dtypeD": "f32", "add": True, "pad": 0},
        # a decoding batch, two experts for each of 16 tokens: bound by reading the experts in use
        {"name": "grouped_32_of_16", "op": "grouped", "G": 16, "M": 32, "N": 4096, "K": 2048, "dtype": "bf16",
         "dtypeD": "bf16", "layoutB": "k_contig", "skew": 0.8, "tail": 0, "pad": 0},
        # a training batch over 16 experts
        {"name": "grouped_8192_of_16", "op": "grouped", "G": 16, "M": 8192, "N": 4096, "K": 4096, "dtype": "bf16",
         "dtypeD": "bf16", "layoutB": "k_contig", "skew": 0.4, "tail": 0, "pad": 0},
        # a short batch of odd sizes over few experts
        {"name": "grouped_grad_777_of_5", "op": "grouped_grad", "G": 5, "M": 1990, "N": 1147, "K": 777, "dtype": "f16",
         "dtypeD": "f32", "add": False, "skew": 0.8, "tail": 9, "pad": 5},
        # the weight gradients of a training batch over 16 experts
        {"name": "grouped_grad_8192_of_16", "op": "grouped_grad", "G": 16, "M": 4096, "N": 4096, "K": 8192,
         "dtype": "bf16", "dtypeD": "bf16", "add": False, "skew": 0.4, "tail": 0, "pad": 0},
        # a decoding batch over many 8-bit experts
        {"name": "grouped_f8_64_of_32", "op": "grouped_f8", "G": 32, "M": 64, "N": 4096, "K": 4096, "dtypeA": "e4m3",
         "dtypeD": "bf16", "layoutB": "k_contig", "skew": 0.8, "tail": 0, "pad": 0},
        # a long prompt over 8-bit experts, in a buffer with room for more rows
        {"name": "grouped_f8_8192_of_32", "op": "grouped_f8", "G": 32, "M": 8192, "N": 4096, "K": 4096,
         "dtypeA": "e4m3", "dtypeD": "bf16", "layoutB": "k_contig", "skew": 0.6, "tail": 100, "pad": 0},
    ]


def _size(rng, low, high, odd):
    """A size spread over its logarithm; a multiple of 64 (the usual widths of layers) or any."""
    n = math.exp(rng.uniform(math.log(low), math.log(high)))
    return max(low, min(high, int(n) if odd else 64 * max(1, round(n / 64))))


def draw(rng):
    op = rng.choice(["blocks", "f8", "f8", "grouped", "grouped", "grouped_grad", "grouped_f8"])
    odd = rng.random() < 0.3
    pad = rng.randrange(1, 9) if odd else rng.choice([0, 0, 64])
    case = {"op": op, "pad": pad}
    if op == "blocks":
        return case | {"M": _size(rng, 1, 8192, True), "N": _size(rng, 64, 8192, odd),
                       "dtype": rng.choice(["bf16", "f16", "f32"]), "to": rng.choice(["e4m3", "e4m3", "e5m2"]),
                       "block": rng.choice(["1x128", "128x1", "128x128"])}
    if op == "f8":
        # the output and the input gradient of a layer, or its weight gradient
        case |= {"M": _size(rng, 1, 8192, True), "N": _size(rng, 64, 8192, odd), "K": _size(rng, 64, 8192, odd),
                 "dtypeA": rng.choice(["e4m3", "e4m3", "e5m2"]), "dtypeD": rng.choice(["bf16", "bf16", "f16", "f32"]),
                 "add": rng.random() < 0.2}
        if rng.random() < 0.3:
            case |= {"layoutA": "mn_contig", "layoutB": "mn_contig", "blockB": 1}
        else:
            case |= {"layoutA": "k_contig", "layoutB": rng.choice(["k_contig", "k_contig", "mn_contig"]), "blockB": 128}
        if case["dtypeD"] != "bf16":  # (these cost more than a result in bf16)
            case["M"] = min(case["M"], 4096)
        return case
    G = _size(rng, 2, 64, True)
    case |= {"G": G, "skew": round(rng.uniform(0.0, 1.0), 2), "tail": rng.choice([0, 0, rng.randrange(1, 200)])}
    most = 1 << 27  # values of all groups' weights
    N = _size(rng, 64, 8192, odd)
    other = _size(rng, 64, max(64, min(8192, most // (G * N))), odd)
    if op == "grouped_grad":
        dtype = rng.choice(["bf16", "f16"])
        return case | {"M": N, "N": other, "K": _size(rng, 1, 8192, True), "dtype": dtype,
                       "dtypeD": rng.choice([dtype, "f32"]), "add": rng.random() < 0.3}
    case |= {"M": _size(rng, 1, 8192, True), "N": N, "K": other, "layoutB": rng.choice(["k_contig", "mn_contig"])}
    if op == "grouped":
        dtype = rng.choice(["bf16", "f16"])
        return case | {"dtype": dtype, "dtypeD": rng.choice([dtype, dtype, "f32"])}
    return case | {"dtypeA": rng.choice(["e4m3", "e4m3", "e5m2"]), "dtypeD": rng.choice(["bf16", "bf16", "f16", "f32"])}


def group_sizes(case, rows):
    """Rows of each group: uneven shares of all rows, the same for every seed of a case."""
    G, rng = case["G"], random.Random("%d %d %.2f" % (case["G"], rows, case["skew"]))
    share = [math.exp(case["skew"] * rng.gauss(0.0, 1.0)) for _ in range(G)]
    sizes = [0] * G
    for g in rng.choices(range(G), share, k=rows):
        sizes[g] += 1
    return sizes


def _matrix(rows, cols, pad, dtype, fill=None):
    """A rows x cols view of a buffer whose rows lie cols + pad elements apart."""
    t = torch.zeros((rows, cols + pad), dtype=dtype, device="cuda")
    if fill is not None:
        t[:, :cols] = fill.to(dtype)
    return t[:, :cols]


def _blocks_of(t, bm, bn):
    """The largest magnitude of each bm x bn block of the last two dimensions."""
    *lead, m, n = t.shape
    t = torch.nn.functional.pad(t.abs(), (0, -n % bn, 0, -m % bm))
    return t.reshape(*lead, -(-m // bm), bm, -(-n // bn), bn).amax((-3, -1))


def _spread(s, m, n, bm, bn):
    """Each block's value at every element of an m x n matrix."""
    return s.repeat_interleave(bm, -2)[..., :m, :].repeat_interleave(bn, -1)[..., :n]


def _f8_matrix(g, lead, m, n, bm, bn, to, gain, pad):
    """Codes and scales of normal values with a spread of magnitudes between blocks."""
    x = torch.randn((*lead, m, n), generator=g, device="cuda") * gain
    s = torch.randn((*lead, -(-m // bm), -(-n // bn)), generator=g, device="cuda")
    x *= _spread(torch.exp(0.5 * s), m, n, bm, bn)
    scale = _blocks_of(x, bm, bn) / LARGEST[to]
    q = (x / _spread(scale, m, n, bm, bn)).clamp_(-LARGEST[to], LARGEST[to])
    codes = torch.zeros((*lead, m, n + pad), dtype=torch.uint8, device="cuda")
    codes[..., :n] = q.to(DTYPES[to]).view(torch.uint8)
    return codes[..., :n], scale


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, M, N, pad = case["op"], case["M"], case["N"], case["pad"]
    s = {"case": case}

    def normal(rows, cols, dtype, gain=1.0):
        return _matrix(rows, cols, pad, DTYPES[dtype], torch.randn((rows, cols), generator=g, device="cuda") * gain)

    if op == "blocks":
        bm, bn = (int(b) for b in case["block"].split("x"))
        # a few channels of a residual stream are much larger than the others
        gain = torch.exp(0.5 * torch.randn(N, generator=g, device="cuda"))
        return s | {"x": normal(M, N, case["dtype"], gain), "bm": bm, "bn": bn, "q": _matrix(M, N, pad, torch.uint8),
                    "scale": torch.zeros((-(-M // bm), -(-N // bn)), device="cuda"),
                    "values": _matrix(M, N, pad, DTYPES[case["dtype"]])}
    K = case["K"]
    if op == "f8":
        bb = case["blockB"]
        a = (M, K, 1, BLOCK) if case["layoutA"] == "k_contig" else (K, M, BLOCK, 1)
        b = (N, K, bb, BLOCK) if case["layoutB"] == "k_contig" else (K, N, BLOCK, bb)
        s["a"], s["sa"] = _f8_matrix(g, (), *a, case["dtypeA"], 1.0, pad)
        s["b"], s["sb"] = _f8_matrix(g, (), *b, "e4m3", K ** -0.5, pad)
        s["c"] = normal(M, N, case["dtypeD"]) if case["add"] else None
        s["d"] = _matrix(M, N, pad, DTYPES[case["dtypeD"]])
        return s
    G, tail = case["G"], case["tail"]
    rows = K if op == "grouped_grad" else M
    sizes = group_sizes(case, rows)
    s["offsets"] = torch.tensor([sum(sizes[:i]) for i in range(G + 1)], dtype=torch.int32, device="cuda")
    s["rows"] = rows + tail  # of the buffers
    s["most"] = max(sizes)
    if op == "grouped_grad":
        s["a"], s["b"] = normal(rows + tail, M, case["dtype"], 0.1), normal(rows + tail, N, case["dtype"])
        s["d"] = torch.zeros((G, M, N + pad), dtype=DTYPES[case["dtypeD"]], device="cuda")[..., :N]
        s["c"] = None
        if case["add"]:
            s["c"] = torch.randn((G, M, N + pad), generator=g, device="cuda").to(DTYPES[case["dtypeD"]])[..., :N]
        return s
    b = (N, K, BLOCK, BLOCK) if case["layoutB"] == "k_contig" else (K, N, BLOCK, BLOCK)
    if op == "grouped":
        s["a"] = normal(rows + tail, K, case["dtype"])
        s["b"] = torch.zeros((G, b[0], b[1] + pad), dtype=DTYPES[case["dtype"]], device="cuda")[..., :b[1]]
        s["b"].copy_(torch.randn((G, b[0], b[1]), generator=g, device="cuda") * K ** -0.5)
    else:
        s["a"], s["sa"] = _f8_matrix(g, (), rows + tail, K, 1, BLOCK, case["dtypeA"], 1.0, pad)
        s["b"], s["sb"] = _f8_matrix(g, (G,), *b, "e4m3", K ** -0.5, pad)
    s["d"] = _matrix(rows + tail, N, pad, DTYPES[case["dtypeD"]])
    return s


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _values(codes, to, scale, bm, bn):
    """The binary32 values of block-scaled codes."""
    return codes.view(DTYPES[to]).float() * _spread(scale, codes.shape[-2], codes.shape[-1], bm, bn)


def _by_group(s):
    """Rows of each group in a padded matrix of `most` rows: their indices, and which of them are the group's."""
    first, end = s["offsets"][:-1, None], s["offsets"][1:, None]
    index = first + torch.arange(s["most"], dtype=torch.int32, device="cuda")
    return index.clamp(max=s["rows"] - 1).long(), index < end


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "blocks":
        dt, bm, bn = DTYPES[c["dtype"]], s["bm"], s["bn"]
        x, most = s["x"].float(), LARGEST[c["to"]]
        top = _blocks_of(x, bm, bn)
        scale = top / most
        q = (x * most / _spread(top, c["M"], c["N"], bm, bn)).nan_to_num_(nan=0.0)
        return {"values": (q.to(DTYPES[c["to"]]).float() * _spread(scale, c["M"], c["N"], bm, bn)).to(dt), "scale": scale}
    if op == "f8":
        bb = c["blockB"]
        ba, bb = (1, BLOCK) if c["layoutA"] == "k_contig" else (BLOCK, 1), (bb, BLOCK) if c["layoutB"] == "k_contig" else (BLOCK, bb)
        a, b = _values(s["a"], c["dtypeA"], s["sa"], *ba), _values(s["b"], "e4m3", s["sb"], *bb)
        d = (a if c["layoutA"] == "k_contig" else a.T) @ (b.T if c["layoutB"] == "k_contig" else b)
        return {"d": (d if s["c"] is None else d + s["c"].float()).to(DTYPES[c["dtypeD"]])}
    index, mine = _by_group(s)
    if op == "grouped_grad":
        a = s["a"].float()[index] * mine[..., None]
        d = torch.bmm(a.transpose(1, 2).contiguous(), s["b"].float()[index])
        return {"d": (d if s["c"] is None else d + s["c"].float()).to(DTYPES[c["dtypeD"]])}
    if op == "grouped":
        a, b = s["a"].float(), s["b"].float()
    else:
        a, b = _values(s["a"], c["dtypeA"], s["sa"], 1, BLOCK), _values(s["b"], "e4m3", s["sb"], BLOCK, BLOCK)
    b = b.transpose(1, 2).contiguous() if c["layoutB"] == "k_contig" else b.contiguous()
    d = torch.bmm(a[index], b)
    s["d"][index[mine]] = d[mine].to(DTYPES[c["dtypeD"]])
    return {"d": s["d"]}


def _ld(t):
    return 0 if t is None else t.stride(-2)


def _run_own(s):
    import matrix_core_gemm_amd as mcg
    c = s["case"]
    op, M, N = c["op"], c["M"], c["N"]
    if op == "blocks":
        mcg.quantize_blocks(c["dtype"], c["to"], s["bm"], s["bn"], M, N, s["x"], _ld(s["x"]), s["q"], _ld(s["q"]),
                            s["scale"], _ld(s["scale"]))
        mcg.dequantize_blocks(c["to"], c["dtype"], s["bm"], s["bn"], M, N, s["q"], _ld(s["q"]), s["scale"],
                              _ld(s["scale"]), s["values"], _ld(s["values"]))
        return {"values": s["values"], "scale": s["scale"]}
    K = c["K"]
    if op == "f8":
        mcg.gemm_f8_blocks(c["dtypeA"], "e4m3", c["layoutA"], c["layoutB"], c["blockB"], M, N, K, s["a"], _ld(s["a"]),
                           s["sa"], _ld(s["sa"]), s["b"], _ld(s["b"]), s["sb"], _ld(s["sb"]), s["c"], s["d"],
                           _ld(s["d"]), c["dtypeD"], 0.0 if s["c"] is None else 1.0)
        return {"d": s["d"]}
    G = c["G"]
    if op == "grouped_grad":
        mcg.gemm_grouped_grad(c["dtype"], G, M, N, s["rows"], s["offsets"], s["a"], _ld(s["a"]), s["b"], _ld(s["b"]),
                              s["c"], s["d"], _ld(s["d"]), s["d"].stride(0), c["dtypeD"], 0.0 if s["c"] is None else 1.0)
    elif op == "grouped":
        mcg.gemm_grouped(c["dtype"], c["layoutB"], G, s["rows"], N, K, s["offsets"], s["a"], _ld(s["a"]), s["b"],
                         _ld(s["b"]), s["b"].stride(0), s["d"], _ld(s["d"]), c["dtypeD"])
    else:
        mcg.gemm_grouped_f8_blocks(c["dtypeA"], "e4m3", c["layoutB"], G, s["rows"], N, K, s["offsets"], s["a"],
                                   _ld(s["a"]), s["sa"], _ld(s["sa"]), s["b"], _ld(s["b"]), s["b"].stride(0), s["sb"],
                                   _ld(s["sb"]), s["sb"].stride(0), s["d"], _ld(s["d"]), c["dtypeD"])
    return {"d": s["d"]}


def work(case):
    op, M, N = case["op"], case["M"], case["N"]
    size = {"bf16": 2, "f16": 2, "f32": 4}
    if op == "blocks":
        bm, bn = (int(b) for b in case["block"].split("x"))
        # x read, the codes written and read, the values written; the scales both ways
        return {"bytes": M * N * (2 * size[case["dtype"]] + 2) + 8 * -(-M // bm) * -(-N // bn), "flops": 5 * M * N}
    K, out = case["K"], size[case["dtypeD"]]
    kb = -(-K // BLOCK)
    if op == "f8":
        scales = 4 * kb * (M + -(-N // case["blockB"]))
        return {"bytes": M * K + N * K + scales + M * N * out * (2 if case["add"] else 1), "flops": 2 * M * N * K}
    G = case["G"]
    used = sum(n > 0 for n in group_sizes(case, K if op == "grouped_grad" else M))
    if op == "grouped_grad":
        return {"bytes": 2 * K * (M + N) + G * M * N * out * (2 if case["add"] else 1), "flops": 2 * M * N * K}
    if op == "grouped":
        return {"bytes": 2 * M * K + 2 * used * N * K + M * N * out, "flops": 2 * M * N * K}
    return {"bytes": M * K + 4 * M * kb + used * (N * K + 4 * kb * -(-N // BLOCK)) + M * N * out, "flops": 2 * M * N * K}


def exact(case, seed):
    s = prepare(case, seed)
    op, M, N = case["op"], case["M"], case["N"]

    def weighed(codes, to, scale, along):
        """64-bit values of codes by their blocks: `along` says at which places of 128 a dimension changes blocks."""
        r, c = (torch.arange(n, device="cuda") // (BLOCK if b else 1) for n, b in zip(codes.shape[-2:], along))
        return scale.double()[..., r, :][..., c] * codes.contiguous().view(DTYPES[to]).double()

    def near(x, mantissa, low):
        """x to the nearest value with so many bits behind the first, none finer than 2^low, ties to even."""
        e = torch.frexp(x).exponent - 1
        step = torch.ldexp(torch.ones_like(x), torch.clamp(e - mantissa, min=low))
        return torch.round(x / step) * step

    if op == "blocks":
        x, bm, bn = s["x"].double(), s["bm"], s["bn"]
        r, c = torch.arange(M, device="cuda") // bm, torch.arange(N, device="cuda") // bn
        at = (r[:, None] * s["scale"].shape[1] + c).flatten()
        top = torch.zeros(s["scale"].numel(), dtype=torch.float64, device="cuda")
        top = top.scatter_reduce(0, at, x.abs().flatten(), "amax")
        most, t = LARGEST[case["to"]], top[at].reshape(M, N)
        q = near(torch.where(t > 0, x / t * most, torch.zeros_like(x)), *((3, -9) if case["to"] == "e4m3" else (2, -16)))
        return {"values": q * t / most, "scale": (top / most).reshape(s["scale"].shape)}
    if op == "f8":
        a = weighed(s["a"], case["dtypeA"], s["sa"], (case["layoutA"] != "k_contig", case["layoutA"] == "k_contig"))
        b = weighed(s["b"], "e4m3", s["sb"], (True, True) if case["blockB"] == BLOCK else
                    (case["layoutB"] != "k_contig", case["layoutB"] == "k_contig"))
        if case["layoutA"] != "k_contig":
            a = a.T
        d = torch.mm(a, b if case["layoutB"] != "k_contig" else b.T)
        return {"d": d + s["c"].double() if case["add"] else d}
    ends = s["offsets"].tolist()
    d = torch.zeros(s["d"].shape, dtype=torch.float64, device="cuda")
    for i, (r0, r1) in enumerate(zip(ends, ends[1:])):
        if op == "grouped_grad":
            d[i] = s["a"][r0:r1].double().T @ s["b"][r0:r1].double()
            if case["add"]:
                d[i] += s["c"][i].double()
            continue
        if r1 == r0:
            continue
        if op == "grouped":
            a, b = s["a"][r0:r1].double(), s["b"][i].double()
        else:
            a = weighed(s["a"][r0:r1], case["dtypeA"], s["sa"][r0:r1], (False, True))
            b = weighed(s["b"][i], "e4m3", s["sb"][i], (True, True))
        d[r0:r1] = a @ (b.T if case["layoutB"] == "k_contig" else b)
    return {"d": d}
