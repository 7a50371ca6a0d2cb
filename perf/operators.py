"""Measured calls of the operators on lists of gradients and on microscaled
4-bit matrices (blocks of 32 elements, 4-bit e2m1 values, 8-bit power-of-two
scales).

Where ``own`` is false, ``run`` computes an operator in its plain form with
elementary torch operations; where it is true, it makes the library's calls.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ESIZE = {"f32": 4, "bf16": 2, "f16": 2}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # gradients of the two grouped value networks at the headline shape:
        # 12 small tensors, where the launches are what counts
        dict(name="norm_two_value_networks", op="norm", net="value", copies=2, S=128, H=128, dtype="f32", kind=2),
        # a stack of four layers of width 2048, all gradients in bfloat16:
        # the norm that a training log shows, with each tensor's own
        dict(name="norm_stack_bf16", op="norm", net="stack", copies=4, S=0, H=2048, dtype="bf16", kind=2),
        # odd widths and three types in one list, largest magnitude
        dict(name="norm_max_mixed_odd", op="norm", net="stack", copies=6, S=0, H=777, dtype="mixed", kind=0),
        # the budgeted network (four value networks): its gradients clipped
        # into one flat vector, as the gradient budget takes them
        dict(name="clip_flat_budget_network", op="clip", net="value", copies=4, S=128, H=128, dtype="f32",
             flat=True, active=True),
        # 1 GiB of fp32 gradients clipped into the flat vector
        dict(name="clip_flat_stack_f32", op="clip", net="stack", copies=4, S=0, H=2048, dtype="f32", flat=True,
             active=True),
        # in place, with a norm below the bound, the usual step of a settled run
        dict(name="clip_in_place_f16", op="clip", net="stack", copies=6, S=0, H=1000, dtype="f16", flat=False,
             active=False),
        # the states of one headline batch
        dict(name="quantize_states", op="quantize", rows=16384, cols=128, dtype="f32", axis=1),
        # half-precision activations of odd sizes, quantised along the batch
        # (the operand of a weight gradient)
        dict(name="quantize_odd_f16_columns", op="quantize", rows=5001, cols=777, dtype="f16", axis=0),
        # a large weight, quantised along its rows
        dict(name="quantize_weight_bf16", op="quantize", rows=8192, cols=8192, dtype="bf16", axis=1),
        # one row through a layer whose weights are held in 4 bits
        dict(name="product_one_row", op="product", M=1, N=4096, K=4096, left="bf16", out="bf16", bias=True,
             relu=False),
        # first layer of the widest value network over its largest batch
        dict(name="product_states_layer", op="product", M=65536, N=512, K=256, left="f32", out="bf16", bias=True,
             relu=True),
        # both operands in 4 bits, a large square product
        dict(name="product_square", op="product", M=8192, N=8192, K=8192, left="mx4", out="bf16", bias=False,
             relu=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "clip", "quantize", "quantize", "product", "product"])
    if op in ("norm", "clip"):
        net = rng.choice(["value", "stack"])
        case = dict(op=op, net=net, dtype=rng.choice(["f32", "bf16", "f16", "mixed"]))
        if net == "value":
            case.update(copies=rng.randint(1, 8), S=_log_int(rng, 3, 512), H=_log_int(rng, 16, 1024))
        else:
            copies = rng.randint(1, 6)
            case.update(copies=copies, S=0, H=_log_int(rng, 32, 4096 / math.sqrt(copies)))
        if op == "norm":
            case["kind"] = rng.choice([2, 2, 0])
        else:
            case["flat"] = rng.random() < 0.7
            case["active"] = case["flat"] and rng.random() < 0.8
        return case
    if op == "quantize":
        cols = _log_int(rng, 1, 16384)
        return dict(op=op, rows=_log_int(rng, 1, (1 << 26) / cols), cols=cols,
                    dtype=rng.choice(["f32", "bf16", "f16"]), axis=rng.choice([0, 1]))
    while True:
        M = rng.choice([rng.randint(1, 16), _log_int(rng, 1, 65536)])
        N, K = _log_int(rng, 8, 8192), _log_int(rng, 8, 8192)
        if M * N <= 1 << 26 and M * K <= 1 << 26:
            break
    return dict(op=op, M=M, N=N, K=K, left=rng.choice(["f32", "bf16", "f16", "mx4"]),
                out=rng.choice(["f32", "bf16", "f16"]), bias=rng.random() < 0.5, relu=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs
def _shapes(case):
    H = case["H"]
    if case["net"] == "value":  # W1, b1, W2, b2, w3, b3
        one = [(H, case["S"]), (H,), (H, H), (H,), (H,), (1,)]
    else:                       # four square weights, three of width 4 H, two vectors
        one = [(H, H)] * 4 + [(4 * H, H)] * 2 + [(H, 4 * H)] + [(H,)] * 2
    return one * case["copies"]


def _types(case, count):
    names = ["f32", "bf16", "f16"] if case["dtype"] == "mixed" else [case["dtype"]]
    return [names[i % len(names)] for i in range(count)]


def _numels(case):
    return [math.prod(s) for s in _shapes(case)]


def _rng(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 2654435761 % (1 << 31) + 12345)


def _normal(gen, shape, dtype, scale):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _activations(gen, rows, cols, dtype):
    """Normal values whose columns differ in size, a few of them large, as
    the inputs and hidden activations of a network do."""
    x = torch.randn((rows, cols), generator=gen, device="cuda", dtype=torch.float32)
    x *= torch.exp2(torch.randn((cols,), generator=gen, device="cuda"))
    return x.to(dtype)


def prepare(case, seed):
    gen = _rng(seed)
    st = dict(case=case)
    if case["op"] in ("norm", "clip"):
        shapes = _shapes(case)
        sizes = torch.exp2(torch.rand(len(shapes), generator=gen, device="cuda") * 6 - 8).tolist()
        st["grads"] = [_normal(gen, s, DTYPES[t], z) for s, t, z in zip(shapes, _types(case, len(shapes)), sizes)]
        if case["op"] == "clip":
            # the bound, from the sizes the gradients are drawn with
            expect = math.sqrt(sum(n * z * z for n, z in zip(_numels(case), sizes)))
            st["max_norm"] = expect * (0.25 if case["active"] else 4.0)
    elif case["op"] == "quantize":
        st["x"] = _activations(gen, case["rows"], case["cols"], DTYPES[case["dtype"]])
    else:
        M, N, K = case["M"], case["N"], case["K"]
        st["w"] = _plain_quantize(_normal(gen, (N, K), torch.float32, 1.0 / math.sqrt(K)))
        x = _activations(gen, M, K, DTYPES.get(case["left"], torch.float32))
        st["x"] = _plain_quantize(x) if case["left"] == "mx4" else x
        st["bias"] = _normal(gen, (N,), torch.float32, 0.1) if case["bias"] else None
    if own:
        _prepare_own(st)
    return st


def _prepare_own(st):
    import offline_rl_step_amd as m
    case = st["case"]
    new = lambda *shape, dtype=torch.float32: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
    if case["op"] in ("norm", "clip"):
        st["set"] = m.TensorSet(st["grads"])
        st["ws"] = m.grad_norm_workspace(st["set"])
        st["out"] = new(1 if case["op"] == "norm" else 2)
        if case["op"] == "norm":
            st["each"] = new(len(st["grads"]))
        elif case["flat"]:
            st["flat"] = new(st["set"].numel)
    elif case["op"] == "quantize":
        st["q"] = m.mx4_empty(case["rows"], case["cols"], case["axis"])
        st["values"] = new(st["q"].rows, st["q"].cols)
    else:
        st["wq"] = m.Mx4(*st["w"], case["N"], case["K"])
        if case["left"] == "mx4":
            st["xq"] = m.Mx4(*st["x"], case["M"], case["K"])
        st["y"] = new(case["M"], case["N"], dtype=DTYPES[case["out"]])
        st["ws"] = m.mx4_matmul_workspace(case["M"], case["N"], case["K"])


# --------------------------------------------------------------- plain form
def _blocks(x):
    """[rows, cols] in fp32 as [rows, blocks, 32], padded with zeros."""
    rows, cols = x.shape
    x = x.float()
    pad = -cols % 32
    if pad:
        x = torch.cat([x, x.new_zeros((rows, pad))], 1)
    return x.view(rows, -1, 32)


def _plain_quantize(x):
    """(codes [rows, blocks * 16], scales [rows, blocks]), both uint8; the
    element of even index lies in a byte's low half."""
    b = _blocks(x)
    bits = b.abs().amax(2).view(torch.int32)
    scale = ((bits >> 23) - 2).clamp(min=0)
    y = b * ((254 - scale) << 23).view(torch.float32)[:, :, None]
    a = y.abs()
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
            + (a >= 3.5).int() + (a > 5.0).int())
    code = (code + 8 * (y < 0).int()).view(x.shape[0], -1)
    return (code[:, 0::2] + 16 * code[:, 1::2]).to(torch.uint8), scale.to(torch.uint8)


def _plain_dequantize(codes, scales, cols):
    levels = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    levels = torch.cat([levels, -levels])
    c = codes.int()
    v = torch.stack([levels[c & 15], levels[c >> 4]], 2).view(codes.shape[0], -1, 32)
    return (v * torch.ldexp(torch.ones((), device=codes.device), scales.int() - 127)[:, :, None]).view(
        codes.shape[0], -1)[:, :cols]


def _run_plain(st):
    case = st["case"]
    if case["op"] == "norm":
        if case["kind"] == 0:
            each = torch.stack([g.float().abs().amax() for g in st["grads"]])
            return [each.amax().view(1), each]
        sums = torch.stack([g.float().square().sum(dtype=torch.float64) for g in st["grads"]])
        return [sums.sum().sqrt().float().view(1), sums.sqrt().float()]
    if case["op"] == "clip":
        norm = torch.stack([g.float().square().sum(dtype=torch.float64) for g in st["grads"]]).sum().sqrt()
        c = torch.where(norm > st["max_norm"], st["max_norm"] / norm, torch.ones_like(norm)).float()
        out = torch.stack([norm.float(), c])
        if case["flat"]:
            return [out, torch.cat([g.float().view(-1) for g in st["grads"]]) * c]
        return [out] + [(g.float() * c).to(g.dtype) for g in st["grads"]]
    if case["op"] == "quantize":
        x = st["x"] if case["axis"] == 1 else st["x"].t()
        return _plain_dequantize(*_plain_quantize(x), x.shape[1])
    K = case["K"]
    x = _plain_dequantize(*(st["x"] if case["left"] == "mx4" else _plain_quantize(st["x"])), K)
    y = x @ _plain_dequantize(*st["w"], K).t()
    if st["bias"] is not None:
        y = y + st["bias"]
    if case["relu"]:
        y = torch.relu(y)
    return y.to(DTYPES[case["out"]])


# ------------------------------------------------------------- library calls
def _run_own(st):
    import offline_rl_step_amd as m
    case = st["case"]
    if case["op"] == "norm":
        m.grad_norm(st["set"], st["out"], st["ws"], kind=m.NORM_L2 if case["kind"] == 2 else m.NORM_MAX,
                    out_each=st["each"])
        return [st["out"], st["each"]]
    if case["op"] == "clip":
        m.grad_clip(st["set"], st["max_norm"], st["out"], st["ws"], out_flat=st["flat"] if case["flat"] else None)
        return [st["out"], st["flat"]] if case["flat"] else [st["out"]] + st["grads"]
    if case["op"] == "quantize":
        m.mx4_quantize(st["x"], st["q"], axis=case["axis"])
        m.mx4_dequantize(st["q"], st["values"])
        return st["values"]
    if case["left"] == "mx4":
        m.mx4_matmul(st["xq"], st["wq"], st["y"], st["ws"], bias=st["bias"], relu=case["relu"])
    else:
        m.mx4_linear(st["x"], st["wq"], st["y"], st["ws"], bias=st["bias"], relu=case["relu"])
    return st["y"]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------- least work of a pass
def work(case):
    if case["op"] in ("norm", "clip"):
        numels = _numels(case)
        n = sum(numels)
        read = sum(k * ESIZE[t] for k, t in zip(numels, _types(case, len(numels))))
        if case["op"] == "norm":
            return {"bytes": read + 4 * (len(numels) + 1), "flops": 2 * n}
        if case["flat"]:
            return {"bytes": read + 4 * n + 8, "flops": 3 * n}
        return {"bytes": read + 8, "flops": 2 * n}  # below the bound nothing is written
    if case["op"] == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (ESIZE[case["dtype"]] + 4), "flops": 3 * n}
    M, N, K = case["M"], case["N"], case["K"]
    kp = -(-K // 32) * 32
    packed = kp // 2 + kp // 32
    left = M * packed if case["left"] == "mx4" else M * K * ESIZE[case["left"]]
    return {"bytes": left + N * packed + M * N * ESIZE[case["out"]] + (4 * N if case["bias"] else 0),
            "flops": 2 * M * N * K}


# ------------------------------------------------------------ 64-bit results
def _exact_blocks(x):
    """Values of x [rows, cols] (64 bits) after quantisation along the rows:
    the block's scale is 2^(floor(log2(largest)) - 2), an element the nearest
    multiple of its binade's step, ties to the even multiple, at most 6."""
    rows, cols = x.shape
    padded = torch.zeros((rows, -(-cols // 32) * 32), dtype=torch.float64, device=x.device)
    padded[:, :cols] = x
    b = padded.view(rows, -1, 32)
    _, e = torch.frexp(b.abs().amax(2, keepdim=True))
    e = torch.where(b.abs().amax(2, keepdim=True) > 0, (e - 3).clamp(min=-127), -127).double()
    y = b * torch.exp2(-e)
    _, ye = torch.frexp(y)
    step = torch.exp2((ye - 1).clamp(min=0).double() - 1)
    q = (torch.round(y / step) * step).clamp(-6, 6)
    return (q * torch.exp2(e)).view(rows, -1)[:, :cols]


def _exact_values(pair, cols):
    codes, scales = pair
    c = torch.stack([codes & 15, codes >> 4], 2).view(codes.shape[0], -1).double()
    sign = torch.where(c >= 8, -1.0, 1.0).double()
    c = c % 8
    mag = torch.where(c < 2, c * 0.5, (1 + (c % 2) * 0.5) * torch.exp2(torch.floor(c / 2) - 1))
    s = torch.exp2(scales.double() - 127).repeat_interleave(32, 1)
    return (sign * mag * s)[:, :cols]


def exact(case, seed):
    global own
    keep, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = keep
    if case["op"] == "norm":
        each = [g.double() for g in st["grads"]]
        each = torch.stack([g.abs().max() if case["kind"] == 0 else torch.linalg.vector_norm(g) for g in each])
        return [(each.max() if case["kind"] == 0 else torch.linalg.vector_norm(each)).view(1), each]
    if case["op"] == "clip":
        norm = torch.sqrt(sum(torch.sum(g.double() ** 2) for g in st["grads"]))
        c = min(1.0, st["max_norm"] / norm.item())
        out = torch.tensor([norm.item(), c], dtype=torch.float64, device="cuda")
        if case["flat"]:
            return [out, torch.cat([g.double().view(-1) * c for g in st["grads"]])]
        return [out] + [g.double() * c for g in st["grads"]]
    if case["op"] == "quantize":
        x = st["x"].double()
        return _exact_blocks(x if case["axis"] == 1 else x.t())
    x = _exact_values(st["x"], case["K"]) if case["left"] == "mx4" else _exact_blocks(st["x"].double())
    y = x @ _exact_values(st["w"], case["K"]).t()
    if st["bias"] is not None:
        y += st["bias"].double()
    return y.clamp(min=0) if case["relu"] else y
