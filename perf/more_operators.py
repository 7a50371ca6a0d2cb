"""Measured calls of the operators that train and evaluate a policy over a large
set of discrete actions: the loss of the actions taken (softmax cross entropy of
a linear head, with its gradients) and the orthogonalised update of a list of
weight matrices.

Where ``own`` is false, ``run`` computes an operator in its plain form with
elementary torch operations; where it is true, it makes the library's calls.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ESIZE = {"f32": 4, "bf16": 2, "f16": 2}

# the quintic whose repeated application drives singular values towards 1
QUINTIC = (3.4445, -4.7750, 2.0315)
STEPS = 5
EPS = 1e-7
# a training step's settings
LR, MOMENTUM, DECAY = 0.02, 0.95, 0.1


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one state: the log-probability of the action taken among 32768, as a
        # policy that acts or is evaluated step by step asks for it
        dict(name="loss_one_state", op="loss", rows=1, dim=512, actions=32768, dtype="bf16", bias=True, grad=False),
        # the headline batch: hidden width 128, nine actions
        dict(name="loss_nine_actions", op="loss", rows=16384, dim=128, actions=9, dtype="f32", bias=True, grad=True),
        # odd sizes in half precision
        dict(name="loss_odd_f16", op="loss", rows=777, dim=501, actions=10007, dtype="f16", bias=True, grad=True),
        # evaluation of a batch under the current policy, no gradients
        dict(name="loss_evaluate_bf16", op="loss", rows=16384, dim=512, actions=32768, dtype="bf16", bias=False,
             grad=False),
        # full precision, a head of medium size
        dict(name="loss_f32", op="loss", rows=4096, dim=512, actions=16384, dtype="f32", bias=False, grad=True),
        # the largest: its logits alone would be 2 GiB in fp32
        dict(name="loss_large_bf16", op="loss", rows=8192, dim=2048, actions=65536, dtype="bf16", bias=True,
             grad=True),
        # weight matrices of the two grouped value networks of the headline
        # shape, where the launches are what counts
        dict(name="step_two_value_networks", op="step", net="value", copies=2, S=128, H=128, x="f32", out="f32"),
        # the widest value networks, two trainers'
        dict(name="step_wide_value_network", op="step", net="value", copies=2, S=256, H=512, x="f32", out="f32"),
        # odd widths, binary16 results
        dict(name="orthogonalize_odd_f16", op="orthogonalize", net="stack", copies=1, S=0, H=777, x="f16", out="f16"),
        # a stack of one layer of width 2048, weights and gradients in bfloat16
        dict(name="step_stack_bf16", op="step", net="stack", copies=1, S=0, H=2048, x="bf16", out="bf16"),
        # the same kind of list with everything in fp32
        dict(name="step_stack_f32", op="step", net="stack", copies=1, S=0, H=1024, x="f32", out="f32"),
        # one large square matrix
        dict(name="orthogonalize_square", op="orthogonalize", net="one", copies=1, S=8192, H=8192, x="f32",
             out="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.5:
        while True:
            rows = rng.randint(1, 16) if rng.random() < 0.3 else _log_int(rng, 1, 16384)
            dim, actions = _log_int(rng, 8, 2048), _log_int(rng, 2, 131072)
            if rows * actions <= 1 << 29 and rows * actions * dim <= 1 << 40:
                break
        return dict(op="loss", rows=rows, dim=dim, actions=actions, dtype=rng.choice(["f32", "bf16", "f16"]),
                    bias=rng.random() < 0.5, grad=rng.random() < 0.7)
    case = dict(op=rng.choice(["step", "step", "orthogonalize"]), net=rng.choice(["value", "stack", "one"]))
    if case["net"] == "value":
        case.update(copies=rng.randint(1, 8), S=_log_int(rng, 3, 512), H=_log_int(rng, 16, 1024))
    elif case["net"] == "stack":
        case.update(copies=rng.randint(1, 3), S=0, H=_log_int(rng, 16, 2048))
    else:
        case.update(copies=1, S=_log_int(rng, 1, 8192), H=_log_int(rng, 1, 8192))
    case.update(x=rng.choice(["f32", "bf16", "f16"]), out=rng.choice(["f32", "bf16", "bf16", "f16"]))
    return case


# ------------------------------------------------------------------ inputs
def _shapes(case):
    H, S = case["H"], case["S"]
    if case["net"] == "value":    # W1, W2
        one = [(H, S), (H, H)]
    elif case["net"] == "stack":  # four square weights, three of width 4 H
        one = [(H, H)] * 4 + [(4 * H, H)] * 2 + [(H, 4 * H)]
    else:
        one = [(S, H)]
    return one * case["copies"]


def _rng(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 2654435761 % (1 << 31) + 54321)


def _normal(gen, shape, dtype, scale):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _gradient(gen, shape, dtype):
    """A weight gradient as backward passes leave it: a sum of a few strong
    directions and of many weak ones."""
    rows, cols = shape
    k = min(4, rows, cols)
    strong = torch.randn((rows, k), generator=gen, device="cuda") @ torch.randn((k, cols), generator=gen, device="cuda")
    return ((strong + torch.randn(shape, generator=gen, device="cuda")) * 1e-3).to(dtype)


def prepare(case, seed):
    gen = _rng(seed)
    st = dict(case=case)
    if case["op"] == "loss":
        rows, dim, actions, dtype = case["rows"], case["dim"], case["actions"], DTYPES[case["dtype"]]
        # hidden activations behind a ReLU, columns of different sizes
        h = torch.relu(torch.randn((rows, dim), generator=gen, device="cuda"))
        st["hidden"] = (h * torch.exp2(torch.randn((dim,), generator=gen, device="cuda") * 0.5)).to(dtype)
        st["weight"] = _normal(gen, (actions, dim), dtype, 2.0 / math.sqrt(dim))
        taken = torch.randint(0, actions, (rows,), generator=gen, device="cuda", dtype=torch.int32)
        st["bias"] = None
        if case["bias"]:
            # actions that the state's rules forbid have a bias of minus infinity; none of them was taken
            bias = _normal(gen, (actions,), torch.float32, 0.5)
            allowed = bias.clone()
            bias[torch.rand((actions,), generator=gen, device="cuda") < 0.05] = -math.inf
            bias[taken.long()] = allowed[taken.long()]
            st["bias"] = bias
        if rows > 1:  # rows that hold no action (the padding of a ragged batch)
            taken[torch.rand((rows,), generator=gen, device="cuda") < 0.03] = -1
        st["taken"] = taken
        st["row_weights"] = torch.rand((rows,), generator=gen, device="cuda") * 0.9 + 0.1
    else:
        shapes = _shapes(case)
        st["x"] = [_gradient(gen, s, DTYPES[case["x"]]) for s in shapes]
        if case["op"] == "step":
            st["w"] = [_normal(gen, s, DTYPES[case["out"]], 1.0 / math.sqrt(s[1])) for s in shapes]
            st["m"] = [_gradient(gen, s, torch.float32) * 5 for s in shapes]
        else:
            st["w"] = [torch.empty(s, dtype=DTYPES[case["out"]], device="cuda") for s in shapes]
    if own:
        _prepare_own(st)
    return st


def _prepare_own(st):
    import offline_rl_step_amd as m
    case = st["case"]
    if case["op"] == "loss":
        rows, dim, actions, dtype = case["rows"], case["dim"], case["actions"], DTYPES[case["dtype"]]
        new = lambda shape, t: torch.empty(shape, dtype=t, device="cuda")  # noqa: E731
        st["ws"] = m.policy_loss_workspace(rows, actions, dim, dtype, grad=case["grad"])
        st["loss"] = new((1,), torch.float32)
        st["nll"], st["lse"] = new((rows,), torch.float32), new((rows,), torch.float32)
        if case["grad"]:
            st["d_hidden"], st["d_weight"] = new((rows, dim), dtype), new((actions, dim), dtype)
            st["d_bias"] = new((actions,), torch.float32) if case["bias"] else None
    else:
        st["set"] = m.MatrixSet(st["x"], st["w"], st.get("m"))
        st["ws"] = m.orthogonalize_workspace(st["set"])


# --------------------------------------------------------------- plain form
def _plain_loss(st):
    case, taken = st["case"], st["taken"].long()
    h, w = st["hidden"].float(), st["weight"].float()
    z = h @ w.t()
    if st["bias"] is not None:
        z = z + st["bias"]
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    lse = (top + torch.log(total))[:, 0]
    there = taken >= 0
    at = taken.clamp(min=0)[:, None]
    nll = torch.where(there, lse - z.gather(1, at)[:, 0], 0.0)
    weight = torch.where(there, st["row_weights"], 0.0) / case["rows"]
    loss = (weight.double() * nll.double()).sum().float().view(1)
    out = [loss, nll, lse]
    if case["grad"]:
        g = e.div_(total)
        g.scatter_add_(1, at, torch.full_like(at, -1.0, dtype=torch.float32))
        g.mul_(weight[:, None])
        out += [(g @ w).to(st["hidden"].dtype), (g.t() @ h).to(st["weight"].dtype)]
        if st["bias"] is not None:
            out.append(g.sum(0))
    return out


def _plain_orthogonalize(u):
    a, b, c = QUINTIC
    x = u / (u.double().square().sum().sqrt().float() + EPS)
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.t()
    for _ in range(STEPS):
        s = x @ x.t()
        x = a * x + (b * s + c * (s @ s)) @ x
    return x.t() if tall else x


def _plain_step(g, m, w):
    m.mul_(MOMENTUM).add_(g.float())
    o = _plain_orthogonalize(g.float() + MOMENTUM * m)
    scale = math.sqrt(max(1.0, w.shape[0] / w.shape[1]))
    w.copy_((w.float() * (1.0 - LR * DECAY) - (LR * scale) * o).to(w.dtype))


def _run_plain(st):
    case = st["case"]
    if case["op"] == "loss":
        return _plain_loss(st)
    if case["op"] == "step":
        for g, m, w in zip(st["x"], st["m"], st["w"]):
            _plain_step(g, m, w)
        return st["w"] + st["m"]
    return [_plain_orthogonalize(x.float()).to(w.dtype) for x, w in zip(st["x"], st["w"])]


# ------------------------------------------------------------- library calls
def _run_own(st):
    import offline_rl_step_amd as m
    case = st["case"]
    if case["op"] == "loss":
        m.policy_loss(st["hidden"], st["weight"], st["taken"], st["nll"], st["lse"], st["ws"], bias=st["bias"],
                      row_weights=st["row_weights"], out_loss=st["loss"])
        out = [st["loss"], st["nll"], st["lse"]]
        if case["grad"]:
            m.policy_loss_grad(st["hidden"], st["weight"], st["taken"], st["lse"], st["ws"], bias=st["bias"],
                               row_weights=st["row_weights"], d_hidden=st["d_hidden"], d_weight=st["d_weight"],
                               d_bias=st["d_bias"])
            out += [st["d_hidden"], st["d_weight"]]
            if st["d_bias"] is not None:
                out.append(st["d_bias"])
        return out
    if case["op"] == "step":
        m.muon_step(st["set"], st["ws"], LR, momentum=MOMENTUM, weight_decay=DECAY)
        return st["w"] + st["m"]
    m.orthogonalize(st["set"], st["ws"])
    return st["w"]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------- least work of a pass
def work(case):
    if case["op"] == "loss":
        n, d, v, es = case["rows"], case["dim"], case["actions"], ESIZE[case["dtype"]]
        least = (n + v) * d * es + 8 * n + (4 * v if case["bias"] else 0) + 8 * n + 4
        if case["grad"]:
            least += (n + v) * d * es + (4 * v if case["bias"] else 0)
        return {"bytes": least, "flops": (6 if case["grad"] else 2) * n * d * v}
    least = flops = 0
    for r, c in _shapes(case):
        k, n = min(r, c), max(r, c)
        flops += STEPS * (k * k * n + k * k * k + 2 * k * k * n)  # half of each symmetric product
        least += r * c * (ESIZE[case["x"]] + ESIZE[case["out"]])
        if case["op"] == "step":
            least += r * c * (8 + ESIZE[case["out"]])
    return {"bytes": least, "flops": flops}


# ------------------------------------------------------------ 64-bit results
def _exact_loss(st):
    case = st["case"]
    h, w = (st[k].double().requires_grad_(case["grad"]) for k in ("hidden", "weight"))
    b = torch.zeros((case["actions"],), dtype=torch.float64, device="cuda") if st["bias"] is None else st["bias"].double()
    b.requires_grad_(case["grad"])
    rows = torch.nonzero(st["taken"] >= 0)[:, 0]
    z = torch.addmm(b, h, w.t())
    lse = torch.logsumexp(z, 1)
    nll = torch.zeros((case["rows"],), dtype=torch.float64, device="cuda")
    nll = nll.index_put((rows,), lse[rows] - z[rows, st["taken"][rows].long()])
    loss = torch.dot(nll, st["row_weights"].double()) / case["rows"]
    out = [loss.detach().view(1), nll.detach(), lse.detach()]
    if case["grad"]:
        grads = torch.autograd.grad(loss, [h, w, b])
        out += grads[:2] if st["bias"] is None else grads
    return out


def _exact_orthogonalize(u):
    """p(.. p(x)) on the side of the smaller Gram matrix, x in front or behind."""
    a, b, c = QUINTIC
    x = u / (torch.linalg.matrix_norm(u) + EPS)
    for _ in range(STEPS):
        wide = x.shape[0] <= x.shape[1]
        gram = x @ x.mT if wide else x.mT @ x
        p = gram @ (c * gram)
        p += b * gram
        p.diagonal().add_(a)
        x = p @ x if wide else x @ p
    return x


def exact(case, seed):
    global own
    keep, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = keep
    if case["op"] == "loss":
        return _exact_loss(st)
    if case["op"] == "orthogonalize":
        return [_exact_orthogonalize(x.double()) for x in st["x"]]
    weights, momenta = [], []
    for g, m, w in zip(st["x"], st["m"], st["w"]):
        m = g.double() + MOMENTUM * m.double()
        o = _exact_orthogonalize(g.double() + MOMENTUM * m)
        rate = LR * max(1.0, w.shape[0] / w.shape[1]) ** 0.5
        weights.append(w.double() - LR * DECAY * w.double() - rate * o)
        momenta.append(m)
    return weights + momenta
