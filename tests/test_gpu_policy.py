"""GPU parity of the policy loss and its gradients against the fp64 oracle.

Bounds, element by element, from the operations the kernels make (U = 2^-24 binary32's
half step; the terms' absolute values are summed by the oracle's inputs):
* a logit is an exact sum of dim products rounded at most dim + 8 times, (dim + 8) U
  sum |h w|; binary32 operands are held to 2^-22 each, 2^-21 sum |h w| more, and no better than
  2^-38 of the row's largest element times that of W; then its product with log2(e), the
  bias and the maximum's subtraction, 8 U (|z| + |bias| + |lse|);
* lse and nll carry the largest of their row's logit errors twice, and 16 U (1 + |lse|)
  for the sum, the logarithm and the product with ln 2;
* the exponential instruction gives 0 for results below binary32's smallest normal number, so p
  is off by up to 2^-126 whatever its size (for p = 2^x, x < -126, all of p is lost), taken
  as 2^-125 |scale w| for the subnormal products with it;
* G carries p |w| times the two errors, and one rounding: 2^-8, 2^-11 (with half a smallest
  step of 2^-25 2^-13 of the largest weight) or two planes' 2^-16 and 2^-22;
* dH and dW: G's errors times the other operand, the sum's own (K + 8) U sum |G x|, for
  binary32 2^-21 of it for the operand, and the result's rounding (half a smallest step
  where it is subnormal)."""
import math

import numpy as np
import pytest

from oracle import policy as ref
from tests.gpu_util import dev, sync

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"float32": (2.0 ** -24, 2.0 ** -150), "bfloat16": (2.0 ** -8, 2.0 ** -134), "float16": (2.0 ** -11, 2.0 ** -25)}
TYPES = ["bfloat16", "float16", "float32"]


@pytest.fixture(scope="module")
def m():
    import offline_rl_step_amd as m
    return m


def _case(seed, rows, dim, actions, dtype, bias=True, weights=True, off=0.1, ld=0, shift=0):
    """Device inputs; ld and shift: extra columns of the buffers that hold hidden and weight,
    and the elements their first column lies in."""
    import torch
    g = torch.Generator().manual_seed(seed)
    t = getattr(torch, dtype)
    c = dict(dtype=dtype, keep=[])

    def matrix(r, x):
        buf = torch.full((r, dim + ld + shift), 777.0, dtype=t)
        buf[:, shift:shift + dim] = x.to(t)
        buf = buf.to(dev())
        c["keep"].append(buf)
        return buf[:, shift:shift + dim]

    c["hidden"] = matrix(rows, torch.relu(torch.randn(rows, dim, generator=g)) * torch.exp2(torch.randn(dim, generator=g) * 0.5))
    c["weight"] = matrix(actions, torch.randn(actions, dim, generator=g) * (2.0 / math.sqrt(dim)))
    taken = torch.randint(0, actions, (rows,), generator=g, dtype=torch.int32)
    c["bias"] = None
    if bias:
        b = torch.randn(actions, generator=g) * 0.5
        allowed = b.clone()
        b[torch.rand(actions, generator=g) < 0.1] = -math.inf
        b[taken.long()] = allowed[taken.long()]
        c["bias"] = b.to(dev())
    if off and rows > 1:
        taken[torch.rand(rows, generator=g) < off] = -1
    c["taken"] = taken.to(dev())
    c["row_weights"] = (torch.rand(rows, generator=g) * 0.9 + 0.1).to(dev()) if weights else None
    return c


def _run(m, c, grad=True, scale=None, flags=None, stream=None, ws=None):
    import torch
    h, w = c["hidden"], c["weight"]
    rows, actions = h.shape[0], w.shape[0]
    new = lambda *s: torch.full(s, -7.0, device=dev())  # noqa: E731
    if ws is None:
        ws = m.policy_loss_workspace(rows, actions, h.shape[1], h.dtype, grad=grad)
        ws.fill_(0xFF)  # NaN
    out = dict(nll=new(rows), lse=new(rows), loss=new(1))
    kw = dict(bias=c["bias"], row_weights=c["row_weights"], scale=scale, stream=stream)
    m.policy_loss(h, w, c["taken"], out["nll"], out["lse"], ws, out_loss=out["loss"], flags=flags, **kw)
    if grad:
        out.update(dh=torch.full_like(h, -7.0, memory_format=torch.contiguous_format),
                   dw=torch.full_like(w, -7.0, memory_format=torch.contiguous_format), db=new(actions))
        m.policy_loss_grad(h, w, c["taken"], out["lse"], ws, d_hidden=out["dh"], d_weight=out["dw"], d_bias=out["db"], **kw)
    return out


def _host(t):
    return None if t is None else t.detach().double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def _near(got, want, bound, what):
    got = _host(got)
    fine = np.isfinite(want)
    assert np.array_equal(fine, np.isfinite(got)), what
    assert np.array_equal(got[~fine], want[~fine]) or np.all(np.isnan(got[~fine]) == np.isnan(want[~fine])), what
    off = np.abs(got[fine] - want[fine])
    over = off - np.broadcast_to(bound, want.shape)[fine]
    assert over.size == 0 or over.max() <= 0, (what, float(over.max()), float(off.max()))


def _check(c, out, scale=None):
    h, w, b = _host(c["hidden"]), _host(c["weight"]), _host(c["bias"])
    taken, rw, dtype = _host(c["taken"]), _host(c["row_weights"]), c["dtype"]
    rows, dim = h.shape
    actions = w.shape[0]
    scale = 1.0 / rows if scale is None else scale
    kw = dict(bias=b, row_weights=rw, scale=scale)
    loss, nll, lse = ref.loss(h, w, taken, **kw)
    there, on = ref.on_rows(taken, actions, rw)
    ah, aw = np.abs(h), np.abs(w)
    with np.errstate(invalid="ignore"):
        z = ref.logits(h, w, b)
        ez = (dim + 8) * U * (ah @ aw.T) + 8 * U * np.where(np.isfinite(z), np.abs(z) + 1, 0)
        if b is not None:
            ez += 8 * U * np.where(np.isfinite(b), np.abs(b), 0)[None, :]
        if dtype == "float32":
            ez += 2.0 ** -21 * (ah @ aw.T) + 2.0 ** -37 * dim * ah.max(1, initial=0)[:, None] * aw.max()
        ez += 8 * U * np.where(np.isfinite(lse), np.abs(lse), 0)[:, None]
    err = ez.max(axis=1) + 16 * U * (1 + np.where(np.isfinite(lse), np.abs(lse), 0))
    _near(out["lse"], lse, err, "lse")
    _near(out["nll"], nll, 2 * err, "nll")
    wn = np.ones(rows) if rw is None else rw
    if math.isfinite(loss):
        assert abs(float(out["loss"]) - loss) <= abs(scale) * np.sum((np.abs(wn) * 2 * err)[on]) + U * 1.01 * abs(loss)
    if "dh" not in out:
        return
    g = ref.logit_grads(h, w, taken, **kw)
    two = rows <= 64 or dtype == "float32"
    half = (2.0 ** -22 if dtype != "bfloat16" else 2.0 ** -16) if two else HALF[dtype][0]
    p = np.abs(g) + np.zeros_like(g)
    p[np.arange(rows)[on], taken[on]] = np.abs(scale * wn[on])  # at most
    flushed = 2.0 ** -125 * np.abs(scale * np.where(on, wn, 0))[:, None]
    eg = p * (ez + err[:, None] + 4 * U) + half * np.abs(g) + flushed
    if dtype != "bfloat16":
        eg = eg + abs(scale) * np.abs(wn[on]).max(initial=0) * 2.0 ** -38 * (on[:, None] * 1.0)
    eg[~on] = 0
    k = 2.0 ** -21 if dtype == "float32" else 0.0
    ag = np.abs(g) + eg
    hh = np.where(on[:, None], ah, 0)
    rel, least = HALF[dtype]
    dh, dw, db = ref.grads(h, w, taken, **kw)
    bound = eg @ aw + ((actions + 8) * U + k) * (ag @ aw)
    _near(out["dh"], dh, bound + rel * (np.abs(dh) + bound) + least, "d_hidden")
    bound = eg.T @ hh + ((rows + 8) * U + k) * (ag.T @ hh)
    _near(out["dw"], dw, bound + rel * (np.abs(dw) + bound) + least, "d_weight")
    # not rounded to the inputs' type
    e = p * (ez + err[:, None] + 4 * U) + flushed
    e[~on] = 0
    _near(out["db"], db, e.sum(0) + (rows + 8) * U * ag.sum(0) + U * np.abs(db) + 2.0 ** -149, "d_bias")


SIZES = [(1, 1, 1), (1, 8, 2), (1, 64, 1000), (2, 7, 3), (3, 65, 129), (16, 64, 64), (17, 33, 300), (64, 200, 257),
         (65, 40, 300), (129, 65, 257), (130, 512, 9), (300, 128, 1), (257, 24, 1030), (1000, 1, 40), (40, 1100, 77)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,dim,actions", SIZES)
def test_loss_and_gradients(m, rows, dim, actions, dtype):
    c = _case(rows * 7 + dim, rows, dim, actions, dtype)
    out = _run(m, c)
    sync()
    _check(c, out)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,dim,actions", [(5, 12, 70), (140, 40, 300)])
def test_without_bias_and_weights_and_with_a_scale(m, rows, dim, actions, dtype):
    c = _case(5, rows, dim, actions, dtype, bias=False, weights=False, off=0)
    out = _run(m, c, scale=0.37)
    sync()
    _check(c, out, scale=0.37)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("ld,shift", [(8, 0), (3, 0), (16, 8), (5, 3), (0, 1)])
@pytest.mark.parametrize("rows", [3, 133])
def test_strided_and_unaligned_matrices(m, rows, ld, shift, dtype):
    import torch
    c = _case(11, rows, 56, 150, dtype, ld=ld, shift=shift)
    out = _run(m, c)
    # results into columns of wider buffers, what lies beside them untouched
    gh = torch.full((rows, 70), 3.0, dtype=c["hidden"].dtype, device=dev())
    gw = torch.full((150, 70), 3.0, dtype=c["hidden"].dtype, device=dev())
    ws = m.policy_loss_workspace(rows, 150, 56, c["hidden"].dtype, grad=True)
    m.policy_loss_grad(c["hidden"], c["weight"], c["taken"], out["lse"], ws, bias=c["bias"], row_weights=c["row_weights"],
                       d_hidden=gh[:, 5:61], d_weight=gw[:, 9:65])
    sync()
    _check(c, out)
    assert torch.equal(gh[:, 5:61], out["dh"]) and torch.equal(gw[:, 9:65], out["dw"])
    assert bool((gh[:, :5] == 3).all()) and bool((gh[:, 61:] == 3).all())
    assert bool((gw[:, :9] == 3).all()) and bool((gw[:, 65:] == 3).all())
    for buf in c["keep"]:
        assert bool((buf[:, :shift] == 777).all()) and bool((buf[:, shift + 56:] == 777).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [9, 200])
def test_rows_that_are_off_hold_anything(m, rows, dtype):
    """NaN, infinities and huge values in the hidden rows without an action, or of weight 0, do not
    reach the loss, dW or the other rows."""
    import torch
    c = _case(21, rows, 48, 90, dtype)
    c["taken"][1], c["taken"][2], c["taken"][3], c["taken"][4] = -1, -1, -1, 90
    c["row_weights"][5] = 0.0
    clean = _run(m, c)
    flags = torch.zeros(1, dtype=torch.int32, device=dev())
    c["hidden"][1], c["hidden"][2], c["hidden"][3] = math.nan, math.inf, 6e4
    c["hidden"][5, ::2] = math.nan
    c["row_weights"][1] = math.nan
    out = _run(m, c, flags=flags)
    sync()
    assert flags.item() == m.FLAG_BAD_INDEX
    on = torch.ones(rows, dtype=torch.bool, device=dev())
    on[[1, 2, 3, 5]] = False
    for k in ("nll", "lse", "dh"):
        assert torch.equal(out[k][on], clean[k][on]), k
    assert torch.equal(out["loss"], clean["loss"]) and torch.equal(out["dw"], clean["dw"]) and torch.equal(out["db"], clean["db"])
    assert bool((out["nll"][[1, 2, 3, 4]] == 0).all()) and bool((out["dh"][[1, 2, 3, 4, 5]] == 0).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [4, 150])
def test_actions_of_probability_zero(m, rows, dtype):
    import torch
    c = _case(31, rows, 40, 200, dtype, off=0)
    c["bias"][7] = -math.inf
    c["taken"][2] = 7
    flags = torch.zeros(1, dtype=torch.int32, device=dev())
    out = _run(m, c, flags=flags)
    sync()
    assert out["nll"][2].item() == math.inf and out["loss"].item() == math.inf and flags.item() == m.FLAG_NONFINITE_LOSS
    _check(c, out)
    # every action forbidden
    c["bias"].fill_(-math.inf)
    out = _run(m, c)
    sync()
    assert bool((out["lse"] == -math.inf).all()) and bool((out["nll"] == math.inf).all())
    _check(c, out)
    c["row_weights"].fill_(0.0)
    out = _run(m, c)
    sync()
    assert out["loss"].item() == 0 and bool((out["dh"] == 0).all()) and bool((out["dw"] == 0).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [4, 150])
def test_non_finite_rows_stay_with_themselves(m, rows, dtype):
    import torch
    c = _case(41, rows, 40, 200, dtype, off=0)
    clean = _run(m, c)
    c["hidden"][1, 3] = math.nan
    flags = torch.zeros(1, dtype=torch.int32, device=dev())
    out = _run(m, c, flags=flags)
    sync()
    assert math.isnan(out["loss"].item()) and flags.item() == m.FLAG_NONFINITE_LOSS
    others = torch.arange(rows, device=dev()) != 1
    for k in ("nll", "lse", "dh"):
        assert torch.equal(out[k][others], clean[k][others]), k
    assert math.isnan(out["nll"][1].item()) and bool(out["dh"][1].isnan().all())


@pytest.mark.parametrize("dtype", TYPES)
def test_large_logits(m, dtype):
    """Sharp distributions: one action takes nearly all."""
    import torch
    c = _case(51, 100, 64, 300, dtype)
    c["weight"].copy_((c["weight"].float() * 40).to(c["weight"].dtype))
    out = _run(m, c)
    sync()
    assert out["lse"].max().item() > 100
    _check(c, out)


@pytest.mark.parametrize("dtype", TYPES)
def test_several_pieces_of_the_actions(m, dtype):
    """16384 rows take the actions in pieces; the reference is binary64 on the device."""
    import torch
    rows, dim, actions = 16384, 24, 17011
    c = _case(61, rows, dim, actions, dtype)
    out = _run(m, c)
    sync()
    h, w = c["hidden"].double(), c["weight"].double()
    z = torch.addmm(c["bias"].double(), h, w.t())
    lse = torch.logsumexp(z, 1)
    on = c["taken"] >= 0
    at = c["taken"].clamp(min=0).long()[:, None]
    nll = torch.where(on, lse - z.gather(1, at)[:, 0], 0.0)
    wn = torch.where(on, c["row_weights"].double(), 0.0) / rows
    g = z.sub_(lse[:, None]).exp_()
    g.scatter_add_(1, at, torch.full_like(at, -1, dtype=torch.float64))
    g *= wn[:, None]
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())  # noqa: E731
    # norm-wise: two logit errors and the logarithm's, 64 U; G's rounding and the result's
    assert rel(out["lse"], lse) <= 64 * U and rel(out["nll"], nll) <= 64 * U and rel(out["loss"], (wn * nll).sum().view(1)) <= 64 * U
    tol = {"bfloat16": 2 * 2.0 ** -8, "float16": 2 * 2.0 ** -11, "float32": 2.0 ** -20}[dtype]
    # results below the type's normal numbers (binary16's start at 6e-5) are rounded by up to half its smallest step
    # each, 2^-25 sqrt(n) of n elements' norm
    for key, want in (("dh", g @ w), ("dw", g.t() @ h)):
        off = float((out[key].double() - want).norm())
        assert off <= tol * float(want.norm()) + HALF[dtype][1] * math.sqrt(want.numel()), key
    assert rel(out["db"], g.sum(0)) <= 2.0 ** -19


def test_results_repeat_and_other_streams(m):
    import torch
    c = _case(71, 300, 72, 1500, "bfloat16")
    first = _run(m, c)
    side = torch.cuda.Stream()
    sync()
    busy = torch.empty(1 << 26, device=dev())
    for rep in range(3):
        busy.fill_(rep)
        got = _run(m, c)
        other = _run(m, c, stream=side)
        sync()
        for k in first:
            assert torch.equal(first[k], got[k]), k
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = _run(m, c)
    sync()
    for k in first:
        assert torch.equal(first[k], other[k]), k


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [2, 300])
def test_graph_replays(m, rows, dtype):
    import torch
    c = _case(81, rows, 72, 600, dtype)
    ws = m.policy_loss_workspace(rows, 600, 72, c["hidden"].dtype, grad=True)
    _run(m, c, ws=ws)
    sync()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _run(m, c, ws=ws)
    for rep in range(4):
        d = _case(90 + rep, rows, 72, 600, dtype)
        for k in ("hidden", "weight", "taken", "bias", "row_weights"):
            c[k].copy_(d[k])
        graph.replay()
        sync()
        eager = _run(m, c)
        sync()
        for k in out:
            assert torch.equal(out[k], eager[k]), (rep, k)


def test_gradient_against_differences(m):
    """Directional derivatives of the loss itself, in binary32: the loss's error 2^-22 over the step, and
    the second difference's quarter of the step's change."""
    import torch
    c = _case(101, 64, 32, 200, "float32")
    out = _run(m, c)
    g = torch.Generator().manual_seed(5)
    h, w, b = _host(c["hidden"]), _host(c["weight"]), _host(c["bias"])
    rw, taken = _host(c["row_weights"]), _host(c["taken"])
    for key, grad in (("hidden", "dh"), ("weight", "dw"), ("bias", "db")):
        d = torch.randn(c[key].shape, generator=g).to(dev())
        keep = c[key].clone()
        got = []
        step = 2.0 ** -7
        for s in (step, -step):
            c[key].copy_(keep + s * d)
            got.append(float(_run(m, c, grad=False)["loss"]))
        c[key].copy_(keep)
        want = float((out[grad].double() * d.double()).sum())
        x = {"hidden": h, "weight": w, "bias": b}
        exact = []
        for s in (step, -step):
            y = dict(x)
            y[key] = x[key] + s * d.double().cpu().numpy()
            exact.append(ref.loss(y["hidden"], y["weight"], taken, y["bias"], rw, 1 / 64)[0])
        curve = abs((exact[0] - exact[1]) / (2 * step) - want)  # what the oracle's own difference is off
        assert abs((got[0] - got[1]) / (2 * step) - want) <= curve + 2 * 2.0 ** -20 * abs(exact[0]) / (2 * step), key


def test_single_gradients_equal_the_three_together(m):
    import torch
    c = _case(111, 200, 40, 500, "bfloat16")
    out = _run(m, c)
    ws = m.policy_loss_workspace(200, 500, 40, torch.bfloat16, grad=True)
    for key, arg in (("dh", "d_hidden"), ("dw", "d_weight"), ("db", "d_bias")):
        alone = torch.zeros_like(out[key])
        m.policy_loss_grad(c["hidden"], c["weight"], c["taken"], out["lse"], ws, bias=c["bias"], row_weights=c["row_weights"],
                           **{arg: alone})
        sync()
        assert torch.equal(alone, out[key]), key


def test_binding_refuses(m):
    import torch
    c = _case(121, 6, 16, 20, "bfloat16")
    ws = m.policy_loss_workspace(6, 20, 16, torch.bfloat16, grad=True)
    f = torch.zeros(6, device=dev())
    ok = dict(hidden=c["hidden"], weight=c["weight"], taken=c["taken"], out_nll=f, out_lse=f.clone(), workspace=ws)
    m.policy_loss(**ok)
    for bad, word in ((dict(weight=c["weight"].float()), "weight"), (dict(hidden=c["hidden"].t()), "neighbouring columns"),
                      (dict(taken=c["taken"].long()), "int32"), (dict(taken=c["taken"][:5]), "6 elements"),
                      (dict(out_nll=f[:5]), "out_nll"), (dict(bias=f), "bias"), (dict(row_weights=f.double()), "row_weights"),
                      (dict(weight=c["weight"][:, :8]), "weight"), (dict(workspace=ws.cpu()), "workspace"),
                      (dict(flags=f), "flags"), (dict(out_loss=f.half()), "out_loss")):
        with pytest.raises(ValueError, match=word):
            m.policy_loss(**{**ok, **bad})
    with pytest.raises(m.IqlhError, match="too small"):
        m.policy_loss(**{**ok, "workspace": ws[:64]})
    with pytest.raises(m.IqlhError, match="share memory"):
        m.policy_loss(**{**ok, "out_lse": f})
    grad = dict(hidden=c["hidden"], weight=c["weight"], taken=c["taken"], lse=f, workspace=ws)
    with pytest.raises(m.IqlhError, match="no gradient"):
        m.policy_loss_grad(**grad)
    with pytest.raises(ValueError, match="type of hidden"):
        m.policy_loss_grad(**grad, d_hidden=torch.zeros(6, 16, device=dev()))
    with pytest.raises(ValueError, match="type of weight"):
        m.policy_loss_grad(**grad, d_weight=torch.zeros(20, 16, device=dev()))
