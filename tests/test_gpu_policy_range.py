"""Policy loss: rows that are off with weights of any size, operands of many magnitudes.

Binary32 operands of the tile kernels are two binary16 planes behind a power of two that takes the
largest of what shares it to [2^13, 2^14): 22 bits, and no better than half of binary16's smallest step, 2^-25
there, 2^-38 of that largest.  With c[d] the largest |weight| of column d among the actions that are not forbidden:
* logits: hidden[r][d] c[d] shares a row's, weight[v][d] / c[d] an action's, c within a factor of 2, so
  a product is off by up to 2^-36 of the two largest;
* d_hidden: G shares |scale w| of its row, weight[.][d] its column's;
* d_weight: hidden[r][d] w[r] shares its column's, w within a factor of 2.
The other terms as in test_gpu_policy.py."""
import math

import numpy as np
import pytest

from oracle import policy as ref
from tests.gpu_util import dev, sync
from tests.test_gpu_policy import TYPES, U, _case, _check, _host, _near, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import offline_rl_step_amd as m
    return m


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [9, 200])
@pytest.mark.parametrize("weight", [1e9, -1e30])
def test_finite_weights_of_rows_that_are_off(m, rows, dtype, weight):
    """A row without an action adds nothing whatever its weight is: not to the factor that G is held with either."""
    import torch
    c = _case(23, rows, 48, 90, dtype)
    c["taken"][1], c["taken"][4] = -1, 90
    clean = _run(m, c)
    for row in (1, 4):
        c["row_weights"][row] = weight
        out = _run(m, c)
        sync()
        for k in out:
            assert torch.equal(out[k], clean[k]), (k, row)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("rows", [9, 200])
def test_off_rows_next_to_an_infinite_weight(m, rows, dtype):
    """An action whose weights hold minus infinity where hidden is positive has probability 0: nothing of it in
    its weight's and bias's gradients, whatever the rows that are off hold."""
    import torch
    c = _case(27, rows, 48, 90, dtype)
    c["taken"][:3] = torch.tensor([-1, 90, -1], dtype=torch.int32)
    c["taken"][c["taken"] == 17] = 18
    c["bias"].copy_(torch.nan_to_num(c["bias"], neginf=0.0))
    c["hidden"][:, 5] = 1.0
    c["weight"][17, 5] = -math.inf
    out = _run(m, c)
    sync()
    on = c["taken"] >= 0
    on &= c["taken"] < 90
    assert bool(out["lse"][on].isfinite().all()) and math.isfinite(float(out["loss"]))
    assert bool(out["dw"].isfinite().all()) and bool(out["db"].isfinite().all())
    assert bool((out["dw"][17] == 0).all()) and float(out["db"][17]) == 0


def _check_planes(c, out):
    """float32 on the tiles' kernels, element by element."""
    h, w, b, taken, rw = (_host(c[k]) for k in ("hidden", "weight", "bias", "taken", "row_weights"))
    rows, dim = h.shape
    actions, scale = w.shape[0], 1.0 / rows
    kw = dict(bias=b, row_weights=rw, scale=scale)
    loss, nll, lse = ref.loss(h, w, taken, **kw)
    _, on = ref.on_rows(taken, actions, rw)
    ah, aw = np.abs(h), np.abs(w)
    col = aw[np.isfinite(b)].max(0)
    with np.errstate(invalid="ignore", divide="ignore"):
        z = ref.logits(h, w, b)
        ez = (dim + 8) * U * (ah @ aw.T) + 8 * U * np.where(np.isfinite(z), np.abs(z) + 1, 0)
        ez += 8 * U * np.where(np.isfinite(b), np.abs(b), 0)[None, :]
        ez += 2.0 ** -21 * (ah @ aw.T) + 2.0 ** -36 * dim * np.outer((ah * col).max(1), np.where(col > 0, aw / col, 0).max(1))
        ez = np.where(np.isfinite(b)[None, :], ez, 0)
        ez += 8 * U * np.abs(lse)[:, None]
    err = ez.max(axis=1) + 16 * U * (1 + np.abs(lse))
    _near(out["lse"], lse, err, "lse")
    _near(out["nll"], nll, 2 * err, "nll")
    g = ref.logit_grads(h, w, taken, **kw)
    mine = np.where(on, np.abs(scale * rw), 0)[:, None]  # |scale w|
    p = np.abs(g)
    p[np.arange(rows)[on], taken[on]] = mine[on, 0]
    eg = p * (ez + err[:, None] + 4 * U) + 2.0 ** -22 * np.abs(g) + mine * (2.0 ** -38 + 2.0 ** -125)
    eg[:, np.isneginf(b)] = 0
    ag, hh = np.abs(g) + eg, np.where(on[:, None], ah, 0)
    dh, dw, db = ref.grads(h, w, taken, **kw)
    half, least = 2.0 ** -24, 2.0 ** -149
    bound = eg @ aw + ((actions + 8) * U + 2.0 ** -21) * (ag @ aw) + 2.0 ** -38 * ag.sum(1)[:, None] * col
    _near(out["dh"], dh, bound + half * (np.abs(dh) + bound) + least, "d_hidden")
    rel = np.divide(ag, mine, out=np.zeros_like(ag), where=mine > 0).sum(0)
    bound = eg.T @ hh + ((rows + 8) * U + 2.0 ** -21) * (ag.T @ hh) + 2.0 ** -37 * np.outer(rel, (hh * mine).max(0))
    _near(out["dw"], dw, bound + half * (np.abs(dw) + bound) + least, "d_weight")
    e = p * (ez + err[:, None] + 4 * U) + 2.0 ** -125 * mine
    e[:, np.isneginf(b)] = 0
    _near(out["db"], db, e.sum(0) + (rows + 8) * U * ag.sum(0) + U * np.abs(db) + least, "d_bias")


def _spread(c, kind, seed=5):
    import torch
    g = torch.Generator().manual_seed(seed)
    h, w, b, rw = (c[k] for k in ("hidden", "weight", "bias", "row_weights"))
    rows, dim = h.shape
    if kind == "a feature":  # large activations that the head hardly uses
        h[:, 5] *= 2.0 ** 30
        w[:, 5] *= 2.0 ** -30
    elif kind == "features":
        e = torch.exp2(torch.randint(-40, 41, (dim,), generator=g).float()).to(dev())
        h *= e
        w /= e
    elif kind == "an action":  # forbidden, with weights far from the others'
        b[7] = -math.inf
        c["taken"][c["taken"] == 7] = 8
        b[8] = 0.25
        w[7] *= 2.0 ** 30
    elif kind == "unused":  # a feature without weights
        h[:, 5] *= 2.0 ** 40
        w[:, 5] = 0
    elif kind == "padding":  # forbidden actions that hold anything finite
        w[b == -math.inf] *= torch.exp2(torch.randint(-90, 91, (dim,), generator=g).float()).to(dev())
    elif kind == "actions":
        w *= torch.exp2(torch.randint(-30, 1, (w.shape[0], 1), generator=g).float()).to(dev())
    elif kind == "rows":
        h *= torch.exp2(torch.randint(-40, 1, (rows, 1), generator=g).float()).to(dev())
    elif kind == "weights":
        rw *= torch.exp2(torch.randint(-40, 1, (rows,), generator=g).float()).to(dev())
    elif kind == "large":  # products near the largest binary32 values, logits of the usual size
        h *= 2.0 ** 120
        w *= 2.0 ** -120
    elif kind == "small":
        h *= 2.0 ** -100
        w *= 2.0 ** 100
        rw *= 2.0 ** -100


@pytest.mark.parametrize("kind", ["a feature", "features", "unused", "an action", "padding", "actions", "rows", "weights", "large",
                                  "small"])
@pytest.mark.parametrize("rows,dim,actions", [(30, 24, 70), (200, 72, 300), (150, 600, 130)])
def test_float32_of_many_magnitudes(m, rows, dim, actions, kind):
    c = _case(29, rows, dim, actions, "float32")
    _spread(c, kind)
    out = _run(m, c)
    sync()
    _check_planes(c, out)


@pytest.mark.parametrize("kind", ["features", "weights"])
def test_float32_of_many_magnitudes_in_pieces(m, kind):
    """33000 rows take 1900 actions in pieces of 1792."""
    c = _case(63, 33000, 24, 1900, "float32")
    _spread(c, kind)
    out = _run(m, c)
    sync()
    _check_planes(c, out)


def test_no_rows_and_no_actions_are_refused_as_sizes(m):
    import torch
    z = lambda *s: torch.zeros(s, device=dev())  # noqa: E731
    ws = torch.zeros(1 << 16, dtype=torch.uint8, device=dev())
    for rows, actions in ((0, 4), (4, 0)):
        taken = torch.zeros(rows, dtype=torch.int32, device=dev())
        with pytest.raises(m.IqlhError):
            m.policy_loss(z(rows, 8), z(actions, 8), taken, z(rows), z(rows), ws)
        with pytest.raises(m.IqlhError):
            m.policy_loss_grad(z(rows, 8), z(actions, 8), taken, z(rows), ws, d_hidden=z(rows, 8))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,dim,actions", [(1, 8, 2), (7, 33, 400), (65, 40, 300), (200, 72, 3000), (1300, 520, 8200),
                                              (16384, 24, 9001)])
def test_nothing_is_written_behind_the_workspace(m, rows, dim, actions, dtype):
    import torch
    c = _case(33, rows, dim, actions, dtype)
    for grad in (False, True):
        n = m.policy_loss_workspace(rows, actions, dim, c["hidden"].dtype, grad=grad).numel()
        buf = torch.full((n + 4096,), 0x5A, dtype=torch.uint8, device=dev())
        _run(m, c, grad=grad, ws=buf[:n])
        sync()
        assert bool((buf[n:] == 0x5A).all()), grad


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [3, 300])
def test_stream_argument(m, rows, dtype):
    """stream=: the results of the call on a side stream, whose buffers are there before it, are those of the current
    one's, also while that one is busy."""
    import torch
    c = _case(71, rows, 72, 1500, dtype)
    first = _run(m, c)
    side = torch.cuda.Stream()
    sync()
    busy = torch.empty(1 << 26, device=dev())
    kw = dict(bias=c["bias"], row_weights=c["row_weights"])
    for rep in range(3):
        ws = m.policy_loss_workspace(rows, 1500, 72, c["hidden"].dtype, grad=True)
        ws.fill_(0xFF)
        out = {k: torch.full_like(t, -7.0) for k, t in first.items()}
        side.wait_stream(torch.cuda.current_stream())
        busy.fill_(rep)
        m.policy_loss(c["hidden"], c["weight"], c["taken"], out["nll"], out["lse"], ws, out_loss=out["loss"], stream=side, **kw)
        m.policy_loss_grad(c["hidden"], c["weight"], c["taken"], out["lse"], ws, d_hidden=out["dh"], d_weight=out["dw"],
                           d_bias=out["db"], stream=side, **kw)
        sync()
        for k in first:
            assert torch.equal(out[k], first[k]), (rep, k)


@pytest.mark.parametrize("dtype", ["float16", "float32"])
@pytest.mark.parametrize("rows", [3, 20])
def test_more_than_2_to_31_weights(m, rows, dtype):
    """262221 actions of dim 8200: offsets beyond 32 bits in weight, its planes and its gradient.  Only the last
    actions and one in the middle have a bias above the others', so that all of the batch's probability is there."""
    import torch
    dim, actions = 8200, 262221
    t = getattr(torch, dtype)
    g = torch.Generator(device=dev()).manual_seed(3)
    weight = torch.empty(actions, dim, dtype=t, device=dev())
    for a in range(0, actions, 16384):
        weight[a:a + 16384] = torch.randn(weight[a:a + 16384].shape, generator=g, device=dev()) / 64
    hidden = torch.relu(torch.randn(rows, dim, generator=g, device=dev())).to(t)
    far = torch.tensor([131072, *range(actions - 40, actions)], device=dev())
    bias = torch.full((actions,), -60.0, device=dev())
    bias[far] = torch.randn(41, generator=g, device=dev())
    taken = far[torch.randint(0, 41, (rows,), generator=g, device=dev())].int()
    new = lambda *s: torch.full(s, -7.0, device=dev())  # noqa: E731
    nll, lse, loss, db = new(rows), new(rows), new(1), new(actions)
    ws = m.policy_loss_workspace(rows, actions, dim, t, grad=True)
    dh, dw = torch.full_like(hidden, -7.0), torch.full_like(weight, -7.0)
    m.policy_loss(hidden, weight, taken, nll, lse, ws, bias=bias, out_loss=loss)
    m.policy_loss_grad(hidden, weight, taken, lse, ws, bias=bias, d_hidden=dh, d_weight=dw, d_bias=db)
    sync()
    h, w = hidden.double(), weight[far].double()
    z = h @ w.t() + bias[far].double()
    want = torch.logsumexp(z, 1)  # the others add below e^-50
    at = (far[None, :] == taken[:, None]).double()
    # dim + 8 binary32 roundings of the terms, of sign at random: 2^-18 of |z| and of the largest term sizes
    tol = 2.0 ** -18 * (1 + float(z.abs().max()))
    assert float((lse.double() - want).abs().max()) <= tol
    assert float((nll.double() - (want - (z * at).sum(1))).abs().max()) <= 2 * tol
    gr = (torch.exp(z - want[:, None]) - at) / rows
    rel = {"float16": 2.0 ** -9, "float32": 2.0 ** -16}[dtype]
    for got, ref64 in ((dh, gr @ w), (dw[far], gr.t() @ h), (db[far], gr.sum(0))):
        assert float((got.double() - ref64).norm()) <= (rel + tol) * float(ref64.norm())
    others = torch.ones(actions, dtype=torch.bool, device=dev())
    others[far] = False
    assert float(db[others].abs().max()) < 1e-20
    for a in range(0, actions, 16384):
        rows_there = others[a:a + 16384]
        assert float(dw[a:a + 16384][rows_there].abs().max()) < 1e-7


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,actions", [(1 << 24, 3), (1 << 24, 17), (1, 1 << 24), (5, 1 << 24), (70, 3000000)])
def test_the_most_rows_and_actions(m, rows, actions, dtype):
    """Up to 2^24 of each, against binary64 on the device, norm-wise: the types' rounding of G and the result, and
    2^-16 for binary32 sums of 2^24 terms in parts of thousands."""
    import torch
    dim = 8
    c = _case(35, rows, dim, actions, dtype, off=0.1 if rows > 5 else 0)
    out = _run(m, c)
    sync()
    h, w, b, taken = c["hidden"].double(), c["weight"].double(), c["bias"].double(), c["taken"]
    on = taken >= 0
    wn = torch.where(on, c["row_weights"].double(), 0.0) / rows
    nll, lse = torch.zeros(rows, dtype=torch.float64, device=dev()), torch.zeros(rows, dtype=torch.float64, device=dev())
    dh, dw, db = torch.zeros_like(h), torch.zeros_like(w), torch.zeros_like(b)
    step = max(1, (1 << 27) // actions)
    for r in range(0, rows, step):
        s = slice(r, min(r + step, rows))
        z = torch.addmm(b, h[s], w.t())
        lse[s] = torch.logsumexp(z, 1)
        at = taken[s].clamp(min=0).long()[:, None]
        nll[s] = torch.where(on[s], lse[s] - z.gather(1, at)[:, 0], 0.0)
        g = z.sub_(lse[s][:, None]).exp_()
        g.scatter_add_(1, at, torch.full_like(at, -1, dtype=torch.float64))
        g *= wn[s][:, None]
        dh[s] = g @ w
        dw += g.t() @ h[s]
        db += g.sum(0)
    off = lambda a, b: float((a.double() - b).norm() / b.norm())  # noqa: E731
    assert off(out["lse"], lse) <= 2.0 ** -20 and off(out["nll"], nll) <= 2.0 ** -20
    assert off(out["loss"], (wn * nll).sum().view(1)) <= 2.0 ** -20
    tol = {"bfloat16": 2 * 2.0 ** -8, "float16": 2 * 2.0 ** -11, "float32": 0.0}[dtype] + 2.0 ** -16
    least = {"bfloat16": 0.0, "float16": 2.0 ** -25, "float32": 0.0}[dtype]  # half of the smallest step, each element's
    for key, want in (("dh", dh), ("dw", dw)):
        assert float((out[key].double() - want).norm()) <= tol * float(want.norm()) + least * math.sqrt(want.numel()), key
    assert off(out["db"], db) <= 2.0 ** -16


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("rows,actions", [(300, 12), (30, 200), (200, 300)])
@pytest.mark.parametrize("scale", [2.0 ** -118, -1e-30, 1e30])
def test_scales_far_from_one(m, rows, actions, dtype, scale):
    """G of a small scale is not below what the products take."""
    c = _case(37, rows, 40, actions, dtype)
    out = _run(m, c, scale=scale)
    sync()
    _check(c, out, scale)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [9, 200])
def test_biases_of_the_lowest_value_forbid(m, rows, dtype):
    """A bias of binary32's lowest value is that of a forbidden action, in the loss, the gradients and where it is
    taken all the same."""
    import torch
    for actions in (12, 200):
        c = _case(43, rows, 40, actions, dtype, off=0)
        c["taken"][3] = 5
        got = []
        for low in (-math.inf, torch.finfo(torch.float32).min):
            c["bias"][c["bias"] < -1e30] = low
            c["bias"][5] = low
            got.append(_run(m, c))
        sync()
        assert got[0]["nll"][3].item() == math.inf
        for k in got[0]:
            assert torch.equal(got[0][k], got[1][k]), (actions, k)


@pytest.mark.parametrize("rows", [30, 20000])
def test_a_forbidden_action_that_is_taken_has_its_weights_in_d_hidden(m, rows):
    """float32: its row's d_hidden is -scale w of its weights (and what the other actions add), however large they are
    beside the others'; the loss is infinite."""
    import torch
    c = _case(45, rows, 24, 70, "float32")
    last = int((c["taken"] >= 0).nonzero()[-1])
    c["bias"][7] = -math.inf
    c["taken"][c["taken"] == 7] = 8
    c["bias"][8] = 0.25
    c["taken"][last] = 7
    c["weight"][7] *= 2.0 ** 60
    out = _run(m, c)
    sync()
    assert out["loss"].item() == math.inf and out["nll"][last].item() == math.inf
    want = -c["weight"][7].double() * c["row_weights"][last].double() / rows
    # G and the weight to 2^-22 each, the result's rounding
    assert bool(((out["dh"][last].double() - want).abs() <= 2.0 ** -20 * want.abs()).all())
