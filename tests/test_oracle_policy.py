"""The policy loss oracle against closed forms, torch autograd in binary64 and
central differences."""
import math

import numpy as np
import pytest
import torch

from oracle import policy as ref


def _case(seed, rows=7, dim=5, actions=11):
    g = np.random.default_rng(seed)
    return dict(hidden=g.normal(size=(rows, dim)), weight=g.normal(size=(actions, dim)),
                taken=g.integers(0, actions, rows), bias=g.normal(size=actions),
                row_weights=g.uniform(0.1, 1.0, rows), scale=1.0 / rows)


def test_uniform_logits_and_a_hand_worked_row():
    loss, nll, lse = ref.loss(np.zeros((3, 4)), np.zeros((8, 4)), [0, 3, 7])
    assert np.allclose(nll, math.log(8)) and np.allclose(lse, math.log(8)) and math.isclose(loss, 3 * math.log(8))
    z = np.log([1.0, 2.0, 5.0])
    _, nll, lse = ref.loss([[1.0]], z[:, None], [2])
    assert math.isclose(lse[0], math.log(8.0)) and math.isclose(nll[0], math.log(8 / 5))
    g = ref.logit_grads([[1.0]], z[:, None], [2], row_weights=[0.5], scale=4.0)
    assert np.allclose(g, 2.0 * np.array([[1 / 8, 2 / 8, 5 / 8 - 1]]))


@pytest.mark.parametrize("seed", range(4))
def test_against_autograd(seed):
    c = _case(seed)
    c["taken"][0] = -1
    t = {k: torch.tensor(c[k], requires_grad=True) for k in ("hidden", "weight", "bias")}
    z = t["hidden"] @ t["weight"].T + t["bias"]
    nll = torch.nn.functional.cross_entropy(z[1:], torch.tensor(c["taken"][1:]), reduction="none")
    loss = (nll * torch.tensor(c["row_weights"][1:])).sum() * c["scale"]
    loss.backward()
    got, got_nll, lse = ref.loss(**c)
    assert math.isclose(got, loss.item(), rel_tol=1e-12)
    assert np.allclose(got_nll[1:], nll.detach().numpy(), rtol=1e-12) and got_nll[0] == 0
    assert np.allclose(lse, torch.logsumexp(z, 1).detach().numpy(), rtol=1e-12)
    for x, k in zip(ref.grads(**c), ("hidden", "weight", "bias")):
        assert np.allclose(x, t[k].grad.numpy(), rtol=1e-11, atol=1e-14), k


def test_central_differences():
    c = _case(9, rows=3, dim=4, actions=6)
    for got, k in zip(ref.grads(**c), ("hidden", "weight", "bias")):
        for at in np.ndindex(c[k].shape):
            both = []
            for h in (1e-5, -1e-5):
                x = c[k].copy()
                x[at] += h
                both.append(ref.loss(**{**c, k: x})[0])
            assert abs((both[0] - both[1]) / 2e-5 - got[at]) < 1e-9


def test_rows_and_actions_that_are_off():
    c = _case(3)
    c["bias"][4] = -np.inf
    c["taken"][:] = 1
    c["taken"][2] = 4
    loss, nll, _ = ref.loss(**c)
    assert nll[2] == np.inf and loss == np.inf
    c["row_weights"][2] = 0.0
    c["taken"][5] = 99
    c["hidden"][5] = np.nan
    loss, nll, _ = ref.loss(**c)
    assert math.isfinite(loss) and nll[5] == 0
    dh, dw, db = ref.grads(**c)
    assert np.all(dh[2] == 0) and np.all(dw[4] == 0) and db[4] == 0 and np.all(np.isfinite(dw)) and np.all(dh[5] == 0)
    c["bias"][:] = -np.inf
    _, nll, lse = ref.loss(**c)
    assert lse[0] == -np.inf and nll[0] == np.inf
    g = ref.logit_grads(**c)
    assert g[0, 1] == -c["row_weights"][0] * c["scale"] and np.count_nonzero(g[0]) == 1
