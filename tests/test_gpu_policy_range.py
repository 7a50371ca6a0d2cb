"""Policy loss: rows that are off, whatever their weights are."""
import math

import pytest

from tests.gpu_util import sync
from tests.test_gpu_policy import TYPES, _case, _run

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
