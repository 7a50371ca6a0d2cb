"""Policy loss: rows that are off, whatever their weights are."""
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
