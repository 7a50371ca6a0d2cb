"""Orthogonalised updates of matrices whose norm is far below eps, and the weights' decay."""
import numpy as np
import pytest

from oracle import ortho as ref
from tests.gpu_util import dev, sync
from tests.test_gpu_ortho import HALF, _host, _moved, _ortho, _planes, _t, _update

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import offline_rl_step_amd as m
    return m


@pytest.mark.parametrize("norm,steps", [(1e-9, 5), (1e-13, 5), (1e-17, 5), (1e-25, 5), (1e-13, 12), (1e-17, 19)])
@pytest.mark.parametrize("shape", [(20, 30), (70, 90), (300, 200), (200, 513)])
def test_norms_below_eps(m, shape, norm, steps):
    """With |U| far below eps the result is that much smaller than orthogonal (after many steps it is orthogonal
    again), and as exact relative to its own size as any other."""
    import torch
    for out in ("float32", "bfloat16"):
        u = _update(9, shape, "float32", scale=1.0)
        u = (u.double() * (norm / u.double().norm())).float()
        o = torch.empty(shape, dtype=_t(out), device=dev())
        _ortho(m, [u], [o], steps=steps)
        sync()
        want = ref.orthogonalize(_host(u), steps)
        planes = _planes(m, shape, out)
        n = np.linalg.norm(want)
        off = np.linalg.norm(_host(o) - want)
        assert off <= 2 * _moved(_host(u), planes, want, steps=steps) + HALF[out] * n, (out, off / n)
