"""The oracle of orthogonalised updates against the singular value
decomposition and closed forms."""
import math

import numpy as np
import pytest

from oracle import ortho as ref


@pytest.mark.parametrize("shape", [(1, 1), (1, 5), (6, 1), (7, 7), (5, 12), (12, 5), (40, 33)])
@pytest.mark.parametrize("steps", [1, 5])
def test_singular_values_go_through_the_polynomial(shape, steps):
    u = np.random.default_rng(shape[0] * 100 + shape[1]).normal(size=shape)
    p, s, q = np.linalg.svd(u, full_matrices=False)
    want = p @ np.diag(ref.scalar(s / (np.linalg.norm(u) + 1e-7), steps)) @ q
    assert np.allclose(ref.orthogonalize(u, steps), want, rtol=0, atol=1e-12 * 4 ** steps)


def test_five_steps_take_singular_values_near_one():
    s = np.geomspace(0.01, 1.0, 1000)
    y = ref.scalar(s)
    assert 0.67 < y.min() and y.max() < 1.21
    assert ref.scalar(1e-6) == pytest.approx(ref.A ** 5 * 1e-6, rel=1e-6)


def test_the_bounds_that_the_operand_scale_rests_on():
    s = np.linspace(0.0, 1.0, 100001)
    top = (ref.A * s + ref.B * s ** 3 + ref.C * s ** 5).max()
    assert top < 1.2025
    s = np.linspace(0.0, 1.2025, 100001)
    y = ref.A * s + ref.B * s ** 3 + ref.C * s ** 5
    assert 0 <= y.min() and y.max() < 1.2025
    t = s * s
    assert np.abs(ref.B * t + ref.C * t * t).max() < 2.81


def test_zeros_and_scale():
    assert np.all(ref.orthogonalize(np.zeros((3, 4))) == 0)
    u = np.random.default_rng(1).normal(size=(4, 6))
    assert np.allclose(ref.orthogonalize(u), ref.orthogonalize(u * 1e6), atol=1e-4)


def test_a_step_on_known_values():
    w, m = ref.muon([[2.0]], [[1.0]], [[3.0]], 0.5, mu=0.5, weight_decay=0.1)
    assert m[0, 0] == 3.5 and math.isclose(w[0, 0], 0.95 * 2 - 0.5 * ref.scalar(4.75 / (4.75 + 1e-7)), rel_tol=1e-12)
    w, m = ref.muon([[2.0]], [[1.0]], [[-3.0]], 0.5, mu=0.5, nesterov=False, weight_decay=0.0)
    assert m[0, 0] == -2.5 and w[0, 0] > 2
    assert ref.rate(1.0, (8, 2)) == 2.0 and ref.rate(1.0, (2, 8)) == 1.0 and ref.rate(1.0, (25, 4), ref.RMS) == 1.0
    assert ref.muon([[1.0]], [[0.0]], [[np.nan]], 0.1)[1] is None
