"""Numbers that binary32 does not hold are refused by the policy loss and the orthogonalised step, before any HIP
call."""
import ctypes

import pytest

from tests import test_ortho_cpu as ortho
from tests import test_policy_cpu as policy


@pytest.fixture(scope="module")
def m():
    import offline_rl_step_amd as m
    return m


def test_scales_above_binary32(m):
    for call in (policy._loss, policy._grad):
        for bad in (1e39, -1e300):
            assert call(m, scale=bad) == m.EINVAL and "scale" in m.last_error()


def test_rates_above_binary32(m):
    """The rate times the largest s, 256, and lr weight_decay are binary32 numbers."""
    rc, _, st = ortho._fill(m, [ortho._matrix(m, 100, 30)])
    assert rc == m.OK
    st.d_table = ortho.BASE

    def step(lr, wd, mu=0.9):
        return m._lib_muon_step(ctypes.byref(st), lr, mu, 1, wd, 0, 5, 1e-7, None, ortho.BASE, st.workspace_bytes, None)

    for lr, wd in ((1e300, 0.0), (-2e36, 0.0), (1.0, 1e39), (1e20, 1e20)):
        assert step(lr, wd) == m.EINVAL and "lr" in m.last_error(), (lr, wd, m.last_error())
    assert step(1e36, 1.0, mu=1.0) == m.EINVAL and "mu" in m.last_error()


def test_workspace_has_no_partial_sums_where_products_are_whole(m):
    """8192 rows, 65536 actions, dim 2048 in bfloat16: the copies of hidden and weight, a piece of G of 256 MB, d_hidden
    over the pieces, a part of the bias's gradient, and a few numbers a row; not d_weight's sums in binary32."""
    rows, actions, dim = 8192, 65536, 2048
    rc, n = policy._bytes(m, rows, actions, dim, m.BF16, 1)
    piece = 1 << 14
    assert rc == m.OK
    assert n <= 2 * dim * (rows + actions) + 2 * rows * piece + 4 * rows * dim + 4 * piece * rows // 128 + 64 * rows
    # one piece, d_hidden in one part too
    rows, actions, dim = 1024, 8192, 8192
    rc, n = policy._bytes(m, rows, actions, dim, m.BF16, 1)
    assert rc == m.OK and n <= 2 * dim * (rows + actions) + 2 * rows * actions + 4 * actions * rows // 128 + 64 * rows
