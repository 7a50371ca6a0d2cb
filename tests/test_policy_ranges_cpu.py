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
