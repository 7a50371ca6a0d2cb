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
