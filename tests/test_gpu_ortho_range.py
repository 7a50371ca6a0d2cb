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


@pytest.mark.parametrize("shape", [(100, 100), (400, 300)])
def test_decay_alone_is_rounded_once(m, shape):
    """Without a gradient the weights shrink by lr weight_decay, here 1e-6: as a binary32 factor 1 - 1e-6 is off by
    a hundredth of that decay, step after step."""
    import torch
    g = torch.Generator().manual_seed(3)
    w = torch.randn(shape, generator=g).to(dev())
    x, mom = torch.zeros(shape, device=dev()), torch.zeros(shape, device=dev())
    s = m.MatrixSet([x], [w], [mom])
    ws = m.orthogonalize_workspace(s)
    was = _host(w)
    m.muon_step(s, ws, 1e-4, weight_decay=1e-2)
    sync()
    want = was * (1.0 - 1e-6)
    # half a step, and that of lr weight_decay itself and of its product
    assert np.all(np.abs(_host(w) - want) <= 2.0 ** -24 * np.abs(want) + 2.0 ** -23 * 1e-6 * np.abs(was))


@pytest.mark.parametrize("decay", [0.0, 0.5])
@pytest.mark.parametrize("shape", [(40, 60), (200, 180)])
def test_infinite_weights_stay_infinite(m, shape, decay):
    import torch
    g = torch.Generator().manual_seed(4)
    clean = torch.randn(shape, generator=g).to(dev())
    got = clean.clone()
    got[3, 5], got[7, 9] = np.inf, -np.inf
    for w in (clean, got):
        x, mom = _update(2, shape, "float32"), torch.zeros(shape, device=dev())
        s = m.MatrixSet([x], [w], [mom])
        m.muon_step(s, m.orthogonalize_workspace(s), 0.1, weight_decay=decay)
    sync()
    assert got[3, 5].item() == np.inf and got[7, 9].item() == -np.inf
    got[3, 5], got[7, 9] = clean[3, 5], clean[7, 9]
    assert torch.equal(got, clean)


def test_more_than_2_to_31_elements(m):
    """65536 x 32784 of one sign pattern, u v^T: one step gives p(1) of it, every element of one size.  Sums of up to
    65536 equal terms, 16 to an addition, are off by up to 4096 half steps of binary32, operands by one of binary16."""
    import torch
    r, c = 65536, 32784
    g = torch.Generator(device=dev()).manual_seed(5)
    sign = lambda n: torch.where(torch.rand(n, generator=g, device=dev()) < 0.5, -1.0, 1.0)  # noqa: E731
    u, v = sign(r), sign(c)
    x = torch.empty(r, c, dtype=torch.bfloat16, device=dev())
    torch.mul(u[:, None].bfloat16(), v[None, :].bfloat16(), out=x)
    out = torch.full((r, c), 3.0, dtype=torch.bfloat16, device=dev())
    s = m.MatrixSet([x], [out])
    ws = m.orthogonalize_workspace(s)
    m.orthogonalize(s, ws, steps=1)
    sync()
    want = (ref.A + ref.B + ref.C) / np.sqrt(r * c)
    # each of the three products and of the four operands moves p(1) = A + B + C by up to its coefficients' sum
    tol = (abs(ref.A) + abs(ref.B) + abs(ref.C)) / (ref.A + ref.B + ref.C) * (4 * 2.0 ** -11 + 3 * 2.0 ** -12) + HALF["bfloat16"]
    for a in range(0, r, 4096):
        got = out[a:a + 4096].float() * u[a:a + 4096, None] * v
        lo, hi = float(got.min()), float(got.max())
        assert want * (1 - tol) <= lo and hi <= want * (1 + tol), (a, lo, hi, want)
