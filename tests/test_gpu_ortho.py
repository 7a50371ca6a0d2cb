"""GPU parity of orthogonalised updates and of the step that uses them against
the fp64 oracle.

How far a result may be off is what roundings of the operands make of it, taken from
the oracle itself: its operands and sums are moved by u of their size with random signs, and
the kernel, whose roundings are at most u each, may be off by twice the largest move of
several draws, norm-wise, and its elements by ten times that of their root mean square (the
errors of a million elements stay within 5.5 of their deviations; a misplaced element is
off by about one).  u = 2^-11 for binary16 operands (half a step of 2^-11, and the sum's); two
planes are off by 2^-23 and their sums by 2^-24 for each of at most sqrt(K / 8) additions,
2^-20 up to K = 4096.  Then the result's own rounding: half a step, 2^-24, 2^-8 or 2^-11."""
import math

import numpy as np
import pytest

from oracle import ortho as ref
from tests.gpu_util import dev, sync

pytestmark = pytest.mark.gpu

HALF = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}
NOISE = {"one": 2.0 ** -11, "two": 2.0 ** -20}


@pytest.fixture(scope="module")
def m():
    import offline_rl_step_amd as m
    return m


def _t(name):
    import torch
    return getattr(torch, name)


def _update(seed, shape, dtype, scale=1e-3, strong=2):
    import torch
    g = torch.Generator().manual_seed(seed)
    r, c = shape
    k = min(strong, r, c)
    x = torch.randn(r, c, generator=g) + torch.randn(r, k, generator=g) @ torch.randn(k, c, generator=g)
    return (x * scale).to(_t(dtype)).to(dev())


def _host(t):
    return t.detach().double().cpu().numpy()


def _planes(m, shape, dtype, compute=None):
    if compute is None:
        compute = m.F16 if dtype == "bfloat16" else m.F32
    return "two" if compute == m.F32 or min(shape) < 64 else "one"


def _moved(u, planes, want, draws=None, **kw):
    """Largest norm-wise move of the oracle's result by noise of the kernel's size."""
    draws = (8 if u.size < 4096 else 2) if draws is None else draws
    return max(np.linalg.norm(ref.orthogonalize(u, noise=NOISE[planes], seed=s, **kw) - want) for s in range(draws))


def _near(got, want, tol, half, what):
    """tol: norm of the allowed difference; half: relative rounding of each element."""
    d = got - want
    assert np.all(np.isfinite(got)), what
    n = np.linalg.norm(want)
    assert np.linalg.norm(d) <= tol + half * n, (what, np.linalg.norm(d) / n, tol / n)
    each = 10 * tol / math.sqrt(want.size) + half * np.abs(want) + 2.0 ** -25
    assert np.all(np.abs(d) <= each), (what, float((np.abs(d) - each).max()))


def _ortho(m, xs, outs, **kw):
    s = m.MatrixSet(xs, outs, compute_dtype=kw.pop("compute", None))
    ws = m.orthogonalize_workspace(s)
    ws.fill_(0xFF)  # NaN
    m.orthogonalize(s, ws, **kw)
    return s, ws


SHAPES = [(1, 1), (1, 9), (9, 1), (2, 3), (3, 100), (64, 64), (63, 65), (65, 63), (128, 128), (129, 127), (100, 260),
          (260, 100), (192, 320), (333, 200), (513, 257), (64, 700), (700, 64)]


@pytest.mark.parametrize("out", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_every_shape_and_type(m, shape, out):
    import torch
    for i, x in enumerate(("float32", "bfloat16", "float16")):
        u = _update(shape[0] * 3 + i, shape, x)
        o = torch.full(shape, -7.0, dtype=_t(out), device=dev())
        _ortho(m, [u], [o])
        sync()
        want = ref.orthogonalize(_host(u))
        planes = _planes(m, shape, out)
        _near(_host(o), want, 2 * _moved(_host(u), planes, want), HALF[out], (shape, x, out))


@pytest.mark.parametrize("steps", [1, 2, 7])
@pytest.mark.parametrize("shape", [(48, 130), (200, 130)])
def test_steps_and_compute_types(m, shape, steps):
    import torch
    for compute in (m.F16, m.F32):
        u = _update(steps, shape, "float32", scale=3.0)
        o = torch.empty(shape, device=dev())
        _ortho(m, [u], [o], steps=steps, compute=compute)
        sync()
        want = ref.orthogonalize(_host(u), steps)
        planes = _planes(m, shape, "float32", compute)
        _near(_host(o), want, 2 * _moved(_host(u), planes, want, steps=steps), HALF["float32"], (shape, steps, compute))


def test_singular_vectors_stay(m):
    """A matrix of known singular values and vectors: rows of a scaled permutation, for which every product has
    one term, so that the result is the polynomial of one number within a few roundings of each operand."""
    import torch
    g = torch.Generator().manual_seed(3)
    for n in (64, 200):
        p = torch.zeros(n, n)
        p[torch.arange(n), torch.randperm(n, generator=g)] = torch.where(torch.rand(n, generator=g) < 0.5, -5.0, 5.0)
        o = torch.empty(n, n, device=dev())
        _ortho(m, [p.to(dev())], [o])
        sync()
        want = ref.scalar(1 / math.sqrt(n))
        got = o.cpu()
        assert torch.equal(got == 0, p == 0)
        moved = max(abs(ref.orthogonalize(np.array([[1.0 / math.sqrt(n)]]) , 5, 1 - 1 / math.sqrt(n), NOISE["two"], s)[0, 0]
                        - want) for s in range(16))
        assert float(((got.double() * torch.sign(p).double())[p != 0] - want).abs().max()) <= 2 * moved + 2.0 ** -24 * 1.3


def test_a_list_of_many(m):
    """Matrices of all kinds in one list give what each gives alone, bit for bit."""
    import torch
    shapes = [(1, 1), (300, 70), (64, 64), (5, 1000), (128, 128), (257, 400), (31, 33), (640, 96)]
    types = ["float32", "bfloat16", "float16"]
    xs = [_update(i, s, types[i % 3]) for i, s in enumerate(shapes)]
    outs = [torch.empty(s, dtype=_t(types[(i + 1) % 3]), device=dev()) for i, s in enumerate(shapes)]
    _ortho(m, xs, outs)
    for x, o in zip(xs, outs):
        alone = torch.empty_like(o)
        _ortho(m, [x], [alone])
        sync()
        assert torch.equal(o, alone), tuple(x.shape)


@pytest.mark.parametrize("shape", [(40, 72), (150, 130), (130, 150)])
def test_strided_rows_and_what_lies_beside_them(m, shape):
    import torch
    r, c = shape
    for dtype in ("float32", "bfloat16", "float16"):
        u = _update(7, shape, dtype)
        wide = torch.full((r, c + 9), math.nan, dtype=_t(dtype), device=dev())
        wide[:, 3:3 + c] = u
        out = torch.full((r + 2, c + 7), 3.0, dtype=_t(dtype), device=dev())
        _ortho(m, [wide[:, 3:3 + c]], [out[1:-1, 2:2 + c]])
        plain = torch.empty_like(u)
        _ortho(m, [u], [plain])
        sync()
        assert torch.equal(out[1:-1, 2:2 + c], plain)
        out[1:-1, 2:2 + c] = 3.0
        assert bool((out == 3).all())


def test_zeros_and_non_finite_matrices(m):
    import torch
    for shape in ((20, 30), (200, 180)):
        good = _update(1, shape, "float32")
        zero = torch.zeros(shape, device=dev())
        nan, inf = good.clone(), good.clone()
        nan[3, 4], inf[7, 8] = math.nan, -math.inf
        outs = [torch.full(shape, 5.0, device=dev()) for _ in range(4)]
        flags = torch.zeros(1, dtype=torch.int32, device=dev())
        _ortho(m, [good, zero, nan, inf], outs, flags=flags)
        alone = torch.empty(shape, device=dev())
        clean = torch.zeros(1, dtype=torch.int32, device=dev())
        _ortho(m, [good], [alone], flags=clean)
        sync()
        assert flags.item() == m.FLAG_NONFINITE_GRAD and clean.item() == 0
        assert torch.equal(outs[0], alone) and bool((outs[1] == 0).all())
        assert bool(outs[2].isnan().all()) and bool(outs[3].isnan().all())


@pytest.mark.parametrize("scale", [1e-30, 1e-4, 1e15, 3e37])
def test_any_magnitude(m, scale):
    """Up to the largest binary32 values; below eps the result is that much smaller than orthogonal."""
    import torch
    u = _update(9, (70, 90), "float32", scale=scale / 10)
    o = torch.empty(70, 90, device=dev())
    eps = 1e-7 * min(1.0, scale)
    _ortho(m, [u], [o], eps=eps)
    sync()
    want = ref.orthogonalize(_host(u), eps=eps)
    _near(_host(o), want, 2 * _moved(_host(u), "two", want, eps=eps), HALF["float32"], scale)


# ------------------------------------------------------------------ the step
def _step_case(seed, shapes, w_type, g_type):
    import torch
    g = torch.Generator().manual_seed(seed)
    w = [(torch.randn(s, generator=g) / math.sqrt(s[1])).to(_t(w_type)).to(dev()) for s in shapes]
    x = [_update(seed + i, s, g_type) for i, s in enumerate(shapes)]
    mom = [_update(seed + 50 + i, s, "float32", scale=5e-3) for i, s in enumerate(shapes)]
    return x, w, mom


@pytest.mark.parametrize("w_type,g_type", [("float32", "float32"), ("bfloat16", "bfloat16"), ("float16", "float32"),
                                           ("float32", "float16")])
@pytest.mark.parametrize("nesterov,scale,decay", [(True, 0, 0.1), (False, 1, 0.0)])
def test_a_step_matches_the_oracle(m, w_type, g_type, nesterov, scale, decay):
    import torch
    shapes = [(128, 42), (128, 128), (1, 128), (300, 96), (70, 500)]
    x, w, mom = _step_case(3, shapes, w_type, g_type)
    before = [(_host(a), _host(b), _host(c)) for a, b, c in zip(x, w, mom)]
    keep = [t.clone() for t in x]
    s = m.MatrixSet(x, w, mom)
    ws = m.orthogonalize_workspace(s)
    ws.fill_(0xFF)
    m.muon_step(s, ws, 0.02, momentum=0.9, nesterov=nesterov, weight_decay=decay, scale=scale)
    sync()
    for i, (g, w0, m0) in enumerate(before):
        assert torch.equal(x[i], keep[i])
        want_w, want_m = ref.muon(w0, m0, g, 0.02, 0.9, nesterov, decay, scale)
        # binary32: mu's own rounding, and the product with it and the sum in one
        assert np.all(np.abs(_host(mom[i]) - want_m) <= 2.0 ** -24 * (np.abs(want_m) + np.abs(0.9 * m0)) + 2.0 ** -149)
        u = g + 0.9 * want_m if nesterov else want_m
        planes = _planes(m, shapes[i], w_type)
        o = ref.orthogonalize(u)
        rate = ref.rate(0.02, shapes[i], scale)
        # three binary32 operations on the weight before its rounding
        _near(_host(w[i]), want_w, 2 * rate * _moved(u, planes, o) + 3 * 2.0 ** -24 * np.linalg.norm(w0), HALF[w_type],
              (shapes[i], w_type))


def test_a_step_that_is_not_finite_changes_nothing_of_that_matrix(m):
    import torch
    shapes = [(20, 30), (150, 140), (20, 30), (150, 140)]
    x, w, mom = _step_case(5, shapes, "float32", "float32")
    x[0][1, 1] = math.nan
    mom[3][140, 130] = math.inf
    keep = [t.clone() for t in w + mom]
    flags = torch.zeros(1, dtype=torch.int32, device=dev())
    s = m.MatrixSet(x, w, mom)
    m.muon_step(s, m.orthogonalize_workspace(s), 0.02, flags=flags)
    sync()
    assert flags.item() == m.FLAG_NONFINITE_GRAD
    for i in range(4):
        same = i in (0, 3)
        assert torch.equal(w[i], keep[i]) == same and torch.equal(mom[i], keep[4 + i]) == same, i


def test_results_repeat_in_graphs_and_on_other_streams(m):
    import torch
    shapes = [(128, 128), (300, 200), (64, 500)]

    def fresh():
        return _step_case(7, shapes, "bfloat16", "bfloat16")

    def steps(n, call):
        x, w, mom = fresh()
        s = m.MatrixSet(x, w, mom)
        ws = m.orthogonalize_workspace(s)
        sync()
        for _ in range(n):
            call(s, ws)
        sync()
        return w + mom

    eager = steps(3, lambda s, ws: m.muon_step(s, ws, 0.02))
    side = torch.cuda.Stream()
    for a, b in zip(eager, steps(3, lambda s, ws: m.muon_step(s, ws, 0.02, stream=side))):
        assert torch.equal(a, b)
    x, w, mom = fresh()
    s = m.MatrixSet(x, w, mom)
    ws = m.orthogonalize_workspace(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.muon_step(s, ws, 0.02)
    for rep in range(3):
        graph.replay()
        sync()
        torch.empty(1 << 20, device=dev()).fill_(float(rep))
        sync()
    for a, b in zip(eager, w + mom):
        assert torch.equal(a, b)


def test_a_dropped_set_keeps_its_memory_for_a_call_on_another_stream(m):
    import torch
    u = _update(1, (200, 200), "float32")
    want = torch.empty(200, 200, device=dev())
    _ortho(m, [u], [want])
    side = torch.cuda.Stream()
    sync()
    for rep in range(5):
        o = torch.empty(200, 200, device=dev())
        s = m.MatrixSet([u.clone()], [o])
        ws = m.orthogonalize_workspace(s)
        side.wait_stream(torch.cuda.current_stream())
        m.orthogonalize(s, ws, stream=side)
        del s, ws
        junk = [torch.full((200, 200), math.nan, device=dev()) for _ in range(20)]
        sync()
        assert torch.equal(o, want), rep
        del junk


def test_binding_refuses(m):
    import torch
    z = lambda *s, **k: torch.zeros(s, device=dev(), **k)  # noqa: E731
    for args, word in ((([z(2, 3)], [z(3, 2)]), "out"), (([z(2, 3).t()], [z(3, 2)]), "neighbouring"),
                       (([z(6)], [z(2, 3)]), "no matrix"), (([z(2, 3)], [z(2, 3)], [z(2, 3, dtype=torch.bfloat16)]), "float32"),
                       (([z(2, 3, dtype=torch.float64)], [z(2, 3)]), "none of")):
        with pytest.raises(ValueError, match=word):
            m.MatrixSet(*args)
    a = z(2, 3)
    with pytest.raises(m.IqlhError, match="share memory"):
        m.MatrixSet([a], [a])
    s = m.MatrixSet([a], [z(2, 3)])
    ws = m.orthogonalize_workspace(s)
    with pytest.raises(m.IqlhError, match="no momentum"):
        m.muon_step(s, ws, 0.1)
    large = m.MatrixSet([z(300, 300)], [z(300, 300)])
    with pytest.raises(m.IqlhError, match="too small"):
        m.orthogonalize(large, m.orthogonalize_workspace(large)[:-1])
    with pytest.raises(m.IqlhError, match="steps"):
        m.orthogonalize(s, ws, steps=0)
    with pytest.raises(ValueError, match="workspace"):
        m.orthogonalize(s, ws.cpu())
