"""The clip in place rounds each product once: elements whose product with the
factor lies so close to the middle of two 16-bit values that binary32 rounds it
onto the middle, from where a second rounding goes to the even one.

With the largest-magnitude norm, an element of 1 as the largest and a bound
b < 1, the factor is b itself (b / 1 is exact), so it can be chosen: for a
significand X of p bits and a middle m of two results, C = round(m / X) gives a
product at most X / 2 away from m, within half a step of binary32 (24 bits) of
it.  The reference rounds the exact product (p + 24 bits, exact in binary64) once."""
import numpy as np
import pytest

from tests.gpu_util import dev, sync

pytestmark = pytest.mark.gpu

# significand bits, smallest exponent (of the last place of a subnormal)
TYPES = {"float16": (11, -24), "bfloat16": (8, -133)}


@pytest.fixture(scope="module")
def m():
    import offline_rl_step_amd as m
    return m


def _round(x, bits, smallest):
    """float64 values to the nearest of `bits` significand bits, ties to even,
    steps no smaller than 2^smallest."""
    _, e = np.frexp(x)
    step = np.exp2(np.maximum(e - bits, smallest).astype(np.float64))
    return np.rint(x / step) * step


def _factors(bits, n):
    """binary32 factors in [0.5, 1), each with an element of which the product
    is next to a middle but not on it, and rounds another way in two steps."""
    g = np.random.default_rng(bits)
    out = []
    while len(out) < n:
        X = int(g.integers(1 << (bits - 1), 1 << bits)) | 1
        mid = (2 * int(g.integers(1 << (bits - 1), 1 << bits)) + 1) << 23  # bits + 1 significant bits of bits + 24
        C = round(mid / X)
        if not (1 << 23) <= C < (1 << 24) or X * C == mid:
            continue
        p = np.float64(X) * np.float64(C)
        if _round(p, bits, -200) != _round(np.float64(np.float32(p)), bits, -200):
            out.append((X / 2.0 ** bits, C / 2.0 ** 24))
    return out


@pytest.mark.parametrize("name", sorted(TYPES))
@pytest.mark.parametrize("scale", [1.0, 2.0 ** -10, "smallest"])
def test_products_next_to_a_middle_round_once(m, name, scale):
    """Whole significand ranges and the crafted ones, at 16-byte boundaries and
    off them; `smallest`: products among the type's subnormal values."""
    import torch
    bits, smallest = TYPES[name]
    pairs = _factors(bits, 24)
    scale = 2.0 ** (smallest + 3) if scale == "smallest" else scale
    every = np.arange(1 << (bits - 1), 1 << bits) / 2.0 ** bits
    x = np.concatenate([[1.0], every, [p for p, _ in pairs], -every])
    x[1:] = _round(x[1:] * scale, bits, smallest)
    different = 0
    for lead in (0, 1):
        for _, c in pairs:
            t = torch.zeros(len(x) + lead, dtype=torch.float64)
            t[lead:] = torch.from_numpy(x)
            t = t.to(getattr(torch, name)).to(dev())[lead:]
            assert np.array_equal(t.double().cpu().numpy(), x)
            s = m.TensorSet([t])
            out = torch.zeros(2, device=dev())
            m.grad_clip(s, c, out, m.grad_norm_workspace(s), kind=m.NORM_MAX)
            sync()
            assert out.tolist() == [1.0, c]
            want = _round(x * c, bits, smallest)
            different += int(np.sum(want != _round((x * c).astype(np.float32).astype(np.float64), bits, smallest)))
            got = t.double().cpu().numpy()
            assert np.array_equal(got, want), (c, x[got != want], got[got != want], want[got != want])
    if scale >= 2.0 ** -10:
        assert different >= 24  # the crafted elements are there


@pytest.mark.parametrize("name", sorted(TYPES))
def test_whole_pieces_round_once(m, name):
    """The same over a tensor of many whole pieces (32 MB and more)."""
    import torch
    bits, smallest = TYPES[name]
    pairs = _factors(bits, 3)
    x = np.concatenate([np.arange(1 << (bits - 1), 1 << bits) / 2.0 ** bits, [p for p, _ in pairs], [1.0]])
    reps = (20 << 20) // len(x) + 1
    for _, c in pairs:
        t = torch.from_numpy(x).to(getattr(torch, name)).to(dev()).repeat(reps)
        s = m.TensorSet([t])
        out = torch.zeros(2, device=dev())
        m.grad_clip(s, c, out, m.grad_norm_workspace(s), kind=m.NORM_MAX)
        sync()
        assert out.tolist() == [1.0, c]
        want = torch.from_numpy(_round(x * c, bits, smallest)).to(getattr(torch, name)).to(dev())
        assert bool((t.view(reps, -1) == want).all())


@pytest.mark.parametrize("flat", [False, True])
def test_the_factor_of_any_bound_is_rounded_once(m, flat):
    """c = bound / norm for bounds that binary32 does not hold: at most half a
    step of binary32 from the quotient (the norm's own error, n 2^-53 of it, far
    below); rounding the bound first would take up to two halves."""
    import torch
    x = torch.tensor([3.0, 4.0], device=dev())  # norm 5, exact
    s = m.TensorSet([x])
    ws, out, dst = m.grad_norm_workspace(s), torch.zeros(2, device=dev()), torch.zeros(2, device=dev())
    g = np.random.default_rng(3)
    apart = 0
    for bound in g.uniform(0.5, 5.0, 400):
        x.copy_(torch.tensor([3.0, 4.0]))
        m.grad_clip(s, float(bound), out, ws, out_flat=dst if flat else None)
        sync()
        c, want = float(out[1]), bound / 5.0
        assert c == float(np.float32(want)), bound
        apart += c != float(np.float32(np.float64(np.float32(bound)) / 5.0))
        y = (dst if flat else x).cpu().numpy()
        assert np.array_equal(y, np.float32(c) * np.array([3.0, 4.0], np.float32))
    assert apart > 20  # bounds whose rounding shows in the factor are among them
