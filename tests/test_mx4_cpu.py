"""Microscaled 4-bit matrices without a GPU: refusals of the entry points, each
before any HIP call, and the oracle against the format's definition."""
import ctypes

import numpy as np
import pytest

from oracle import mx4 as ref

P = ctypes.c_void_p
A = 1 << 20


@pytest.fixture(scope="module")
def m():
    import offline_rl_step_amd as m
    return m


def _q(m, rows=64, cols=64, codes=A, scales=A):
    return ctypes.byref(m.Mx4Struct(codes, scales, rows, cols))


def test_quantize_refusals(m):
    def call(x=P(A), dt=0, ld=64, tr=0, q=None):
        return m._lib_mx4_quantize(x, dt, ld, tr, _q(m) if q is None else q, None)
    assert m._lib_mx4_quantize(P(A), 0, 64, 0, None, None) == m.EINVAL
    assert call(x=None) == m.EINVAL
    assert call(dt=3) == m.EINVAL and call(dt=-1) == m.EINVAL
    assert call(x=P(A + 2)) == m.EINVAL and "aligned" in m.last_error()
    assert call(x=P(A + 1), dt=1) == m.EINVAL
    assert call(ld=63) == m.EINVAL and call(tr=1, ld=63) == m.EINVAL
    assert call(tr=2) == m.EINVAL
    assert call(q=_q(m, rows=0)) == m.EINVAL and call(q=_q(m, cols=0)) == m.EINVAL
    assert call(q=_q(m, rows=(1 << 30) + 1)) == m.EINVAL
    assert call(q=_q(m, codes=None)) == m.EINVAL and call(q=_q(m, scales=None)) == m.EINVAL
    assert call(q=_q(m, codes=A + 8)) == m.EINVAL and "16-byte" in m.last_error()
    assert m._lib_mx4_dequantize(_q(m), P(A), 0, 63, None) == m.EINVAL
    assert m._lib_mx4_dequantize(_q(m), None, 0, 64, None) == m.EINVAL
    assert m._lib_mx4_dequantize(None, P(A), 0, 64, None) == m.EINVAL


def test_product_refusals(m):
    ws = ctypes.c_size_t()
    assert m._lib_mx4_ws(64, 64, 64, ctypes.byref(ws)) == m.OK and ws.value > 0
    for bad in ((0, 1, 1), (1, 0, 1), (1, 1, 0), ((1 << 30) + 1, 1, 1)):
        assert m._lib_mx4_ws(*bad, ctypes.byref(ws)) == m.EINVAL
    assert m._lib_mx4_ws(64, 64, 64, None) == m.EINVAL
    m._lib_mx4_ws(64, 64, 64, ctypes.byref(ws))

    def mm(a=None, b=None, relu=0, out=P(A), dt=0, ld=64, w=P(A), wb=ws.value):
        return m._lib_mx4_matmul(a or _q(m), b or _q(m), None, relu, out, dt, ld, w, wb, None)

    def lin(b=None, relu=0, out=P(A), dt=0, ld=64, w=P(A), wb=ws.value, M=64, x=P(A), xdt=0, xld=64):
        return m._lib_mx4_linear(x, xdt, xld, M, b or _q(m), None, relu, out, dt, ld, w, wb, None)

    for call in (mm, lin):
        assert call(relu=2) == m.EINVAL
        assert call(out=None) == m.EINVAL and call(out=P(A + 2)) == m.EINVAL
        assert call(dt=7) == m.EINVAL and call(ld=63) == m.EINVAL
        assert call(w=None) == m.EINVAL and call(w=P(A + 8)) == m.EINVAL
        assert call(wb=ws.value - 1) == m.EINVAL and "workspace" in m.last_error()
        assert call(b=_q(m, codes=A + 4)) == m.EINVAL
    assert mm(a=_q(m, cols=96)) == m.EINVAL and "columns" in m.last_error()
    assert lin(M=0) == m.EINVAL and lin(M=(1 << 30) + 1) == m.EINVAL
    assert lin(x=None) == m.EINVAL and lin(xdt=5) == m.EINVAL and lin(xld=63) == m.EINVAL
    assert lin(b=_q(m, rows=1 << 30), ld=1 << 30, M=1 << 30, wb=1 << 60) == m.ESHAPE
    assert lin(b=_q(m, rows=1 << 29), ld=1 << 29, M=1, wb=1 << 60) == m.ESHAPE  # 2^25 workgroups of 512


def test_launches_that_would_hold_too_many_threads_are_refused(m):
    big = lambda rows, cols: _q(m, rows=rows, cols=cols)  # noqa: E731
    assert m._lib_mx4_quantize(P(A), 1, 4096, 0, big(1 << 28, 4096), None) == m.ESHAPE and "launch" in m.last_error()
    assert m._lib_mx4_quantize(P(A), 1, 1 << 28, 1, big(1 << 28, 4096), None) == m.ESHAPE
    assert m._lib_mx4_dequantize(big(1 << 28, 4096), P(A), 1, 4096, None) == m.ESHAPE
    assert m._lib_mx4_dequantize(big(1 << 30, 257), P(A), 0, 257, None) == m.ESHAPE
    # a product whose tiles one launch takes, of an x whose quantisation it does not
    assert m._lib_mx4_linear(P(A), 1, 8192, 1 << 28, big(1, 8192), None, 0, P(A), 1, 1, P(A), 1 << 60,
                             None) == m.ESHAPE and "x of" in m.last_error()


def test_forward_refusals(m):
    b = ctypes.c_size_t()
    assert m._lib_forward_mx4_ws(None, 4, ctypes.byref(b)) == m.EINVAL
    assert m._lib_forward_mx4(None, P(A), 0, 4, 1, P(A), None, None, 0.9, None, P(A), 1 << 20, None) == m.EINVAL


def test_binding_checks_the_storage(m):
    import torch
    with pytest.raises(ValueError):
        m.Mx4(torch.zeros((2, 16), dtype=torch.uint8), torch.zeros((2, 2), dtype=torch.uint8), 2, 32)
    with pytest.raises(ValueError):
        m.Mx4(torch.zeros((2, 16), dtype=torch.int8), torch.zeros((2, 1), dtype=torch.uint8), 2, 32)
    q = m.Mx4(torch.zeros((2, 32), dtype=torch.uint8), torch.zeros((2, 2), dtype=torch.uint8), 2, 33)
    assert q.struct.rows == 2 and q.struct.cols == 33
    with pytest.raises(ValueError, match="device memory"):
        m.mx4_quantize(torch.zeros((2, 33)), q)


def test_struct_matches_the_c_compiler(m, tmp_path):
    import os
    import shutil
    import subprocess
    if shutil.which("gcc") is None:
        pytest.skip("gcc not available")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    cls = m.Mx4Struct
    body = "".join(f'printf("%zu\\n", offsetof(iqlh_mx4, {f[0]}));' for f in cls._fields_)
    src = tmp_path / "l.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "iqlher.h"\nint main(void) {'
                   'printf("%zu\\n", sizeof(iqlh_mx4));' + body + "return 0;}")
    subprocess.run(["gcc", "-std=c11", "-Werror", "-I", os.path.join(root, "include"), str(src), "-o",
                    str(tmp_path / "l")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "l")], check=True, capture_output=True,
                                          text=True).stdout.split()]
    assert got == [ctypes.sizeof(cls)] + [getattr(cls, f[0]).offset for f in cls._fields_]


# ------------------------------------------------------------------- oracle
def test_oracle_borders_and_scales():
    # the seven borders between neighbouring magnitudes go to the even code
    assert list(ref.nearest_codes(np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]))) == [0, 2, 2, 4, 4, 6, 6]
    assert list(ref.nearest_codes(np.array([0.26, 0.74, 1.26, 1.74, 2.51, 3.49, 5.01, 7.9]))) == [1, 1, 3, 3, 5, 5, 7, 7]
    assert list(ref.scale_bytes(np.array([0.0, 1.0, 4.0, 6.0, 7.99, 8.0, 2.0 ** -126, 2.0 ** 127]))) == \
        [0, 125, 127, 127, 127, 128, 0, 252]


def test_oracle_round_trip_is_exact_on_representable_blocks():
    g = np.random.default_rng(0)
    for e in (-20, 0, 30):
        x = g.choice(ref.LEVELS, (5, 64)) * g.choice([-1, 1], (5, 64)) * 2.0 ** e
        x[:, ::32] = 4.0 * 2.0 ** e
        assert np.array_equal(ref.round_trip(x), x)
        assert np.array_equal(ref.unpack(ref.pack(ref.quantize(x)[0])), ref.quantize(x)[0])


def test_oracle_error_of_a_block_is_bounded():
    """|x - value| <= 2 scale (above 6 scales) or 1 scale elsewhere, scale <= amax / 4."""
    g = np.random.default_rng(1)
    x = g.standard_normal((50, 96))
    amax = np.repeat(np.abs(x).reshape(50, 3, 32).max(2), 32, 1)
    assert np.all(np.abs(ref.round_trip(x) - x) <= amax / 4)


def test_oracle_non_finite_blocks():
    x = np.ones((1, 64))
    x[0, 40] = np.inf
    v = ref.round_trip(x)
    assert np.all(v[0, :32] == 1.0) and np.all(np.isnan(v[0, 32:]))


def test_oracle_change_bound_covers_perturbations():
    g = np.random.default_rng(2)
    x = g.standard_normal((40, 64))
    eps = np.full_like(x, 1e-2)
    bound = ref.round_trip_change(x, eps)
    base = ref.round_trip(x)
    for _ in range(50):
        moved = ref.round_trip(x + g.uniform(-1, 1, x.shape) * eps)
        assert np.all(np.abs(moved - base) <= bound + 1e-12)
    assert np.any(bound > 0) and np.all(ref.round_trip_change(x, np.zeros_like(x)) == 0)


def test_oracle_value_network_reduces_to_the_plain_one_on_the_grid():
    from oracle import iql
    g = np.random.default_rng(3)
    S, H = 32, 32
    w1 = np.where(np.eye(H, S) > 0, 1.0, 0.0)
    w2 = np.where(np.eye(H) > 0, 0.5, 0.0)
    p = np.concatenate([w1.ravel(), np.zeros(H), w2.ravel(), np.zeros(H), np.ones(H), [0.25]])
    x = g.choice([1.0, 2.0, 4.0, -3.0], (6, S))
    x[:, 0] = 4.0
    want = iql.forward(iql.unflatten(p, S, H, H), x)[0]
    assert np.allclose(ref.value_network(p, S, H, H, x), want, rtol=0, atol=0)
