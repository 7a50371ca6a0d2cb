"""Operands, outputs and workspaces of the 4-bit calls that share memory are
refused before any HIP call; what only interleaves is not.  The addresses are
made up: a call that is not refused fails at its launch, without a device."""
import ctypes

import pytest

P = ctypes.c_void_p
A = 1 << 24
FAR = 1 << 30


@pytest.fixture(scope="module")
def m():
    import torch
    import offline_rl_step_amd as m
    if torch.cuda.is_available():
        pytest.skip("made-up addresses: for a machine without a device")
    return m


def _q(m, rows, cols, codes, scales):
    return ctypes.byref(m.Mx4Struct(codes, scales, rows, cols))


def _refused(m, rc):
    if rc == m.EINVAL:
        assert "share memory" in m.last_error(), m.last_error()
        return True
    assert rc == m.EHIP, (rc, m.last_error())  # past the checks: no device
    return False


# a [64][ld] float matrix at `at`; codes of 64 x 96 take 64 * 48 bytes, scales 64 * 3
@pytest.mark.parametrize("at,ld,dt,codes,scales,want", [
    (A, 96, 0, FAR, 2 * FAR, False),
    (A, 96, 0, A, 2 * FAR, True),
    (A, 96, 0, A + 64 * 96 * 4, 2 * FAR, False),
    (A, 96, 0, A + 64 * 96 * 4 - 16, 2 * FAR, True),
    (A, 96, 0, A - 64 * 48, 2 * FAR, False),
    (A, 96, 0, A - 64 * 48 + 16, 2 * FAR, True),
    (A, 96, 0, FAR, A + 64 * 96 * 4 - 1, True),
    (A, 96, 0, FAR, A - 64 * 3, False),
    (A, 96, 1, A + 64 * 96 * 2, 2 * FAR, False),
    (A, 96, 1, A + 64 * 96 * 2 - 16, 2 * FAR, True),
    # rows 16 KB apart: the codes between two of them, over the next one, behind the last
    (A, 4096, 0, A + 96 * 4, 2 * FAR, False),
    (A, 4096, 0, A + 16384 - 64 * 48, 2 * FAR, False),
    (A, 4096, 0, A + 16384 - 64 * 48 + 16, 2 * FAR, True),
    (A, 4096, 0, A + 63 * 16384 + 96 * 4, 2 * FAR, False),
    (A, 96, 0, FAR, FAR + 64 * 48 - 1, True),  # codes and scales
    (A, 96, 0, FAR, FAR + 64 * 48, False),
])
def test_quantize_and_dequantize(m, at, ld, dt, codes, scales, want):
    q = _q(m, 64, 96, codes, scales)
    assert _refused(m, m._lib_mx4_quantize(P(at), dt, ld, 0, q, None)) == want
    read_only = 0 < scales - codes < 64 * 48  # codes over scales: nothing that dequantize writes
    assert _refused(m, m._lib_mx4_dequantize(q, P(at), dt, ld, None)) == (want and not read_only)
    if ld == 96:  # the transpose: x is [96][64]
        assert _refused(m, m._lib_mx4_quantize(P(at), dt, 64, 1, q, None)) == want


def _product(m, call, **over):
    """A product of 40 x 24 outputs over 96, in places of their own but for `over`."""
    M, N, K = 40, 24, 96
    p = dict(a=1, sa=2, b=3, sb=4, bias=5, out=6, ws=7, x=8)
    p = {k: v * FAR for k, v in p.items()}
    ld, xld, dt, xdt = over.pop("ld", N), over.pop("xld", K), over.pop("dt", 0), over.pop("xdt", 0)
    p.update(over)
    ws = ctypes.c_size_t()
    m._lib_mx4_ws(M, N, K, ctypes.byref(ws))
    b, wb = _q(m, N, K, p["b"], p["sb"]), ws.value + 4096  # more than the call takes
    if call == "matmul":
        return m._lib_mx4_matmul(_q(m, M, K, p["a"], p["sa"]), b, P(p["bias"]), 0, P(p["out"]), dt, ld, P(p["ws"]), wb, None)
    return m._lib_mx4_linear(P(p["x"]), xdt, xld, M, b, P(p["bias"]), 0, P(p["out"]), dt, ld, P(p["ws"]), wb, None)


def test_products(m):
    out = 6 * FAR
    end = out + 40 * 24 * 4
    ws = ctypes.c_size_t()
    m._lib_mx4_ws(40, 24, 96, ctypes.byref(ws))
    for call in ("matmul", "linear"):
        left = ["a", "sa"] if call == "matmul" else ["x"]
        assert not _refused(m, _product(m, call))
        for name in left + ["b", "sb", "bias", "ws"]:
            assert _refused(m, _product(m, call, **{name: out})), (call, name)
            assert _refused(m, _product(m, call, **{name: end - 16})), (call, name)
            assert not _refused(m, _product(m, call, **{name: end})), (call, name)
            if name != "ws":  # the workspace is written too; what lies behind what a call takes of it is not
                assert _refused(m, _product(m, call, **{name: 7 * FAR})), (call, name)
                assert not _refused(m, _product(m, call, **{name: 7 * FAR + (ws.value + 15) // 16 * 16})), (call, name)
        # operands may share memory with each other
        assert not _refused(m, _product(m, call, b=FAR, sb=2 * FAR, x=FAR))


@pytest.mark.parametrize("xdt", [0, 1])
def test_columns_of_one_buffer(m, xdt):
    """x and out as columns of one matrix, side by side; one column over the
    border; and with rows twice as far apart in x (every other row of it)."""
    es = 4 if xdt == 0 else 2
    pitch = 640 // es  # elements; x takes 96 of a row, out 24
    base = 9 * FAR
    for rows in (1, 2):
        over = dict(x=base, xld=pitch * rows, xdt=xdt, dt=xdt, ld=pitch)
        assert not _refused(m, _product(m, "linear", out=base + 96 * es, **over))
        assert _refused(m, _product(m, "linear", out=base + 95 * es, **over))
        assert not _refused(m, _product(m, "linear", out=base + 640 * 3 + 96 * es, **over))
        assert not _refused(m, _product(m, "linear", out=base - 24 * es, **over))
        assert _refused(m, _product(m, "linear", out=base - 23 * es, **over))
        assert _refused(m, _product(m, "linear", out=base + (640 * rows * 39 + 95 * es), **over))
        assert not _refused(m, _product(m, "linear", out=base + (640 * rows * 39 + 96 * es), **over))
    # out's rows are twice as far apart
    over = dict(x=base, xld=pitch, xdt=xdt, dt=xdt, ld=2 * pitch)
    assert not _refused(m, _product(m, "linear", out=base + 96 * es, **over))
    assert _refused(m, _product(m, "linear", out=base + 640 + 95 * es, **over))


def test_pitches_that_meet_in_one_row_only(m):
    """Row 30 of out is the first one to touch a row of x."""
    base = 9 * FAR
    # x rows every 4000 bytes, out rows every 3900: row i of out at base + 384 + 3000 + 3900 i
    over = dict(x=base, xld=1000, ld=975)
    hits = [i for i in range(40) if any(384 + 3000 + 3900 * i < 4000 * j + 384 and 4000 * j < 384 + 3000 + 3900 * i + 96
                                        for j in range(40))]
    assert hits and min(hits) > 20
    assert _refused(m, _product(m, "linear", out=base + 384 + 3000, **over))
    assert not _refused(m, _product(m, "linear", out=base + 384 + 3000, x=base, xld=1000, ld=1000))


def test_small_matrices_against_their_elements(m):
    """Random shapes, pitches and distances: refused exactly where x and out
    have an element's bytes in common."""
    import random
    g = random.Random(1)
    ws = ctypes.c_size_t()
    seen = [0, 0]
    for _ in range(3000):
        M, N, K = g.randint(1, 7), g.randint(1, 9), g.randint(1, 9)
        xld, ld = K + g.randint(0, 12), N + g.randint(0, 12)
        if g.random() < 0.4:
            xld = ld = max(xld, ld)
        d = g.randint(-150, 150)
        assert m._lib_mx4_ws(M, N, K, ctypes.byref(ws)) == m.OK
        rc = m._lib_mx4_linear(P(A), 0, xld, M, _q(m, N, K, FAR, 2 * FAR), None, 0, P(A + 4 * d), 0, ld, P(3 * FAR),
                               ws.value, None)
        common = bool({i * xld + j for i in range(M) for j in range(K)}
                      & {d + i * ld + j for i in range(M) for j in range(N)})
        assert _refused(m, rc) == common, (M, N, K, xld, ld, d)
        seen[common] += 1
    assert min(seen) > 300
