"""Matrix sets without a GPU: the table that iqlh_matrix_set_fill writes and the
refusals of the entry points, each before any HIP call."""
import ctypes

import numpy as np
import pytest

BASE = 1 << 30


@pytest.fixture(scope="module")
def m():
    import offline_rl_step_amd as m
    return m


def _matrix(m, rows, cols, i=0, momentum=True, **kw):
    at = BASE * (1 + 4 * i)
    q = dict(x=at, out=at + BASE, momentum=at + 2 * BASE if momentum else None, rows=rows, cols=cols, ld_x=cols,
             ld_out=cols, ld_momentum=cols, x_dtype=m.BF16, out_dtype=m.F32, compute_dtype=m.F32)
    q.update(kw)
    return m.MatrixStruct(**q)


def _fill(m, ms, short=0, skew=0):
    arr = (m.MatrixStruct * len(ms))(*ms)
    need = ctypes.c_size_t()
    rc = m._lib_matrix_bytes(arr, len(ms), ctypes.byref(need))
    if rc != m.OK:
        return rc, None, None
    buf = np.zeros(need.value + 32, np.uint8)
    lead = -buf.ctypes.data % 16 + skew
    st = m.MatrixSetStruct()
    rc = m._lib_matrix_fill(arr, len(ms), buf.ctypes.data + lead, need.value - short, ctypes.byref(st))
    return rc, buf[lead:lead + need.value], st


MAT = np.dtype([("addr", "<u8", 3), ("ld", "<i8", 3), ("at", "<i8", 4), ("rows", "<i4"), ("cols", "<i4"),
                ("rows_pad", "<i4"), ("cols_pad", "<i4"), ("k_pad", "<i4"), ("x_dtype", "<i4"), ("out_dtype", "<i4"),
                ("planes", "<i4"), ("unit0", "<i4"), ("units", "<i4"), ("unit_rows", "<i4"), ("reserved", "<i4")])
TILE = np.dtype([("mat", "<i4"), ("m", "<u2"), ("n", "<u2")])


@pytest.mark.parametrize("seed", range(12))
def test_tiles_and_pieces_cover_every_matrix_once(m, seed):
    g = np.random.default_rng(seed)
    ms = [_matrix(m, int(r), int(c), i) for i, (r, c) in enumerate(np.exp(g.uniform(0, np.log(5000), (int(g.integers(1, 9)), 2))))]
    rc, img, st = _fill(m, ms)
    assert rc == m.OK and st.count == len(ms) and st.momentum == 1
    mats = img[:st.count * MAT.itemsize].view(MAT)
    n = st.units + st.sym_tiles + st.rect_tiles + st.small
    tiles = img[st.count * MAT.itemsize:][:n * 8].view(TILE)
    units, sym, rect, small = np.split(tiles, np.cumsum([st.units, st.sym_tiles, st.rect_tiles]))
    assert sorted(int(t["mat"]) for t in small) == [i for i, q in enumerate(mats) if q["units"] == 0]
    assert st.count * MAT.itemsize + 8 * n <= st.table_bytes <= img.size
    ranges = [(0, 8 * st.units + 4 * st.count)]
    unit0 = 0
    for i, q in enumerate(mats):
        assert (q["rows"], q["cols"]) == (ms[i].rows, ms[i].cols)
        assert q["rows_pad"] == -(-q["rows"] // 64) * 64 and q["cols_pad"] == -(-q["cols"] // 64) * 64
        assert q["k_pad"] == min(q["rows_pad"], q["cols_pad"]) and q["unit0"] == unit0 and q["units"] <= 512
        if q["units"] == 0:
            assert int(q["rows_pad"]) * int(q["cols_pad"]) <= 49152 and st.small_bytes <= 158 * 1024
            continue
        assert q["units"] * q["unit_rows"] >= q["rows_pad"] > (q["units"] - 1) * q["unit_rows"]
        assert sorted(u["m"] for u in units if u["mat"] == i) == list(range(q["units"]))
        unit0 += q["units"]
        x, s = q["rows_pad"] * q["cols_pad"] * 2 * q["planes"], int(q["k_pad"]) ** 2 * 2 * q["planes"]
        ranges += [(a, a + int(b)) for a, b in zip(q["at"], (x, x, s, s))]
    for i, q in enumerate(mats):
        if q["units"] == 0:
            assert not any(t["mat"] == i for part in (units, sym, rect) for t in part)
            continue
        mine = [(int(t["m"]), int(t["n"])) for t in rect if t["mat"] == i]
        mt, nt = -(-q["rows_pad"] // st.rect_tile), -(-q["cols_pad"] // st.rect_tile)
        assert sorted(mine) == [(a, b) for a in range(mt) for b in range(nt)]
        k = -(-q["k_pad"] // st.sym_tile)
        assert sorted((int(t["m"]), int(t["n"])) for t in sym if t["mat"] == i) == [(a, b) for a in range(k) for b in range(a + 1)]
    ranges.sort()
    assert all(a[1] <= b[0] for a, b in zip(ranges, ranges[1:])) and ranges[-1][1] <= st.workspace_bytes


def test_precision_goes_by_the_type_asked_for_and_small_sides_have_two_planes(m):
    for shape, compute, want in (((64, 64), m.F16, 1), ((64, 64), m.F32, 2), ((63, 500), m.F16, 2), ((500, 63), m.F16, 2),
                                 ((500, 64), m.F16, 1)):
        rc, img, st = _fill(m, [_matrix(m, *shape, compute_dtype=compute)])
        assert rc == m.OK and img[:MAT.itemsize].view(MAT)[0]["planes"] == want, (shape, compute)


def test_bad_lists_are_refused(m):
    one = lambda **kw: [_matrix(m, 8, 8, **kw)]  # noqa: E731
    need = ctypes.c_size_t()
    ok = (m.MatrixStruct * 1)(*one())
    assert m._lib_matrix_bytes(ok, 0, ctypes.byref(need)) == m.EINVAL
    assert m._lib_matrix_bytes(ok, 4097, ctypes.byref(need)) == m.EINVAL
    assert m._lib_matrix_bytes(None, 1, ctypes.byref(need)) == m.EINVAL
    assert m._lib_matrix_bytes(ok, 1, None) == m.EINVAL
    for r, c in ((0, 8), (8, 0), (65537, 8), (8, 65537)):
        assert _fill(m, [_matrix(m, r, c)])[0] == m.ESHAPE
    for kw, word in ((dict(x=None), "NULL"), (dict(out=None), "NULL"), (dict(x=BASE + 1), "aligned"),
                     (dict(out=2 * BASE + 2), "aligned"), (dict(ld_x=7), "row stride"), (dict(ld_out=7), "row stride"),
                     (dict(ld_momentum=7), "row stride"), (dict(x_dtype=3), "float type"), (dict(out_dtype=-1), "float type"),
                     (dict(compute_dtype=m.BF16), "compute_dtype")):
        assert _fill(m, one(**kw))[0] == m.EINVAL and word in m.last_error(), (kw, m.last_error())
    assert _fill(m, one(), short=1)[0] == m.EINVAL
    assert _fill(m, one(), skew=8)[0] == m.EINVAL
    assert _fill(m, [_matrix(m, 8, 8), _matrix(m, 8, 8, 1, momentum=False)])[0] == m.EINVAL and "momentum" in m.last_error()


def test_shared_memory_is_refused_unless_rows_interleave(m):
    a = lambda **kw: _matrix(m, 4, 8, **kw)  # noqa: E731
    assert _fill(m, [a(out=BASE)])[0] == m.EINVAL and "share memory" in m.last_error()
    b = a()
    b.momentum = 2 * BASE + 64
    assert _fill(m, [b])[0] == m.EINVAL and "momentum" in m.last_error()
    b = _matrix(m, 4, 8, 1)
    b.out = 2 * BASE + 32
    assert _fill(m, [a(), b])[0] == m.EINVAL and "of matrix" in m.last_error()
    b.x = BASE  # both read the same update
    b.out = BASE * 6
    assert _fill(m, [a(), b])[0] == m.OK
    # column blocks of one buffer
    left, right = a(ld_out=16), _matrix(m, 4, 8, 1, ld_out=16)
    right.out = left.out + 32
    assert _fill(m, [left, right])[0] == m.OK
    right.out = left.out + 28
    assert _fill(m, [left, right])[0] == m.EINVAL


def test_calls_refuse_bad_arguments(m):
    rc, _, st = _fill(m, [_matrix(m, 100, 30)])
    assert rc == m.OK
    _, _, bare = _fill(m, [_matrix(m, 100, 30, momentum=False)])

    def ortho(s=st, steps=5, eps=1e-7, w=BASE, wb=None):
        return m._lib_orthogonalize(ctypes.byref(s) if s else None, steps, eps, None, w, s.workspace_bytes if wb is None and s else wb or 0, None)

    def step(s=st, steps=5, eps=1e-7, w=BASE, wb=None, lr=0.1, mu=0.9, nest=1, wd=0.0, scale=0):
        return m._lib_muon_step(ctypes.byref(s) if s else None, lr, mu, nest, wd, scale, steps, eps, None, w,
                                s.workspace_bytes if wb is None and s else wb or 0, None)

    for call in (ortho, step):
        assert call() == m.EINVAL and "d_table" in m.last_error()
    st.d_table = bare.d_table = BASE
    for call in (ortho, step):
        assert call(s=None) == m.EINVAL
        for bad in (0, -1, 33):
            assert call(steps=bad) == m.EINVAL and "steps" in m.last_error()
        for bad in (0.0, -1.0, float("nan"), float("inf")):
            assert call(eps=bad) == m.EINVAL and "eps" in m.last_error()
        assert call(w=None) == m.EINVAL and call(w=BASE + 8) == m.EINVAL
        assert call(wb=st.workspace_bytes - 1) == m.EINVAL and "too small" in m.last_error()
    for bad in (float("nan"), float("inf")):
        assert step(lr=bad) == m.EINVAL and step(wd=bad) == m.EINVAL
    for bad in (-0.1, 1.0, float("nan")):
        assert step(mu=bad) == m.EINVAL and "mu" in m.last_error()
    assert step(nest=2) == m.EINVAL and step(scale=2) == m.EINVAL
    assert step(s=bare) == m.EINVAL and "no momentum" in m.last_error()


def test_binding_refuses_lists_the_kernels_cannot_take(m):
    import torch
    z = torch.zeros
    with pytest.raises(ValueError, match="at least one"):
        m.MatrixSet([], [])
    with pytest.raises(ValueError, match="same length"):
        m.MatrixSet([z(2, 2)], [])
    with pytest.raises(ValueError, match="device memory"):
        m.MatrixSet([z(2, 2)], [z(2, 2)])
    with pytest.raises(ValueError, match="compute_dtype"):
        m.MatrixSet([z(2, 2)], [z(2, 2)], compute_dtype=m.BF16)
