"""Tensor lists without a GPU: the piece table that iqlh_tensor_set_fill
writes, the refusals of the norm and clip entry points (each before any HIP
call), and the oracle of the norm and clip."""
import ctypes
import math

import numpy as np
import pytest

from oracle import tensors as ref

BASE = 1 << 20
ES = {0: 4, 1: 2, 2: 2}


@pytest.fixture(scope="module")
def m():
    import offline_rl_step_amd as m
    return m


def _fill(m, ptrs, lens, types, short=0, skew=0):
    k = len(lens)
    lens_a, types_a = (ctypes.c_int64 * k)(*lens), (ctypes.c_int32 * k)(*types)
    need = ctypes.c_size_t()
    assert m._lib_set_bytes(lens_a, types_a, k, ctypes.byref(need)) == m.OK
    buf = np.zeros(need.value + 32, np.uint8)
    lead = -buf.ctypes.data % 16 + skew
    st = m.TensorSetStruct()
    rc = m._lib_set_fill((ctypes.c_void_p * k)(*ptrs), lens_a, types_a, k, buf.ctypes.data + lead,
                         need.value - short, ctypes.byref(st))
    return rc, buf[lead:lead + need.value], st


@pytest.mark.parametrize("seed", range(20))
def test_pieces_cover_every_element_once(m, seed):
    g = np.random.default_rng(seed)
    k = int(g.integers(1, 40))
    lens = [int(x) for x in np.exp(g.uniform(0, math.log(1 << g.integers(4, 22)), k)).astype(int) * (g.random(k) < 0.9)]
    types = [int(x) for x in g.integers(0, 3, k)]
    ptrs, at = [], BASE
    for n, t in zip(lens, types):
        at += ES[t] * int(g.integers(0, 9))
        at += -at % ES[t]
        ptrs.append(at if n else None)
        at += n * ES[t]
    rc, img, st = _fill(m, ptrs, lens, types)
    assert rc == m.OK
    assert st.numel == sum(lens) and st.count == k and st.overlap == 0
    dt = np.dtype([("ptr", "<u8"), ("off", "<i8"), ("n", "<i4"), ("dtype", "<i4"), ("r", "<i4", 2)])
    pieces = img[:st.pieces * 32].view(dt)
    first = img[st.pieces * 32:st.pieces * 32 + 4 * (k + 1)].view("<i4")
    assert st.pieces * 32 + 4 * (k + 1) <= st.table_bytes <= img.size
    assert first[0] == 0 and first[k] == st.pieces
    total = sum(n * ES[t] for n, t in zip(lens, types))
    pb = min(max(-(-(total // 1024) // 4096) * 4096, 4096), 32768)
    off = 0
    for i in range(k):
        e = 0
        for j in range(first[i], first[i + 1]):
            p = pieces[j]
            assert p["ptr"] == ptrs[i] + e * ES[types[i]] and p["off"] == off + e and p["dtype"] == types[i]
            assert e == 0 or p["ptr"] % 16 == 0
            assert 1 <= p["n"] and p["n"] * ES[types[i]] <= pb + 16
            e += int(p["n"])
        assert e == lens[i]
        off += lens[i]


def test_tensors_that_share_memory_are_noticed(m):
    for ptrs, lens, want in (([BASE, BASE + 400], [100, 100], 0), ([BASE, BASE + 396], [100, 100], 1),
                             ([BASE + 396, BASE], [100, 100], 1), ([BASE, BASE], [5, 5], 1),
                             ([BASE, BASE + 40, BASE + 800], [1000, 2, 2], 1), ([BASE, BASE], [0, 5], 0),
                             ([BASE + 8, BASE, BASE + 16], [2, 2, 4], 0)):
        rc, _, st = _fill(m, ptrs, lens, [0] * len(lens))
        assert rc == m.OK and st.overlap == want, (ptrs, lens)


def test_fill_refuses_bad_lists(m):
    ok = ctypes.c_size_t()
    one, f32 = (ctypes.c_int64 * 1)(4), (ctypes.c_int32 * 1)(0)
    assert m._lib_set_bytes(one, f32, 0, ctypes.byref(ok)) == m.EINVAL
    assert m._lib_set_bytes(one, f32, (1 << 20) + 1, ctypes.byref(ok)) == m.EINVAL
    assert m._lib_set_bytes(None, f32, 1, ctypes.byref(ok)) == m.EINVAL
    assert m._lib_set_bytes(one, None, 1, ctypes.byref(ok)) == m.EINVAL
    assert m._lib_set_bytes(one, f32, 1, None) == m.EINVAL
    assert m._lib_set_bytes((ctypes.c_int64 * 1)(-1), f32, 1, ctypes.byref(ok)) == m.EINVAL
    assert m._lib_set_bytes((ctypes.c_int64 * 1)(1 << 41), f32, 1, ctypes.byref(ok)) == m.EINVAL
    assert m._lib_set_bytes((ctypes.c_int64 * 5)(*[1 << 40] * 5), (ctypes.c_int32 * 5)(), 5,
                            ctypes.byref(ok)) == m.EINVAL  # 20 TB
    assert m._lib_set_bytes(one, (ctypes.c_int32 * 1)(3), 1, ctypes.byref(ok)) == m.EINVAL
    assert "float type" in m.last_error()
    assert _fill(m, [None], [4], [0])[0] == m.EINVAL
    assert _fill(m, [BASE + 2], [4], [0])[0] == m.EINVAL and "aligned" in m.last_error()
    assert _fill(m, [BASE + 1], [4], [1])[0] == m.EINVAL
    assert _fill(m, [BASE], [4], [0], short=1)[0] == m.EINVAL
    assert _fill(m, [BASE], [4], [0], skew=4)[0] == m.EINVAL
    assert _fill(m, [None, BASE], [0, 4], [0, 2])[0] == m.OK


def test_calls_refuse_bad_arguments(m):
    rc, _, st = _fill(m, [BASE], [1000], [0])
    ws = ctypes.c_size_t()
    assert m._lib_norm_ws(ctypes.byref(st), ctypes.byref(ws)) == m.OK and ws.value >= 8 * 1024
    assert m._lib_norm_ws(None, ctypes.byref(ws)) == m.EINVAL
    P = ctypes.c_void_p

    def norm(st_=st, kind=0, out=P(BASE), w=P(BASE), wb=ws.value):
        return m._lib_grad_norm(ctypes.byref(st_) if st_ else None, kind, out, None, None, w, wb, None)

    def clip(st_=st, kind=0, mx=1.0, flat=None, out=P(BASE), w=P(BASE), wb=ws.value):
        return m._lib_grad_clip(ctypes.byref(st_) if st_ else None, kind, mx, flat, out, None, w, wb, None)

    for call in (norm, clip):
        assert call() == m.EINVAL and "d_table" in m.last_error()  # not uploaded
    st.d_table = BASE
    for call in (norm, clip):
        assert call(st_=None) == m.EINVAL
        assert call(kind=2) == m.EINVAL and "kind" in m.last_error()
        assert call(out=None) == m.EINVAL
        assert call(w=None) == m.EINVAL
        assert call(w=P(BASE + 4)) == m.EINVAL
        assert call(wb=ws.value - 1) == m.EINVAL and "workspace" in m.last_error()
    for bad in (0.0, -1.0, float("nan")):
        assert clip(mx=bad) == m.EINVAL and "max_norm" in m.last_error()
    st.d_table = BASE + 8
    assert norm() == m.EINVAL
    _, _, two = _fill(m, [BASE, BASE + 4], [8, 8], [0, 0])
    two.d_table = BASE
    assert clip(st_=two, wb=1 << 20) == m.EINVAL and "share memory" in m.last_error()


def test_binding_refuses_what_the_kernels_cannot_take(m):
    import torch
    with pytest.raises(ValueError, match="at least one"):
        m.TensorSet([])
    with pytest.raises(ValueError, match="device memory"):
        m.TensorSet([torch.zeros(4)])


def test_struct_matches_the_c_compiler(m, tmp_path):
    import os
    import shutil
    import subprocess
    if shutil.which("gcc") is None:
        pytest.skip("gcc not available")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    cls = m.TensorSetStruct
    body = "".join(f'printf("%zu\\n", offsetof(iqlh_tensor_set, {f[0]}));' for f in cls._fields_)
    src = tmp_path / "l.c"
    src.write_text('#include <stdio.h>\n#include "iqlher.h"\nint main(void) {printf("%zu\\n", sizeof(iqlh_tensor_set));'
                   + body + "return 0;}")
    subprocess.run(["gcc", "-std=c11", "-Werror", "-I", os.path.join(root, "include"), str(src), "-o",
                    str(tmp_path / "l")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "l")], check=True, capture_output=True,
                                          text=True).stdout.split()]
    assert got == [ctypes.sizeof(cls)] + [getattr(cls, f[0]).offset for f in cls._fields_]


def test_oracle_on_known_values():
    assert ref.norm([[3.0], [], [4.0]]) == 5.0
    assert ref.norm([[3.0], [-4.0]], ref.MAX) == 4.0
    assert ref.norm([[]]) == 0.0 and ref.norm([], ref.MAX) == 0.0
    assert math.isnan(ref.norm([[np.inf], [np.nan]])) and math.isnan(ref.norm([[np.inf, np.nan]], ref.MAX))
    assert ref.norm([[np.inf], [1.0]]) == np.inf
    n, c, t = ref.clip([[3.0], [4.0]], 2.5)
    assert (n, c) == (5.0, 0.5) and t[0][0] == 1.5 and t[1][0] == 2.0
    assert ref.clip([[3.0], [4.0]], 5.0)[1] == 1.0
    assert ref.clip([[np.inf]], 1.0)[1] == 1.0
