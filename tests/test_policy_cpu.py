"""Policy loss without a GPU: sizes of the workspace and the refusals of the
entry points, each before any HIP call."""
import ctypes
import os
import shutil
import subprocess

import pytest

BASE = 1 << 30
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def m():
    import offline_rl_step_amd as m
    return m


def _bytes(m, rows, actions, dim, dtype, grad):
    out = ctypes.c_size_t()
    rc = m._lib_policy_ws(rows, actions, dim, dtype, grad, ctypes.byref(out))
    return rc, out.value


def _head(m, **kw):
    q = dict(hidden=BASE, weight=2 * BASE, bias=None, rows=16, actions=100, dim=8, ld_hidden=8, ld_weight=8,
             dtype=m.BF16)
    q.update(kw)
    return m.PolicyHeadStruct(**q)


def _loss(m, head=None, taken=3 * BASE, w=None, scale=1.0, nll=4 * BASE, lse=5 * BASE, loss=6 * BASE, flags=None,
          ws=7 * BASE, wb=1 << 20):
    return m._lib_policy_loss(ctypes.byref(head or _head(m)), P(taken), w, scale, P(nll), P(lse), P(loss), flags, P(ws),
                              wb, None)


def _grad(m, head=None, taken=3 * BASE, w=None, scale=1.0, lse=5 * BASE, dh=8 * BASE, ldh=8, dw=9 * BASE, ldw=8,
          db=10 * BASE, ws=7 * BASE, wb=1 << 24):
    return m._lib_policy_grad(ctypes.byref(head or _head(m)), P(taken), w, scale, P(lse), P(dh), ldh, P(dw), ldw, P(db),
                              P(ws), wb, None)


def test_workspace_sizes(m):
    for dtype in (m.F32, m.BF16, m.F16):
        for shape in ((1, 1, 1), (16, 100, 8), (777, 10007, 501), (8192, 65536, 2048)):
            rc, plain = _bytes(m, *shape, dtype, 0)
            assert rc == m.OK and plain > 0
            rc, grad = _bytes(m, *shape, dtype, 1)
            assert rc == m.OK and grad > 0
    # the logits themselves would be 2 GiB
    assert _bytes(m, 8192, 65536, 2048, m.BF16, 1)[1] < 1 << 30


def test_sizes_that_are_refused(m):
    for bad in ((0, 4, 4), (4, 0, 4), (4, 4, 0), (-1, 4, 4), ((1 << 24) + 1, 4, 4), (4, (1 << 24) + 1, 4),
                (4, 4, (1 << 14) + 1), (1 << 24, 1 << 15, 4)):
        assert _bytes(m, *bad, m.F32, 0)[0] == m.ESHAPE, bad
    assert _bytes(m, 4, 4, 4, 3, 0)[0] == m.EINVAL and "float type" in m.last_error()
    assert _bytes(m, 4, 4, 4, m.F32, 2)[0] == m.EINVAL
    assert m._lib_policy_ws(4, 4, 4, m.F32, 0, None) == m.EINVAL


def test_arguments_that_are_refused(m):
    for call in (_loss, _grad):
        for kw, word in ((dict(hidden=None), "NULL"), (dict(weight=None), "NULL"), (dict(hidden=BASE + 1), "aligned"),
                         (dict(ld_hidden=7), "row stride"), (dict(ld_weight=7), "row stride"), (dict(dtype=7), "float type")):
            assert call(m, head=_head(m, **kw)) == m.EINVAL and word in m.last_error(), (kw, m.last_error())
        assert call(m, head=_head(m, rows=0)) == m.ESHAPE
        assert call(m, taken=None) == m.EINVAL
        for bad in (float("nan"), float("inf")):
            assert call(m, scale=bad) == m.EINVAL and "scale" in m.last_error()
        assert call(m, ws=None) == m.EINVAL and call(m, ws=7 * BASE + 8) == m.EINVAL
        assert call(m, wb=16) == m.EINVAL and "too small" in m.last_error()
    assert _loss(m, nll=None) == m.EINVAL and _loss(m, lse=None) == m.EINVAL
    assert _grad(m, lse=None) == m.EINVAL
    assert _grad(m, dh=None, dw=None, db=None) == m.EINVAL and "no gradient" in m.last_error()
    assert _grad(m, ldh=7) == m.EINVAL and _grad(m, ldw=7) == m.EINVAL
    assert _grad(m, dh=8 * BASE + 1) == m.EINVAL


def test_shared_memory_is_refused(m):
    for kw in (dict(nll=5 * BASE), dict(loss=4 * BASE + 8), dict(lse=BASE + 16), dict(nll=3 * BASE), dict(ws=2 * BASE),
               dict(ws=4 * BASE - (1 << 20) + 16)):
        assert _loss(m, **kw) == m.EINVAL and "share memory" in m.last_error(), kw
    for kw in (dict(dh=BASE), dict(dw=2 * BASE + 64), dict(dh=9 * BASE + 32), dict(db=5 * BASE), dict(db=7 * BASE)):
        assert _grad(m, **kw) == m.EINVAL and "share memory" in m.last_error(), kw


def test_binding_refuses_tensors_the_kernels_cannot_read(m):
    import torch
    z = torch.zeros
    with pytest.raises(ValueError, match="device memory"):
        m.policy_loss(z(4, 8), z(5, 8), z(4, dtype=torch.int32), z(4), z(4), z(64, dtype=torch.uint8))
    with pytest.raises(ValueError, match="none of"):
        m.policy_loss_workspace(4, 4, 4, torch.float64, device="cpu")


def test_struct_matches_the_c_compiler(m, tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("gcc not available")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    names = {"iqlh_policy_head": m.PolicyHeadStruct, "iqlh_matrix": m.MatrixStruct, "iqlh_matrix_set": m.MatrixSetStruct}
    body = "".join(f'printf("%zu\\n", sizeof({c}));' + "".join(f'printf("%zu\\n", offsetof({c}, {f[0]}));' for f in k._fields_)
                   for c, k in names.items())
    src = tmp_path / "l.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "iqlher.h"\nint main(void) {' + body + "return 0;}")
    subprocess.run(["gcc", "-std=c11", "-Werror", "-I", os.path.join(root, "include"), str(src), "-o",
                    str(tmp_path / "l")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "l")], check=True, capture_output=True, text=True).stdout.split()]
    want = []
    for k in names.values():
        want += [ctypes.sizeof(k)] + [getattr(k, f[0]).offset for f in k._fields_]
    assert got == want
