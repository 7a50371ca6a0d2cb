"""Tensor lists and 4-bit matrices on streams other than the one that their
tensors come from: nothing here waits for the device between a call's
preparation and the call unless its documentation asks for it."""
import numpy as np
import pytest

from oracle import tensors as ref
from tests.gpu_util import dev, sync

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24


@pytest.fixture(scope="module")
def m():
    import offline_rl_step_amd as m
    return m


def _grads(seed, lens):
    import torch
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(n, generator=g).to(dev()) for n in lens]


def _host(ts):
    return [t.double().cpu().numpy() for t in ts]


def test_a_new_workspace_serves_another_stream_at_once(m):
    """The workspace's counter is in place when grad_norm_workspace returns,
    with other work queued on the stream that made it and non-zero bytes where
    the workspace comes to lie."""
    import torch
    ts = _grads(1, [30_000, 77])
    want = ref.norm(_host(ts), 0)
    s = m.TensorSet(ts)
    out = torch.full((8,), -7.0, device=dev())
    busy = torch.empty(1 << 28, device=dev())
    side = torch.cuda.Stream()
    size = m.grad_norm_workspace(s).numel()
    sync()
    for rep in range(8):
        used = torch.full((size,), 0xFF, dtype=torch.uint8, device=dev())
        del used
        busy.fill_(float(rep))
        ws = m.grad_norm_workspace(s)
        m.grad_norm(s, out[rep:rep + 1], ws, stream=side)
        del ws
    sync()
    for x in out.tolist():
        assert abs(x - want) <= (U32 * 1.0001 + 30_077 * 2.0 ** -53) * want


def test_norms_and_factors_of_clips_on_several_streams(m):
    """Sets dropped right after their calls on four streams, outputs that live
    to the end: every norm, factor and flat vector."""
    import torch
    streams = [torch.cuda.Stream() for _ in range(4)]
    lists = [_grads(30 + k, [50_000 + 7 * k, 33, 2000]) for k in range(4)]
    want = [ref.norm(_host(ts), 0) for ts in lists]
    outs = [torch.zeros((8, 2), device=dev()) for _ in range(4)]
    flats = [torch.zeros(sum(t.numel() for t in ts), device=dev()) for ts in lists]
    sync()
    for rep in range(8):
        for k, st in enumerate(streams):
            s = m.TensorSet(lists[k])
            m.grad_clip(s, 0.5, outs[k][rep], m.grad_norm_workspace(s), out_flat=flats[k], stream=st)
            del s
    sync()
    for k in range(4):
        c = 0.5 / want[k]
        for n, f in outs[k].tolist():
            assert abs(n - want[k]) <= (U32 * 1.0001 + 60_000 * 2.0 ** -53) * want[k] and abs(f - c) <= 1.01 * U32 * c
        x = np.concatenate(_host(lists[k]))
        assert np.all(np.abs(flats[k].double().cpu().numpy() - x * c) <= 2 * U32 * 1.001 * np.abs(x * c) + 2.0 ** -149)


def test_calls_on_the_default_stream_of_a_set_made_on_another(m):
    import torch
    ts = _grads(9, [300_000, 5])
    want = ref.norm(_host(ts), 0)
    out = torch.zeros(6, device=dev())
    side = torch.cuda.Stream()
    sync()
    for rep in range(6):
        with torch.cuda.stream(side):
            s = m.TensorSet(ts)
            ws = m.grad_norm_workspace(s)
            m.grad_norm(s, out[rep:rep + 1], ws, stream=torch.cuda.default_stream())
            del s, ws
    sync()
    for x in out.tolist():
        assert abs(x - want) <= (U32 * 1.0001 + 300_005 * 2.0 ** -53) * want


def test_a_sets_memory_stays_when_its_tensors_move(m):
    """A tensor of the set that is given other storage (t.data = ..) leaves its
    old memory to the set: nothing else gets it while the set lives."""
    import torch
    n = 3_000_000
    t = torch.ones(n, device=dev())
    at = t.data_ptr()
    s = m.TensorSet([t])
    t.data = torch.full((n,), 2.0, device=dev())
    others = [torch.full((n,), 9.0, device=dev()) for _ in range(4)]
    assert all(o.data_ptr() != at for o in others)
    out = torch.zeros(1, device=dev())
    m.grad_norm(s, out, m.grad_norm_workspace(s))
    sync()
    assert abs(float(out[0]) - n ** 0.5) <= U32 * 1.0001 * n ** 0.5
