"""Which stream the binding tells torch's allocator of, without a GPU: torch's
stream calls and the tensors' record_stream are stand-ins that keep a log."""
import pytest

HOME, SIDE = 0x1000, 0x2000


@pytest.fixture(scope="module")
def m():
    import offline_rl_step_amd as m
    return m


class Recorded:
    """A tensor as far as record_stream goes."""

    def __init__(self):
        self.streams = []

    def record_stream(self, stream):
        self.streams.append(stream)


@pytest.fixture
def streams(m, monkeypatch):
    import torch

    def external(handle, device=None):
        # what torch does with a handle of 0: a stream of its own pool
        return ("pool", None) if handle == 0 else ("external", handle)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: ("external", 0))
    monkeypatch.setattr(torch.cuda, "ExternalStream", external)


def _set(m, home):
    import torch
    s = object.__new__(m.TensorSet)
    s.table, s.device, s._streams, s._memory = Recorded(), torch.device("cuda", 0), {home}, []
    return s


@pytest.mark.parametrize("home,used", [(HOME, 0), (0, HOME), (HOME, SIDE)])
def test_a_sets_table_is_kept_for_the_stream_that_reads_it(m, streams, home, used):
    s = _set(m, home)
    assert s._used_on(used) == used
    assert s.table.streams == [("external", used)]


def test_a_sets_table_needs_nothing_on_its_own_stream(m, streams):
    for home in (0, HOME):
        s = _set(m, home)
        s._used_on(home)
        assert s.table.streams == []


@pytest.fixture
def calls(m, streams, monkeypatch):
    """The library's calls succeed without doing anything, tensors in host memory
    pass for device memory, HOME is the current stream; the log of
    record_stream, (address of the tensor's memory, stream)."""
    import torch
    log = []
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda self, s: log.append((self.data_ptr(), s)), raising=False)
    monkeypatch.setattr(m, "_need_current", lambda device: 0)
    monkeypatch.setattr(m, "_get_device", lambda: 0)
    monkeypatch.setattr(m, "_raw_stream", lambda index: HOME)
    for name in ("grad_norm", "grad_clip", "mx4_quantize", "mx4_dequantize", "mx4_matmul", "mx4_linear", "forward_mx4"):
        monkeypatch.setattr(m, f"_lib_{name}", lambda *args: m.OK)
    return log


def _jobs(m):
    """(call, the tensors whose memory it touches)"""
    import torch
    f = lambda *shape: torch.zeros(shape)  # noqa: E731
    u = lambda n: torch.zeros(n, dtype=torch.uint8)  # noqa: E731
    grads = [f(40), f(3)]
    s = m.TensorSet(grads)
    norm, each, flags, ws, out, flat = f(1), f(2), torch.zeros(1, dtype=torch.int32), u(1 << 16), f(2), f(43)
    a, b = (m.Mx4(u(64).view(4, 16), u(4).view(4, 1), 4, 32) for _ in range(2))
    x, y, bias, work = f(4, 32), f(4, 4), f(4), u(64)
    values, target, rewards, dones = f(4), f(4), f(4), f(4)
    qa, qb = [a.codes, a.scales], [b.codes, b.scales]
    kept = [s.table, *grads]
    return {
        "grad_norm": (lambda st: m.grad_norm(s, norm, ws, out_each=each, flags=flags, stream=st),
                      kept + [norm, each, flags, ws]),
        "grad_clip": (lambda st: m.grad_clip(s, 1.0, out, ws, out_flat=flat, flags=flags, stream=st),
                      kept + [out, flat, flags, ws]),
        "mx4_quantize": (lambda st: m.mx4_quantize(x, a, stream=st), [x] + qa),
        "mx4_dequantize": (lambda st: m.mx4_dequantize(a, x, stream=st), [x] + qa),
        "mx4_matmul": (lambda st: m.mx4_matmul(a, b, y, work, bias=bias, stream=st), qa + qb + [y, work, bias]),
        "mx4_linear": (lambda st: m.mx4_linear(x, b, y, work, bias=bias, stream=st), qb + [x, y, work, bias]),
        "forward_values_mx4": (lambda st: m.iql_forward_values_mx4(None, x, 4, values, work, rewards, dones, 0.9, target,
                                                                   stream=st), [x, values, work, rewards, dones, target]),
    }


JOBS = ["grad_norm", "grad_clip", "mx4_quantize", "mx4_dequantize", "mx4_matmul", "mx4_linear", "forward_values_mx4"]


@pytest.mark.parametrize("name", JOBS)
def test_a_calls_tensors_are_kept_for_the_stream_it_names(m, calls, name):
    call, tensors = _jobs(m)[name]
    call(SIDE)
    assert sorted(calls) == sorted((t.data_ptr(), ("external", SIDE)) for t in tensors)


@pytest.mark.parametrize("name", JOBS)
def test_calls_on_the_current_stream_record_nothing(m, calls, name):
    call, _ = _jobs(m)[name]
    call(None)
    call(HOME)
    assert calls == []


@pytest.mark.parametrize("capturing", [False, True])
def test_a_workspaces_counter_is_zero_for_any_stream(m, calls, monkeypatch, capturing):
    """When grad_norm_workspace returns, the counter is 0 whatever fills the
    current stream still has to run (here: none has run).  Into a captured graph
    the fill is recorded."""
    import torch
    s = m.TensorSet([torch.zeros(5)])
    empty, fills = torch.empty, []
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing)
    monkeypatch.setattr(torch, "empty", lambda *a, **k: empty(*a, **k).fill_(0xA5))
    monkeypatch.setattr(torch.Tensor, "zero_", lambda self: fills.append(self.numel()) or self)
    ws = m.grad_norm_workspace(s)
    if capturing:
        assert fills == [64]
    else:
        assert ws[:64].tolist() == [0] * 64


def test_a_sets_memory_stays_when_its_tensors_move(m, calls):
    """The storage that the table's addresses lie in lives as long as the set."""
    import gc
    import weakref
    import torch
    t = torch.zeros(1000)
    s = m.TensorSet([t])
    freed = []

    class Canary:
        pass
    canary = Canary()
    weakref.finalize(canary, lambda: freed.append(1))
    t.untyped_storage()._kept = canary  # the storage's Python object lives with it
    old = t.untyped_storage()._cdata
    del canary
    t.data = torch.ones(1000)
    assert t.untyped_storage()._cdata != old
    gc.collect()
    assert not freed
    s = None
    gc.collect()
    assert freed
