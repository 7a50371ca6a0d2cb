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
    s.table, s.device, s._home = Recorded(), torch.device("cuda", 0), home
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
