"""What the binding of V(s) in 4 bits refuses, without a GPU: tensors in host
memory pass for device memory where the check in question is another, and a call
that reaches the library is noted."""
import pytest

GROUPS, S, B = 2, 8, 6


@pytest.fixture(scope="module")
def m():
    import offline_rl_step_amd as m
    return m


def _args():
    import torch
    return dict(next_states=torch.zeros(B, S), batch=B, out_v=torch.zeros(GROUPS, B),
                workspace=torch.zeros(64, dtype=torch.uint8), rewards=torch.zeros(B), dones=torch.zeros(B),
                out_target=torch.zeros(GROUPS, B))


@pytest.fixture
def trainer(m, monkeypatch):
    t = object.__new__(m.IqlTrainer)
    t.h, t.cfg, t.calls = None, m.make_config(S, 32, B, num_groups=GROUPS), []
    monkeypatch.setattr(m, "_lib_forward_mx4", lambda *a: t.calls.append(a) or m.OK)
    monkeypatch.setattr(m.IqlTrainer, "__del__", lambda self: None, raising=False)
    return t


def test_host_memory_is_refused(m, trainer):
    with pytest.raises(ValueError, match="device memory"):
        trainer.forward_values_mx4(**_args())
    assert trainer.calls == []


@pytest.fixture
def on_device(m, monkeypatch):
    monkeypatch.setattr(m, "_need_current", lambda device: 0)
    monkeypatch.setattr(m, "_raw_stream", lambda index: 0)


def test_good_arguments_reach_the_library(m, trainer, on_device):
    import torch
    wide = torch.zeros(B, S + 3)
    for over in ({}, dict(rewards=None, dones=None, out_target=None), dict(next_states=wide[:, :S]),
                 dict(next_states=torch.zeros(B + 1, S)), dict(next_states=torch.zeros(B * S), states_ld=S),
                 dict(next_states=torch.zeros(B, S, dtype=torch.bfloat16)), dict(out_v=torch.zeros(GROUPS * B + 5))):
        trainer.calls.clear()
        trainer.forward_values_mx4(**{**_args(), **over})
        assert len(trainer.calls) == 1
    assert trainer.calls[0][3] == S


@pytest.mark.parametrize("what", ["columns", "rows", "type", "few_columns", "no_rows", "workspace", "out_v", "out_v_type",
                                  "out_v_stride", "rewards", "dones", "out_target"])
def test_bad_arguments_do_not(m, trainer, on_device, what):
    import torch
    over = {"columns": dict(next_states=torch.zeros(S, B).t()),
            "rows": dict(next_states=torch.zeros(B - 1, S)),
            "type": dict(next_states=torch.zeros(B, S, dtype=torch.float16)),
            "few_columns": dict(next_states=torch.zeros(B, S - 1), states_ld=S),
            "no_rows": dict(next_states=torch.zeros(B * S)),
            "workspace": dict(workspace=torch.zeros(64, 2, dtype=torch.uint8)[:, 0]),
            "out_v": dict(out_v=torch.zeros(GROUPS * B - 1)),
            "out_v_type": dict(out_v=torch.zeros(GROUPS, B, dtype=torch.float64)),
            "out_v_stride": dict(out_v=torch.zeros(B, GROUPS).t()),
            "rewards": dict(rewards=torch.zeros(B - 1)),
            "dones": dict(dones=torch.zeros(B, dtype=torch.bool)),
            "out_target": dict(out_target=torch.zeros(B))}[what]
    with pytest.raises(ValueError):
        trainer.forward_values_mx4(**{**_args(), **over})
    assert trainer.calls == []
