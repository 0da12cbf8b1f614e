"""Options of the AdamW optimizer's groups (host)."""
import pytest

torch = pytest.importorskip("torch")

import linear_recurrence_sequence_diag_amd as lr  # noqa: E402


def _param():
    return torch.nn.Parameter(torch.zeros(3))


def test_a_groups_options_have_the_constructors_names():
    groups = [{"params": [_param()], "rate": 1e-4, "weight_decay": 0.0}, {"params": [_param()], "lr": 2e-4},
              {"params": [_param()], "state_bits": 8, "master": True}]
    opt = lr.AdamW(groups, rate=1e-2)
    assert [g["lr"] for g in opt.param_groups] == [1e-4, 2e-4, 1e-2]
    assert [g["weight_decay"] for g in opt.param_groups] == [0.0, 1e-2, 1e-2]
    assert [g["state_bits"] for g in opt.param_groups] == [32, 32, 8]
    assert all("rate" not in g for g in opt.param_groups) and "rate" in groups[0]
    opt.add_param_group({"params": [_param()], "rate": 5e-4})
    assert opt.param_groups[3]["lr"] == 5e-4


def test_refusals():
    for bad in ({"rate": 1e-4, "lr": 1e-4}, {"state_bits": 16}):
        with pytest.raises(ValueError):
            lr.AdamW([{"params": [_param()], **bad}])
    with pytest.raises(TypeError):
        lr.AdamW([_param()]).add_param_group([_param()])
