"""The gated delta rule's kernels: results that agree whatever else a call asks for."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import _delta as D  # noqa: E402
import linear_recurrence_sequence_diag_amd as lr  # noqa: E402

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
NAMES = ("q", "k", "v", "log_decay", "beta")


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lr.library()


def _inputs(B, T, H, HK, K, V, dt, seed):
    x = D.inputs(B, T, H, HK, K, V, DT[dt], seed)
    return x, [x[n].cuda() for n in NAMES], x["grad_out"].cuda()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(2, 200, 4, 2, 128, 128), (1, 1700, 2, 1, 64, 40), (1, 150, 3, 1, 33, 7),
                                   (1, 130, 2, 2, 256, 48)], ids=str)
def test_outputs_do_not_depend_on_the_last_state(shape, dt):
    """Outputs alone, outputs beside the last state and outputs of a row walked in parts have one accuracy."""
    _, args, _ = _inputs(*shape, dt, 1)
    out, last = lr.delta_scan(*args)
    alone, none = lr.delta_scan(*args, with_last=False)
    assert none is None and torch.equal(out, alone)
    none, state = lr.delta_scan(*args, with_out=False)
    assert none is None and torch.equal(last, state)
