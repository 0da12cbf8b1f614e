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


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,dense", [(1024, [(965, 1024)]), (2048, [(65, 128)]), (1700, [(600, 700), (1300, 1310)]),
                                     (1300, [(0, 70), (640, 642), (1299, 1300)])], ids=str)
def test_gradients_of_rows_in_parts_where_segments_start_densely(T, dense, dt):
    """Runs of one-token segments, as of a padding tail, at and around the ends of parts of a row."""
    B, H, HK, K, V = 1, 2, 1, 64, 32
    x, args, go = _inputs(B, T, H, HK, K, V, dt, 2)
    reset = torch.zeros(B, T, dtype=torch.bool)
    for lo, hi in dense:
        reset[:, lo:hi] = True
    ref, f32 = ({n: t for n, t in D.backward(*[x[n].to(kind) for n in NAMES], 0.25, x["grad_out"].to(kind), reset,
                                             x["h0"].to(kind), x["grad_last"].to(kind)).items()}
                for kind in (torch.float64, torch.float32))
    state = dict(h0=x["h0"].cuda(), grad_last=x["grad_last"].cuda(), need_grad_h0=True)
    names = ("grad_q", "grad_k", "grad_v", "grad_log_decay", "grad_beta", "grad_h0")
    for repeat in range(3):
        got = lr.delta_scan_backward(*args, go, scale=0.25, reset=reset.cuda(), **state)
        for n, t in zip(names, got):
            D.check(n, t, ref[n], f32[n], DT[dt])
        if repeat:
            assert all(torch.equal(a, b) for a, b in zip(first, got))
        else:
            first = got
