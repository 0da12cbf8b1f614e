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


@pytest.mark.parametrize("value", [float("nan"), float("inf"), 100.0, 1000.0, float("-inf")])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T", [150, 1700])
def test_a_segments_first_decay_is_not_used(T, dt, value):
    """No value of log_decay where a segment starts changes a bit of any result, in the segment or outside."""
    _, args, go = _inputs(1, T, 2, 1, 64, 32, dt, 3)
    reset = torch.zeros(1, T, dtype=torch.bool, device="cuda")
    cuts = [5, 64, 100, 101, T - 40]
    reset[:, cuts] = True

    def results(log_decay, r):
        x = (*args[:3], log_decay, args[4])
        return lr.delta_scan(*x, reset=r) + lr.delta_scan_backward(*x, go, reset=r)[:5]

    bad, zero = args[3].clone(), args[3].clone()
    at = [0] + cuts  # the row's first token has no state to decay either
    bad[:, at], zero[:, at] = value, 0.0
    for a, b in zip(results(zero, reset), results(bad, reset)):
        assert torch.isfinite(a).all() and torch.equal(a, b)
    bad[:, cuts] = zero[:, cuts]
    for a, b in zip(results(zero, None), results(bad, None)):
        assert torch.isfinite(a).all() and torch.equal(a, b)


@pytest.mark.parametrize("T", [40, 1300])
def test_the_initial_states_gradient_where_there_is_none(T):
    """grad_h0 of a call without h0 is that of a call from zeros, the first step's decay in it."""
    _, args, go = _inputs(2, T, 2, 1, 64, 32, "f32", 4)
    zeros = torch.zeros(2, 2, 64, 32, device="cuda")
    got = lr.delta_scan_backward(*args, go, need_grad_h0=True)
    want = lr.delta_scan_backward(*args, go, h0=zeros, need_grad_h0=True)
    for a, b in zip(got, want):  # both keep the bounds of fp32 blocks, 64 u of the largest each
        assert (a - b).abs().max() <= 2 * 64 * D.U * b.abs().max()
    assert all(torch.equal(a, b) for a, b in zip(got, lr.delta_scan_backward(*args, go)[:5]))


def test_a_prompt_and_its_tokens_one_by_one_agree_at_segment_starts():
    """The steps drop the same decays as the blocks."""
    T = 70
    x, args, _ = _inputs(2, T, 2, 1, 32, 16, "f32", 5)
    reset = torch.zeros(2, T, dtype=torch.bool)
    reset[0, [3, 64]] = reset[1, [20, 66]] = True
    x["log_decay"][reset] = float("nan")
    args[3] = x["log_decay"].cuda()
    ref = D.forward(*[x[n].double() for n in NAMES], 0.25, reset)
    f32 = D.forward(*[x[n] for n in NAMES], 0.25, reset)
    out, last = lr.delta_scan(*args, scale=0.25, reset=reset.cuda())
    state = None
    for t in range(T):
        step, state = lr.delta_step(*[a[:, t] for a in args], state, scale=0.25, reset=reset[:, t].contiguous().cuda())
        D.check("out", step, ref[0][:, t], f32[0][:, t], torch.float32)
    for name, got, a, b in (("out", out, ref[0], f32[0]), ("last", last, ref[1], f32[1]), ("last", state, ref[1], f32[1])):
        D.check(name, got, a, b, torch.float32)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 300, 2, 1, 64, 40), (1, 1300, 2, 2, 128, 33), (1, 140, 1, 1, 200, 20)], ids=str)
def test_outputs_before_a_value_that_is_not_finite(shape, dt, value):
    """The recurrence is causal: a row's outputs in front of such a value, as of padding behind a sequence, are what
    they are without it; from it on, and in the last state, they are not finite where they depend on it."""
    T, V = shape[1], shape[-1]
    x, args, _ = _inputs(*shape, dt, 6)
    ref, f32 = ([t for t in D.forward(*[x[n].to(kind) for n in NAMES], 0.25)[:1]] for kind in (torch.float64, torch.float32))
    clean, last = lr.delta_scan(*args, scale=0.25)
    for t in sorted({0, 1, 15, 16, 40, 63, 64, 97, T - 1}):
        for i, name in enumerate(NAMES):
            bad = [a.clone() for a in args]
            bad[i][:, t] = value
            out, state = lr.delta_scan(*bad, scale=0.25)
            if name in ("q", "v"):  # no rounding before it differs
                assert torch.equal(out[:, :t], clean[:, :t]), (name, t)
            elif t > 0:
                D.check("out", out[:, :t], ref[0][:, :t], f32[0][:, :t], DT[dt])
            if name == "q":
                assert torch.equal(out[:, t + 1:], clean[:, t + 1:]) and torch.equal(state, last)
                assert not torch.isfinite(out[:, t]).any()
            elif name != "log_decay" or t > 0:  # the first one is not used
                assert not torch.isfinite(out[:, t:]).all(-1).any() and not torch.isfinite(state).all(-1).any(), (name, t)
        # one value of one head reaches its column alone
        bad = args[2].clone()
        bad[0, t, 0, V // 2] = value
        out, state = lr.delta_scan(*args[:2], bad, *args[3:], scale=0.25)
        mine = torch.zeros_like(out, dtype=torch.bool)
        mine[:, t:, 0, V // 2] = True
        assert torch.equal(out[~mine], clean[~mine]) and not torch.isfinite(out[mine]).any()
        column = torch.zeros_like(state, dtype=torch.bool)
        column[:, 0, :, V // 2] = True
        assert torch.equal(state[~column], last[~column]) and not torch.isfinite(state[column]).any()


@pytest.mark.parametrize("value", [float("nan"), float("-inf")])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 300, 2, 1, 64, 40), (1, 1300, 2, 2, 128, 33), (1, 140, 1, 1, 200, 20)], ids=str)
def test_gradients_behind_an_outputs_gradient_that_is_not_finite(shape, dt, value):
    """An output does not depend on the steps behind it, so neither do their gradients on its own."""
    T = shape[1]
    _, args, go = _inputs(*shape, dt, 7)
    clean = lr.delta_scan_backward(*args, go)[:5]
    for t in sorted({0, 15, 16, 40, 63, 64, 97, T - 1}):
        bad = go.clone()
        bad[:, t] = value
        for a, b in zip(clean, lr.delta_scan_backward(*args, bad)[:5]):
            assert torch.equal(a[:, t + 1:], b[:, t + 1:]), t
        # and of the queries' gradients, the step's own alone
        assert torch.equal(clean[0][:, :t], lr.delta_scan_backward(*args, bad)[0][:, :t])


def test_values_past_the_type_of_the_products():
    """A finite value that no bf16 holds counts as an infinity, from its own step on."""
    _, args, _ = _inputs(1, 100, 1, 1, 32, 16, "f32", 8)
    clean = lr.delta_scan(*args)[0]
    args[2] = args[2].clone()
    args[2][:, 50] = torch.finfo(torch.float32).max
    out = lr.delta_scan(*args)[0]
    assert torch.equal(out[:, :50], clean[:, :50])
