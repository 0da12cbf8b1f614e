"""The 64-bit form of the gated delta rule, its gradients against differences, the
refusals of the entry points (no GPU), and the sizes of its workspaces."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import _delta as D  # noqa: E402
import linear_recurrence_sequence_diag_amd as lr  # noqa: E402
from test_abi import _lib  # noqa: E402

NAMES = ("q", "k", "v", "log_decay", "beta", "h0")


def test_gradients_against_differences():
    B, T, H, HK, K, V = 2, 7, 4, 2, 5, 3
    x = {n: t.double() for n, t in D.inputs(B, T, H, HK, K, V, torch.float32, 3).items()}
    reset = torch.zeros(B, T, dtype=torch.bool)
    reset[0, 3] = reset[1, 0] = True
    scale = 0.7

    def loss(*a):
        out, last, _ = D.forward(*a[:5], scale, reset, a[5])
        return (out * x["grad_out"]).sum() + (last * x["grad_last"]).sum()

    args = [x[n] for n in NAMES]
    got = D.backward(*args[:5], scale, x["grad_out"], reset, x["h0"], x["grad_last"])
    gen = torch.Generator().manual_seed(1)
    for i, n in enumerate(NAMES):
        for _ in range(4):
            d = torch.randn(args[i].shape, generator=gen, dtype=torch.float64)
            h = 1e-5
            up, down = ([a + s * h * d if j == i else a for j, a in enumerate(args)] for s in (1, -1))
            diff = (loss(*up) - loss(*down)) / (2 * h)
            want = (got["grad_" + n] * d).sum()
            # a central difference errs by h^2 of the third derivative and u64 / h of the loss
            assert abs(diff - want) <= 1e-6 * (1 + abs(want)), n


def test_one_token_by_hand():
    q, k = torch.tensor([0.6, 0.8]).view(1, 1, 1, 2).double(), torch.tensor([1.0, 0.0]).view(1, 1, 1, 2).double()
    v = torch.tensor([2.0]).view(1, 1, 1, 1).double()
    g, beta = torch.tensor([0.5]).log().view(1, 1, 1).double(), torch.tensor([0.25]).view(1, 1, 1).double()
    h0 = torch.tensor([[4.0], [8.0]]).view(1, 1, 2, 1).double()
    out, last, _ = D.forward(q, k, v, g, beta, 1.0, None, h0)
    # a S = (2, 4); it gives 2 for the key, as the value asks: nothing is written
    assert torch.allclose(last.flatten(), torch.tensor([2.0, 4.0]).double())
    assert torch.allclose(out.flatten(), torch.tensor([0.6 * 2 + 0.8 * 4]).double())


P = 256  # a pointer that is never followed


def _call(fn, shape=(2, 100, 4, 2, 64, 32), dtype=0, strides=None, opts=None, scale=1.0, null=None, sizes=None):
    n = {"scan_delta_fwd": 5, "scan_delta_bwd": 5, "scan_delta_step": 5}[fn]
    outs = {"scan_delta_fwd": 2, "scan_delta_bwd": 7, "scan_delta_step": 4}[fn]
    args = [P] * n + [scale] + [P] * outs
    if null is not None:
        for i in null:
            args[i if i < 5 else i + 1] = None
    if fn == "scan_delta_step":
        shape = shape[:1] + shape[2:]
    args += [*shape, dtype, strides, None]
    if fn != "scan_delta_step":
        args.append(opts)
    with pytest.raises(lr.LRScanError) as e:
        getattr(lr, fn)(*args)
    return e.value.status


@pytest.mark.parametrize("fn", ["scan_delta_fwd", "scan_delta_bwd", "scan_delta_step"])
def test_refusals_before_any_work(fn):
    _lib()
    for i in range(5):
        assert _call(fn, null=[i]) == -1
    if fn == "scan_delta_fwd":
        assert _call(fn, null=[5, 6]) == -1
    if fn == "scan_delta_step":
        assert _call(fn, null=[7, 8]) == -1
    for bad in ((0, 100, 4, 2, 64, 32), (2, 100, 4, 0, 64, 32), (2, 100, 4, 2, 0, 32), (2, 100, 4, 2, 64, 0),
                (2, 100, 5, 2, 64, 32), (2, 100, 2, 4, 64, 32), (2, 100, 4, 2, 257, 32), (2, 100, 4, 2, 64, 65537),
                (2, 100, 70000, 2, 64, 32), (1 << 40, 100, 4, 2, 64, 32), (1 << 28, 100, 4, 2, 64, 32)):
        assert _call(fn, shape=bad) == -2, bad
    if fn != "scan_delta_step":
        assert _call(fn, shape=(2, 0, 4, 2, 64, 32)) == -2
        assert _call(fn, shape=(1, (1 << 30) + 1, 4, 2, 64, 32)) == -2
    assert _call(fn, dtype=2) == -3
    for scale in (float("nan"), float("inf")):
        assert _call(fn, scale=scale) == -10
    per = 2 if fn == "scan_delta_step" else 3
    for i in range(5 * per):
        s = [64] * (5 * per)
        s[i] = -1
        assert _call(fn, strides=s) == -10
    if fn != "scan_delta_step":
        for algo in (1, 2, 3, 9):
            assert _call(fn, opts=lr.make_opts(algo)) == -7
        assert _call(fn, opts=lr.make_opts(chunk=64)) == -4
        o = lr.make_opts()
        need = lr.scan_delta_workspace_bytes(2, 100, 4, 2, 64, 32, 0, fn == "scan_delta_bwd")
        o.workspace, o.workspace_bytes = P, need // 2
        assert _call(fn, opts=o) == -5
        o.workspace, o.workspace_bytes = P + 8, 2 * need
        assert _call(fn, opts=o) == -5


def test_workspace_sizes():
    _lib()
    size = lr.scan_delta_workspace_bytes
    assert size(2, 100, 4, 2, 64, 32, 0, 0) >= 2 * 100 * 4 * 2 * 64 * 4
    assert size(2, 100, 4, 2, 64, 32, 0, 1) > size(2, 100, 4, 2, 64, 32, 0, 0)
    assert size(2, 100, 3, 2, 64, 32, 0, 0) == 0 and size(2, 0, 4, 2, 64, 32, 0, 1) == 0


def test_tensor_helpers_refuse():
    x = D.inputs(1, 3, 2, 1, 8, 4, torch.float32, 0)
    args = [x[n] for n in NAMES[:5]]
    for call in (lambda: lr.delta_scan(*args), lambda: lr.delta_scan_backward(*args, x["grad_out"]),
                 lambda: lr.delta_step(*[t[:, 0] for t in args])):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    assert ctypes.sizeof(lr.Opts) > 0
