"""The gated delta rule's kernels against the 64-bit walk: lengths from one token
on, blocks that resets cut, head widths and groups, strided operands, states,
graphs, streams and workspaces."""
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


def _reset(B, T, kind, seed=0):
    if kind is None:
        return None
    r = torch.zeros(B, T, dtype=torch.bool)
    if kind == "all":
        r[:] = True
    elif kind == "some":
        r[torch.rand(B, T, generator=torch.Generator().manual_seed(seed)) < 0.03] = True
        r[0, 0] = True
    elif kind == "edges":  # at, before and behind a block's first token, and the last token
        for t in (63, 64, 65, 128, T - 1):
            if 0 <= t < T:
                r[:, t] = True
    return r


def _case(B, T, H, HK, K, V, dt, kind=None, state=False, seed=0, **more):
    x = D.inputs(B, T, H, HK, K, V, DT[dt], seed, **more)
    return x, _reset(B, T, kind, seed), (x["h0"] if state else None), (x["grad_last"] if state else None)


def _refs(x, reset, h0, gl, scale, back):
    out = []
    for kind in (torch.float64, torch.float32):
        y = {n: t.to(kind) for n, t in x.items()}
        s = None if h0 is None else y["h0"]
        f = dict(zip(("out", "last"), D.forward(*[y[n] for n in NAMES], scale, reset, s)[:2]))
        if back:
            f |= D.backward(*[y[n] for n in NAMES], scale, y["grad_out"], reset, s,
                            None if gl is None else y["grad_last"])
        out.append(f)
    return out


def _run(x, reset, h0, gl, scale, back, dt, call=None):
    dev = {n: t.cuda() for n, t in x.items()}
    args = [dev[n] for n in NAMES]
    r = None if reset is None else reset.cuda()
    s = None if h0 is None else dev["h0"]
    ref, f32 = _refs(x, reset, h0, gl, scale, back)
    got = dict(zip(("out", "last"), lr.delta_scan(*args, scale=scale, h0=s, reset=r)))
    if back:
        g = lr.delta_scan_backward(*args, dev["grad_out"], scale=scale, h0=s, reset=r, need_grad_h0=True,
                                   grad_last=None if gl is None else dev["grad_last"])
        got |= dict(zip(("grad_q", "grad_k", "grad_v", "grad_log_decay", "grad_beta", "grad_h0"), g))
    for n, t in got.items():
        ratio = D.check(n, t, ref[n], f32[n], DT[dt])
        print(f"{n}: {ratio:.2f} of the bound")
    return got, dev


SHAPES = [  # B, T, H, HK, K, V, kind, state
    (1, 1, 1, 1, 1, 1, None, True),
    (2, 1, 4, 2, 64, 64, None, False),
    (1, 2, 2, 1, 33, 7, None, True),
    (2, 63, 2, 2, 64, 32, None, True),
    (1, 64, 2, 2, 128, 128, None, False),
    (1, 65, 3, 1, 128, 128, None, True),
    (2, 200, 4, 2, 128, 128, "some", True),
    (1, 257, 2, 2, 256, 48, "some", True),
    (1, 150, 6, 2, 70, 101, "edges", True),
    (2, 130, 2, 1, 192, 33, "edges", False),
    (1, 70, 1, 1, 96, 256, "all", True),
    (9, 129, 3, 3, 40, 16, "some", True),
]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=["x".join(map(str, s[:6])) + f"-{s[6]}" for s in SHAPES])
def test_forward(shape, dt):
    B, T, H, HK, K, V, kind, state = shape
    x, reset, h0, gl = _case(B, T, H, HK, K, V, dt, kind, state)
    _run(x, reset, h0, gl, 0.25, False, dt)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=["x".join(map(str, s[:6])) + f"-{s[6]}" for s in SHAPES])
def test_backward(shape, dt):
    B, T, H, HK, K, V, kind, state = shape
    x, reset, h0, gl = _case(B, T, H, HK, K, V, dt, kind, state, seed=1)
    _run(x, reset, h0, gl, 0.25, True, dt)
