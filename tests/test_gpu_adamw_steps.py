"""The AdamW optimizer's steps as a training program meets them: refused ones,
groups with options of their own, and autograd beside updates in place."""
import copy
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import linear_recurrence_sequence_diag_amd as lr  # noqa: E402


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lr.library()


def _params(*sizes, dtype=torch.float32, seed=0):
    gen = torch.Generator().manual_seed(seed)
    ps = [torch.nn.Parameter(torch.randn(n, generator=gen).to(dtype).cuda()) for n in sizes]
    for p in ps:
        p.grad = torch.randn(p.shape, generator=gen).to(dtype).cuda()
    return ps


def _held(opt):
    """Weights and states of an optimizer, copied."""
    return ([p.detach().clone() for g in opt.param_groups for p in g["params"]], copy.deepcopy(opt.state_dict()["state"]))


def _same(a, b):
    assert all(torch.equal(x, y) for x, y in zip(a[0], b[0])) and a[1].keys() == b[1].keys()
    for i, s in a[1].items():
        assert s.keys() == b[1][i].keys()
        for name, x in s.items():
            y = b[1][i][name]
            assert torch.equal(x.float(), y.float()) if isinstance(x, torch.Tensor) else x == y, name


@pytest.mark.parametrize("bits,master", [(32, True), (8, False)])
@pytest.mark.parametrize("steps", [0, 2])
def test_a_refused_step_changes_nothing(steps, bits, master):
    """Whatever group the fault is in; the next step is the one that would have come without it."""
    def fresh():
        ps = _params(300, 7, 33, dtype=torch.bfloat16)
        groups = [{"params": ps[:2]}, {"params": ps[2:], "weight_decay": 0.3}]
        return ps, lr.AdamW(groups, rate=1e-2, state_bits=bits, master=master)

    ps, opt = fresh()
    qs, other = fresh()
    for _ in range(steps):
        opt.step()
        other.step()
    before = _held(opt)
    refused = [lambda: opt.step(grad_scale=2.0), lambda: opt.step(grad_scale=torch.ones(1, device="cuda").double())]
    for name, value in (("lr", math.nan), ("betas", (0.9, 1.0)), ("eps", -1.0), ("weight_decay", math.inf)):
        def odd(name=name, value=value):
            group = opt.param_groups[1]
            keep, group[name] = group[name], value
            try:
                opt.step()
            finally:
                group[name] = keep
        refused.append(odd)

    def sparse():
        keep, ps[2].grad = ps[2].grad, None
        ps[2].grad = torch.zeros(33, device="cuda", dtype=torch.bfloat16).to_sparse()
        try:
            opt.step()
        finally:
            ps[2].grad = keep

    refused.append(sparse)
    for call in refused:
        with pytest.raises((ValueError, lr.LRScanError)):
            call()
        _same(before, _held(opt))
    if not steps:  # nothing was taken of the weights either
        for p, q in zip(ps, qs):
            with torch.no_grad():
                p.mul_(2)
                q.mul_(2)
    opt.step()
    other.step()
    _same(_held(other), _held(opt))


@pytest.mark.parametrize("dtype,master", [(torch.float32, False), (torch.bfloat16, True)])
def test_a_graph_from_before_an_update_is_refused(dtype, master):
    """As with torch's optimizers: a backward through weights that a step has changed since raises."""
    (w,) = _params(40, dtype=dtype)
    opt = lr.AdamW([w], master=master)
    loss = (w * w).sum()
    loss.backward(retain_graph=True)
    opt.step()
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        loss.backward()
    (w * w).sum().backward()  # a graph of the weights as they are now
    # the update of lists tells it too
    loss = (w * w).sum()
    states = [torch.zeros(40, device="cuda") for _ in range(2)]
    masters = [w.detach().float()]
    seen = masters[0]._version
    lr.adamw_update([w.detach()], [w.grad], [states[0]], [states[1]], 1, masters=masters)
    assert masters[0]._version > seen
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        loss.backward()


def test_other_results_in_place_are_seen_too():
    z = torch.randn(2, 50, device="cuda", requires_grad=True)
    y = z.exp()
    loss = (y * y).sum()
    lr.adjust_logits(y.detach(), bias_ids=torch.zeros(2, 1, dtype=torch.int64, device="cuda"),
                     bias=torch.ones(2, 1, device="cuda"), out=y.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        loss.backward()
    state = torch.randn(1, 1, 8, 8, device="cuda", requires_grad=True)
    kept = state * 1.0
    loss = (kept * kept).sum()
    rows = [torch.randn(1, 1, 8, device="cuda") for _ in range(3)] + [torch.zeros(1, 1, device="cuda")] * 2
    lr.delta_step(*rows, kept.detach(), out_state=kept.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        loss.backward()
    with torch.inference_mode():  # tensors without a version
        held = torch.zeros(1, 1, 8, 8, device="cuda")
        lr.delta_step(*rows, held, out_state=held)
        x = torch.randn(2, 50, device="cuda")
        lr.adjust_logits(x, out=x)
        p, g, m, v = (torch.ones(9, device="cuda") for _ in range(4))
        lr.adamw_update([p], [g], [m], [v], 1)
