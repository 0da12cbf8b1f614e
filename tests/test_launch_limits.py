"""Sizes whose launches would have 2^32 work-items or more are refused on the host,
before anything is enqueued; the largest ones that are not give what small calls give."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import linear_recurrence_sequence_diag_amd as lr  # noqa: E402

P = 256  # a pointer that is never followed
DIM = -2


@pytest.fixture(autouse=True, scope="module")
def _lib():
    try:
        lr.library()
    except Exception as e:  # not built
        pytest.skip(str(e))


def _status(call):
    with pytest.raises(lr.LRScanError) as e:
        call()
    return e.value.status


def _delta(B, T, H, HK, K=1, V=1, reset=False, back=False):
    opts = lr.make_opts()
    opts.workspace, opts.workspace_bytes = P, 0
    opts.reset = P if reset else None
    if back:
        return lr.scan_delta_bwd(*[P] * 5, 1.0, P, None, *[P] * 5, B, T, H, HK, K, V, 0, None, None, opts)
    return lr.scan_delta_fwd(*[P] * 5, 1.0, P, None, B, T, H, HK, K, V, 0, None, None, opts)


def test_delta():
    """A workspace of no bytes is the next thing that is refused (-5), so that nothing is enqueued here."""
    near = 1 << 23
    for B, T, H, HK, K, V, more, back in (
            (near - 8, 1, 1, 1, 1, 1, {}, False), (near // 64 - 1, 1, 64, 64, 1, 128, {}, False),
            ((1 << 22) - 1, 1, 1, 1, 1, 1, dict(reset=True), False), (1, (1 << 30) - 64, 1, 1, 1, 1, {}, False),
            ((near - 64) // 2, 65, 1, 1, 1, 1, {}, True)):
        assert _status(lambda: _delta(B, T, H, HK, K, V, back=back, **more)) == -5, (B, T, H)
    for B, T, H, HK, K, V, more, back in (
            (near - 7, 1, 1, 1, 1, 1, {}, False), (near // 64, 1, 64, 64, 1, 128, {}, False),
            (near // 128, 1, 64, 64, 1, 129, {}, False), (1 << 22, 1, 1, 1, 1, 1, dict(reset=True), False),
            (1, (1 << 30) - 63, 1, 1, 1, 1, {}, False), (near // 2, 65, 1, 1, 1, 1, {}, True),
            (1 << 17, 64 * 64, 2, 1, 1, 1, {}, False)):
        assert _status(lambda: _delta(B, T, H, HK, K, V, back=back, **more)) == DIM, (B, T, H)
    size = lr.scan_delta_workspace_bytes
    assert size(near - 8, 1, 1, 1, 1, 1, 0, 0) > 0 and size(near - 7, 1, 1, 1, 1, 1, 0, 0) == 0
    assert size(near // 2, 65, 1, 1, 1, 1, 0, 0) > 0 and size(near // 2, 65, 1, 1, 1, 1, 0, 1) == 0

    def step(B, H, V):
        return lr.scan_delta_step(*[P] * 5, 1.0, None, None, P, P, B, H, H, 1, V, 0, None, None)

    assert _status(lambda: step(1 << 24, 1, 1)) == DIM and _status(lambda: step(1 << 17, 64, 65)) == DIM


def test_adamw():
    for n in ((1 << 36) - 4095, 1 << 36, 1 << 40):
        table = (ctypes.c_int64 * 8)(P, P, 0, P, P, 0, 0, n)
        assert _status(lambda: lr.scan_adamw(ctypes.addressof(table), 1, 32, 1e-3, 0.9, 0.99, 1e-8, 0.0, 1, None, None, 0,
                                             None)) == DIM


def test_logits():
    for B, V in ((1 << 23, 32), (1 << 22, 4097), (1 << 16, 128 * 4096)):
        assert _status(lambda: lr.scan_logits(P, V, 2 * P, V, None, 0, 0, None, None, None, None, None, None, None, 0, None,
                                              8, B, V, 0, None)) == DIM


@pytest.mark.gpu
def test_the_largest_logits():
    B, V = (1 << 23) - 1, 3
    gen = torch.Generator(device="cuda").manual_seed(0)
    z = torch.randn(B, V, generator=gen, device="cuda")
    ids = torch.randint(0, V, (B, 1), generator=gen, device="cuda")
    bias = torch.randn(B, 1, generator=gen, device="cuda")
    want = z.scatter_add(1, ids, bias)
    assert torch.equal(lr.adjust_logits(z, bias_ids=ids, bias=bias, out=z), want)


@pytest.mark.gpu
def test_the_largest_step_and_the_largest_batch_of_rows():
    """States of one number: out = scale q S, S = beta k v from nothing."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    for B, T in (((1 << 24) - 1, 0), ((1 << 23) - 8, 1)):
        lead = (B, T) if T else (B,)
        q, k, v = (torch.randn(*lead, 1, 1, generator=gen, device="cuda") for _ in range(3))
        g = -torch.rand(*lead, 1, generator=gen, device="cuda")
        beta = torch.rand(*lead, 1, generator=gen, device="cuda")
        out, last = (lr.delta_scan if T else lr.delta_step)(q, k, v, g, beta, scale=0.5)
        state = beta.double().unsqueeze(-1) * k.double() * v.double()
        # a product each of beta, k, v, q and the scale, and the parts of operands: fewer than 16 u
        for got, want in ((last.view_as(state), state), (out, 0.5 * q.double() * state)):
            assert ((got.double() - want).abs() <= 16 * 2.0 ** -24 * want.abs() + 1e-30).all()
        del q, k, v, g, beta, out, last, state
