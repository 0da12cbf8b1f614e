"""The short causal convolution on the GPU against its 64-bit form (bounds
derived in _operators.py)."""
import numpy as np
import pytest

import _operators as ref
from _gpu import host, log
from test_gpu_gated import DT, close, put

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import linear_recurrence_sequence_diag_amd as lr  # noqa: E402


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lr.library()


class Case:
    def __init__(self, B, T, D, K, dtype, act="silu", reset=None, state=False, bias=True):
        r = np.random.default_rng(1000 * B + 10 * T + D + K)
        self.dtype, self.act = dtype, act
        self.x = put(r.standard_normal((B, T, D)), dtype)
        self.w = put(r.normal(0, 0.6, (K, D)), "f32")
        self.b = put(r.standard_normal(D), "f32") if bias else None
        self.g = put(r.standard_normal((B, T, D)), dtype)
        self.s = put(r.standard_normal((B, K - 1, D)), dtype) if state else None
        self.gl = put(r.standard_normal((B, K - 1, D)), dtype) if state else None
        m = {None: None, "some": r.random((B, T)) < 0.15, "all": np.ones((B, T), bool)}[reset]
        self.m = None if m is None else torch.from_numpy(m).cuda()
        self.ref = ref.Conv(host(self.x), host(self.w), None if self.b is None else host(self.b), act == "silu", m,
                            None if self.s is None else host(self.s))

    def forward(self, **kw):
        return lr.short_conv(self.x, self.w, self.b, state=self.s, reset=self.m, activation=self.act, **kw)

    def backward(self, **kw):
        return lr.short_conv_backward(self.x, self.w, self.b, self.g, state=self.s, grad_last=self.gl, reset=self.m,
                                      activation=self.act, need_grad_state=True, **kw)

    def check(self):
        out, last = self.forward()
        worst = {"out": close("out", out, (self.ref.out, self.ref.E), self.dtype)}
        assert np.array_equal(host(last), self.ref.last)
        want = self.ref.grad(host(self.g), None if self.gl is None else host(self.gl))
        for name, got in zip(("grad_x", "grad_weight", "grad_bias", "grad_state"), self.backward()):
            if got is not None:
                worst[name] = close(name, got, want[name], self.dtype if name in ("grad_x", "grad_state") else "f32")
        log(" ".join(f"{k} {v:.3f}" for k, v in worst.items()))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 2), (2, 2, 5, 4), (1, 3, 8, 4), (3, 33, 24, 3), (2, 130, 100, 4),
                                   (1, 500, 520, 4), (2, 64, 1031, 2), (65, 4, 40, 4), (1, 2100, 8, 3)])
def test_shapes(shape, dtype):
    log(f"{shape} {dtype}")
    Case(*shape, dtype).check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("T", [1, 2, 3, 31, 32, 33, 70])
@pytest.mark.parametrize("reset", [None, "some", "all"])
def test_resets_and_states(reset, T, K, dtype):
    log(f"K {K} T {T} {dtype} {reset}")
    Case(3, T, 24, K, dtype, reset=reset, state=True).check()


@pytest.mark.parametrize("act", [None, "silu"])
@pytest.mark.parametrize("bias", [True, False])
def test_activation_and_bias(bias, act):
    Case(2, 50, 36, 4, "f32", act=act, bias=bias, reset="some", state=True).check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strided_operands(dtype):
    B, T, D = 3, 70, 40
    c = Case(B, T, D, 4, dtype, reset="some", state=True)
    out, last = c.forward()
    grads = c.backward()
    wide = torch.full((T, B, 2 * D + 1), 3.0, device="cuda", dtype=DT[dtype])
    wide[..., 1:D + 1] = c.x.transpose(0, 1)
    c.x = wide[..., 1:D + 1].transpose(0, 1)
    out2, last2 = c.forward()
    assert torch.equal(out, out2) and torch.equal(last, last2)
    into = torch.full((T, B, D + 2), 5.0, device="cuda", dtype=DT[dtype])
    got = c.backward(grad_x=into[..., 1:D + 1].transpose(0, 1))
    for a, b in zip(got, grads):
        assert torch.equal(a, b)
    assert (into[..., 0] == 5.0).all() and (into[..., -1] == 5.0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_reset_stops_infinities_and_nans(dtype):
    c = Case(2, 120, 24, 4, dtype)
    m = torch.zeros(2, 120, dtype=torch.bool, device="cuda")
    m[:, [40, 65]] = True
    c.m = m
    out, last = c.forward()
    gx = c.backward()[0]
    clean = torch.ones(120, dtype=torch.bool, device="cuda")
    clean[40:65] = False
    c.x, c.g = c.x.clone(), c.g.clone()
    c.x[:, 63], c.x[:, 64] = float("inf"), float("nan")
    c.g[:, 40] = float("nan")
    out2, last2 = c.forward()
    assert torch.equal(out[:, clean], out2[:, clean]) and torch.equal(last, last2)
    assert torch.equal(gx[:, clean], c.backward()[0][:, clean])
    # and a state that a reset drops at once
    c = Case(2, 5, 24, 4, dtype, state=True)
    c.m = torch.zeros(2, 5, dtype=torch.bool, device="cuda")
    c.m[:, 0] = True
    out, _ = c.forward()
    c.s = torch.full_like(c.s, float("nan"))
    assert torch.equal(c.forward()[0], out)


def test_activation_at_its_ends():
    """Large pre-activations: y goes to z or 0, its slope to 1 or 0, none to NaN."""
    z = torch.tensor([-1e30, -300.0, -90.0, -80.0, 0.0, 80.0, 300.0, 1e30], device="cuda")
    x = z[None, :, None].expand(1, 8, 8).contiguous()
    w = torch.zeros(2, 8, device="cuda")
    w[1] = 1.0
    out, _ = lr.short_conv(x, w, activation="silu")
    want = ref.Conv(host(x), host(w), None, True)
    close("out", out, (want.out, want.E + 1e-30), "f32")
    gx, gw, _, _ = lr.short_conv_backward(x, w, None, torch.ones_like(x), activation="silu")
    assert torch.isfinite(gx).all()
    close("grad_x", gx, (want.grad(np.ones((1, 8, 8)))["grad_x"][0], 1e-6), "f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [1, 9, 64])
def test_steps_give_the_rows(D, dtype):
    c = Case(3, 20, D, 4, dtype, reset="some", state=True)
    out, last = c.forward()
    state = c.s.clone()
    for t in range(20):
        o, new = lr.short_conv_step(c.x[:, t], c.w, c.b, state, reset=c.m[:, t].contiguous(), activation="silu",
                                    out_state=state if t % 2 else None)
        assert torch.equal(o, out[:, t])
        state = new
    assert torch.equal(state, last)
    a, _ = lr.short_conv_step(c.x[:, 0], c.w, c.b, activation="silu")
    b, _ = lr.short_conv_step(c.x[:, 0], c.w, c.b, torch.zeros_like(state), activation="silu")
    assert torch.equal(a, b)


def test_autograd_workspace_and_repeatability():
    c = Case(3, 200, 96, 4, "bf16", reset="some")
    leaves = [t.detach().clone().requires_grad_() for t in (c.x, c.w, c.b)]
    out = lr.short_convolution(*leaves, reset=c.m, activation="silu")
    out.backward(c.g)
    assert torch.equal(out, c.forward()[0])
    grads = c.backward()
    for leaf, w in zip(leaves, grads):
        assert torch.equal(leaf.grad, w)
    ws = torch.zeros(lr.scan_conv_workspace_bytes(3, 200, 96, 4, lr.BF16) // 4 + 64, device="cuda")
    for a, b in zip(c.backward(workspace=ws), grads):
        assert torch.equal(a, b)
    plain = lr.short_convolution(leaves[0], leaves[1])
    plain.sum().backward()


def test_refusals():
    c = Case(2, 8, 16, 4, "f32")
    for bad in (lambda: lr.short_conv(c.x, c.w[:, :4]), lambda: lr.short_conv(c.x, c.w.bfloat16()),
                lambda: lr.short_conv(c.x, c.w, activation="relu"), lambda: lr.short_conv(c.x, c.w, c.b[:3]),
                lambda: lr.short_conv(c.x, c.w, state=torch.zeros(2, 2, 16, device="cuda")),
                lambda: lr.short_conv(c.x.transpose(1, 2), c.w),
                lambda: lr.short_conv(c.x, c.w, reset=torch.zeros(2, 9, dtype=torch.bool, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: lr.short_conv(c.x, torch.zeros(1, 16, device="cuda")),
                lambda: lr.short_conv(c.x, torch.zeros(5, 16, device="cuda")),
                lambda: lr.short_conv(c.x[:, :0], c.w),
                lambda: lr.short_conv_backward(c.x, c.w, c.b, c.g, workspace=torch.zeros(4, device="cuda"))):
        with pytest.raises(lr.LRScanError):
            bad()


def test_offsets_past_32_bits():
    B, T, D, n = 2, 150000, 8192, 40
    x = torch.zeros(B, T, D, device="cuda", dtype=torch.bfloat16)
    r = np.random.default_rng(0)
    part, gp = (put(r.standard_normal((1, n, D)), "bf16") for _ in range(2))
    x[-1, -n:] = part[0]
    w = put(r.normal(0, 0.6, (4, D)), "f32")
    g = torch.zeros_like(x)
    g[-1, -n:] = gp[0]
    out, last = lr.short_conv(x, w, activation="silu")
    c = ref.Conv(host(part), host(w), None, True)
    close("out", out[-1:, -n:], (c.out, c.E), "bf16")
    assert np.array_equal(host(last[-1:]), c.last) and not out[:, :-n].any()
    gx, gw, _, _ = lr.short_conv_backward(x, w, None, g, activation="silu")
    want = c.grad(host(gp))
    close("grad_x", gx[-1:, -n:], want["grad_x"], "bf16")
    close("grad_weight", gw, want["grad_weight"], "f32")
    assert not gx[:, :-n - 3].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("D", [132, 260, 1031])
@pytest.mark.parametrize("reset", ["some", "all"])
def test_resets_of_wide_rows(reset, D, K, dtype):
    """Rows that a wavefront walks alone, several chunks long: starts on every place of a chunk."""
    log(f"{D} {K} {dtype} {reset}")
    Case(2, 203, D, K, dtype, reset=reset, state=True).check()


# Whose reverse walks are the longest, in groups of six tokens: 14 of them, 12, 11 and 12; 14 of four with three taps.
LONG_WALKS = [(8, 4096, 2560, 4, "bf16"), (8, 2048, 4096, 4, "f32"), (42, 2938, 277, 4, "bf16"),
              (4, 32768, 289, 4, "f32"), (8, 4096, 2560, 3, "bf16")]


@pytest.mark.parametrize("shape", LONG_WALKS)
def test_resets_in_long_walks(shape):
    """Starts at every distance from a chunk's first token, against the 64-bit form on some columns."""
    B, T, D, K, dtype = shape
    log(f"{shape}")
    gen = torch.Generator(device="cuda").manual_seed(D + K)
    x, g = (torch.randn(B, T, D, generator=gen, device="cuda").to(DT[dtype]) for _ in range(2))
    w, b = torch.randn(K, D, generator=gen, device="cuda") * 0.6, torch.randn(D, generator=gen, device="cuda")
    m = torch.rand(B, T, generator=gen, device="cuda") < 0.04
    cols = np.r_[0:8, D // 2:D // 2 + 4, D - 8:D]
    c = ref.Conv(host(x[..., cols]), host(w[:, cols]), host(b[cols]), True, host(m).astype(bool))
    out, last = lr.short_conv(x, w, b, reset=m, activation="silu")
    close("out", out[..., cols], (c.out, c.E), dtype)
    assert np.array_equal(host(last[..., cols]), c.last)
    want = c.grad(host(g[..., cols]))
    gx, gw, gb, _ = lr.short_conv_backward(x, w, b, g, reset=m, activation="silu")
    close("grad_x", gx[..., cols], want["grad_x"], dtype)
    close("grad_weight", gw[:, cols], want["grad_weight"], "f32")
    close("grad_bias", gb[cols], want["grad_bias"], "f32")
    # an infinity and a NaN stay in their segment: of the other tokens every bit stays
    t = torch.arange(T, device="cuda")
    m[:, (t % 97 == 5) | (t % 97 == 70)] = True
    gx = lr.short_conv_backward(x, w, b, g, reset=m, activation="silu")[0]
    bad = (t % 97 >= 5) & (t % 97 < 70)
    x[:, t % 97 == 68], x[:, t % 97 == 69], g[:, t % 97 == 5] = float("inf"), float("nan"), float("nan")
    gx2 = lr.short_conv_backward(x, w, b, g, reset=m, activation="silu")[0]
    assert torch.equal(gx[:, ~bad], gx2[:, ~bad])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [24, 260])
@pytest.mark.parametrize("K", [2, 3, 4])
def test_no_token_past_the_last_takes_part(K, D, dtype):
    """The last input belongs to the last tap's gradient alone, an early tap to no gradient of the last token: an
    infinity in one leaves the others as they are, bit for bit."""
    for T in (50, 64, 203):
        c = Case(2, T, D, K, dtype, act=None)
        grads = c.backward()
        c.x = c.x.clone()
        c.x[:, -1] = float("inf")
        got = c.backward()
        assert torch.equal(got[0], grads[0]) and torch.equal(got[2], grads[2])
        assert torch.equal(got[1][:-1], grads[1][:-1]) and not torch.isfinite(got[1][-1]).any()
        c.w = c.w.clone()
        c.w[0] = float("inf")
        assert torch.equal(c.backward()[0][:, T - K + 1:], grads[0][:, T - K + 1:])
