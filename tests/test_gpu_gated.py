"""The gated scan on the GPU against its 64-bit form (bounds derived in
_operators.py, and not taken from what the kernels give): ragged and unaligned
shapes, gates as halves of a projection, resets, states, special values, one
step at a time, and the same bits from every call."""
import numpy as np
import pytest

import _operators as ref
from _gpu import host, log

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import linear_recurrence_sequence_diag_amd as lr  # noqa: E402

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lr.library()


def close(name, got, pair, dtype):
    val, bound = pair
    tol = ref.store(bound, val, dtype)
    err = np.abs(host(got) - val)
    worst = float(np.max(err / tol)) if err.size else 0.0
    assert np.all(err <= tol), f"{name}: {np.sum(~(err <= tol))} of {err.size} outside their bounds, worst {worst}"
    return worst


def put(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda().to(DT[dtype])


class Case:
    def __init__(self, B, T, D, dtype, reset=None, states=False, proj=False, seed=0, gate_sd=1.5):
        r = np.random.default_rng(seed + 1000 * B + 10 * T + D)
        self.dtype, self.proj = dtype, proj
        self.x = put(r.standard_normal((B, T, D)), dtype)
        both = put(r.normal(0, gate_sd, (B, T, 2 * D)), dtype)
        self.gr, self.gi = both[..., :D], both[..., D:]
        if not proj:
            self.gr, self.gi = self.gr.contiguous(), self.gi.contiguous()
        # the slowest decay of a channel between 0.9 and 0.999, as such layers start with
        a = r.uniform(0.9, 0.999, D)
        self.decay = put(np.log(np.expm1(-np.log(a) / 8.0)), "f32")
        self.g = put(r.standard_normal((B, T, D)), dtype)
        self.h0 = put(r.standard_normal((B, D)), "f32") if states else None
        self.gl = put(r.standard_normal((B, D)), "f32") if states else None
        m = {None: None, "some": r.random((B, T)) < 0.05, "all": np.ones((B, T), bool),
             "first": np.arange(T)[None].repeat(B, 0) == 0}[reset]
        self.m = None if m is None else torch.from_numpy(m).cuda()
        self.ref = ref.Gated(host(self.x), host(self.gr), host(self.gi), host(self.decay), 8.0, m,
                             None if self.h0 is None else host(self.h0))

    def forward(self, **kw):
        return lr.gated_scan(self.x, self.gr, self.gi, self.decay, h0=self.h0, reset=self.m, **kw)

    def backward(self, out, **kw):
        return lr.gated_scan_backward(self.x, self.gr, self.gi, self.decay, out, self.g, grad_last=self.gl,
                                      h0=self.h0, reset=self.m, need_grad_h0=True, **kw)

    def check(self, **kw):
        out, last = self.forward(**kw)
        worst = {"out": close("out", out, (self.ref.h, self.ref.E), self.dtype),
                 "last": close("last", last, (self.ref.h[:, -1], self.ref.E[:, -1]), "f32")}
        want = self.ref.grad(host(out), host(self.g), None if self.gl is None else host(self.gl))
        for name, got in zip(("grad_x", "grad_r", "grad_i", "grad_decay", "grad_h0"), self.backward(out, **kw)):
            worst[name] = close(name, got, want[name], "f32" if name in ("grad_decay", "grad_h0") else self.dtype)
        log(" ".join(f"{k} {v:.3f}" for k, v in worst.items()))
        # the state-only forward gives the same last state
        none, last2 = self.forward(with_out=False, **kw)
        assert none is None and torch.equal(last, last2)
        return out, last


ALGOS = ["auto", "seq", "fused"]
SHAPES = [(1, 1, 1), (2, 3, 5), (3, 17, 8), (2, 64, 64), (1, 65, 131), (2, 257, 130), (1, 300, 72), (5, 129, 520),
          (2, 700, 33), (3, 513, 256), (70, 5, 100), (1, 2100, 24),
          (64, 130, 256), (700, 700, 5)]  # wide tiles over many chains; tall tiles, many of them


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_shapes(shape, dtype, algo):
    log(f"{shape} {dtype} {algo}")
    Case(*shape, dtype).check(algo=algo)


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(2, 40, 16), (2, 300, 72), (3, 1100, 9), (4, 6, 40)])
@pytest.mark.parametrize("reset", [None, "some", "all", "first"])
def test_resets_states_and_projected_gates(reset, shape, dtype, algo):
    log(f"{shape} {dtype} {algo} {reset}")
    Case(*shape, dtype, reset=reset, states=True, proj=True).check(algo=algo)


@pytest.mark.parametrize("reset", [None, "some"])
@pytest.mark.parametrize("algo", ["seq", "fused"])
@pytest.mark.parametrize("shape", [(1051, 7, 1999), (1051, 32, 500)])
def test_the_last_states_gradient_may_cancel_the_last_rows(shape, algo, reset):
    """Among this many channels some where both, and the sum of the row before, are nearly nothing."""
    log(f"{shape} {algo} {reset}")
    Case(*shape, "f32", reset=reset, states=True).check(algo=algo)


@pytest.mark.parametrize("algo", ["auto", "seq"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(2101, 3, 1000), (2101, 2, 1001), (4203, 4, 500), (1051, 7, 1999)])
def test_short_sequences_that_share_a_channels_rate(shape, dtype, algo):
    """Several batch rows to a thread, the last thread's fewer; states and resets of each row its own."""
    log(f"{shape} {dtype} {algo}")
    Case(*shape, dtype, reset="some", states=True).check(algo=algo)


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strided_operands(dtype, algo):
    """Rows apart from each other, time before batch, broadcast rows, an odd base."""
    B, T, D = 3, 150, 40
    c = Case(B, T, D, dtype, reset="some", states=True)
    want, last = c.forward(algo=algo)
    grads = c.backward(want, algo=algo)
    wide = torch.full((T, B, 3 * D + 1), 7.0, device="cuda", dtype=DT[dtype])
    for k, t in enumerate((c.x, c.gr, c.gi)):
        wide[..., k * D + 1:(k + 1) * D + 1] = t.transpose(0, 1)
    c.x, c.gr, c.gi = (wide[..., k * D + 1:(k + 1) * D + 1].transpose(0, 1) for k in range(3))
    out, last2 = c.forward(algo=algo)
    assert torch.equal(out, want) and torch.equal(last, last2)
    into = torch.full((T, B, 3 * D + 2), 5.0, device="cuda", dtype=DT[dtype])
    views = [into[..., k * D + 1:(k + 1) * D + 1].transpose(0, 1) for k in range(3)]
    got = c.backward(out, algo=algo, grads=views)
    for a, b in zip(got, grads):
        assert torch.equal(a, b)
    assert (into[..., 0] == 5.0).all() and (into[..., -1] == 5.0).all()  # nothing written beside them
    one = torch.randn(1, T, D, device="cuda").to(DT[dtype])
    c.gr = one.expand(B, T, D)
    a, _ = c.forward(algo=algo)
    c.gr = c.gr.contiguous()
    b, _ = c.forward(algo=algo)
    assert torch.equal(a, b)


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_reset_stops_infinities_and_nans(bad, dtype, algo):
    """A segment that holds them leaves the other segments' results as they are, bit for bit."""
    B, T, D = 2, 700, 72
    c = Case(B, T, D, dtype)
    m = torch.zeros(B, T, dtype=torch.bool, device="cuda")
    m[:, [0, 210, 395, 640]] = True
    c.m = m
    out, last = c.forward(algo=algo)
    grads = c.backward(out, algo=algo)
    clean = torch.ones(T, dtype=torch.bool, device="cuda")
    clean[210:395] = False
    c.x = c.x.clone()
    c.x[:, 300] = bad
    c.gi = c.gi.clone()
    c.gi[0, 377, :5] = float("nan")
    out2, last2 = c.forward(algo=algo)
    assert not torch.isfinite(out2[:, 394]).any()
    assert torch.equal(out[:, clean], out2[:, clean]) and torch.equal(last, last2)
    c.g = c.g.clone()
    c.g[:, 350] = bad
    grads2 = c.backward(out2, algo=algo)
    for a, b in zip(grads[:3], grads2[:3]):
        assert torch.equal(a[:, clean], b[:, clean])
    assert torch.equal(grads[4], grads2[4])


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_extreme_gates_and_decays(dtype, algo):
    """Gates at the ends of the sigmoid and decays at the ends of softplus: the
    limits of the formula, with finite gradients."""
    B, T, D = 2, 90, 16
    c = Case(B, T, D, dtype)
    inf = float("inf")
    c.gr = c.gr.clone()
    c.gi = c.gi.clone()
    c.gr[:, :, 0], c.gr[:, :, 1], c.gr[:, :, 2], c.gr[:, :, 3] = 200.0, -200.0, inf, -inf
    c.gi[:, :, 4], c.gi[:, :, 5], c.gi[:, :, 6], c.gi[:, :, 7] = 200.0, -200.0, inf, -inf
    c.gr[:, :, 8], c.gi[:, :, 9] = -88.5, -88.5
    c.decay = c.decay.clone()
    c.decay[10], c.decay[11], c.decay[12], c.decay[13] = -120.0, 60.0, -inf, -17.0
    c.ref = ref.Gated(host(c.x), np.clip(host(c.gr), -500, 500), np.clip(host(c.gi), -500, 500),
                      np.clip(host(c.decay), -500, 500), 8.0)
    out, last = c.forward(algo=algo)
    close("out", out, (c.ref.h, c.ref.E + 1e-18), dtype)
    want = c.ref.grad(host(out), host(c.g))
    for name, got in zip(("grad_x", "grad_r", "grad_i", "grad_decay"), c.backward(out, algo=algo)):
        val, bound = want[name]
        assert torch.isfinite(got).all(), name
        # where 1 - a^2 is below 2^-126 the kernels take its limit: beta up to 1e-19, of sums of 90 terms
        close(name, got, (val, bound + 1e-16), "f32" if name == "grad_decay" else dtype)


def test_a_nan_gate_is_not_hidden():
    c = Case(1, 20, 8, "f32")
    for gate in ("gr", "gi"):
        t = getattr(c, gate).clone()
        keep = getattr(c, gate)
        t[0, 4, 3] = float("nan")
        setattr(c, gate, t)
        for algo in ALGOS:
            out, last = c.forward(algo=algo)
            assert torch.isnan(out[0, 4:, 3]).all() and torch.isnan(last[0, 3])
            assert torch.isfinite(out[0, :4]).all() and torch.isfinite(out[0, :, :3]).all()
            g = c.backward(out, algo=algo)
            assert torch.isnan(g[0][0, 4, 3]) and torch.isnan(g[1 if gate == "gr" else 2][0, 4, 3])
        setattr(c, gate, keep)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [1, 9, 64, 100])
def test_steps_give_the_rows(D, dtype):
    """Chained steps, in place and not, are the per-lane walk bit for bit."""
    B, T = 5, 12
    c = Case(B, T, D, dtype, reset="some", states=True, proj=True)
    out, last = c.forward(algo="seq")
    state = c.h0.clone()
    for t in range(T):
        o, new = lr.gated_step(c.x[:, t], c.gr[:, t], c.gi[:, t], c.decay, state, reset=c.m[:, t].contiguous(),
                               out_state=state if t % 2 else None)
        assert torch.equal(o, out[:, t])
        assert (new.data_ptr() == state.data_ptr()) == bool(t % 2)
        state = new
    assert torch.equal(state, last)
    a, _ = lr.gated_step(c.x[:, 0], c.gr[:, 0], c.gi[:, 0], c.decay)  # from a zero state
    b, _ = lr.gated_step(c.x[:, 0], c.gr[:, 0], c.gi[:, 0], c.decay, torch.zeros_like(state))
    assert torch.equal(a, b)
    none, s = lr.gated_step(c.x[:, 0], c.gr[:, 0], c.gi[:, 0], c.decay, with_out=False)
    assert none is None and s.shape == (B, D)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("reset", [None, "some"])
def test_tiles_that_do_not_wait(reset, dtype):
    """With one poll a tile derives the maps it misses: the same bits."""
    for B, T, D in ((1, 3000, 40), (2, 1500, 257), (1, 20000, 64)):
        log(f"{B} {T} {D}")
        c = Case(B, T, D, dtype, reset=reset, states=True) if T < 5000 else Case(B, T, D, dtype, reset=reset)
        out, last = c.forward(algo="fused")
        grads = c.backward(out, algo="fused")
        for _ in range(2):
            out1, last1 = c.forward(algo="fused", polls=1)
            assert torch.equal(out, out1) and torch.equal(last, last1)
            for a, b in zip(grads, c.backward(out, algo="fused", polls=1)):
                assert a is b or torch.equal(a, b)


def test_autograd_and_repeatability():
    c = Case(3, 400, 96, "bf16", reset="some", proj=True)
    leaves = [t.detach().clone().requires_grad_() for t in (c.x, c.gr, c.gi, c.decay)]
    both = torch.cat([leaves[1], leaves[2]], -1)
    gr, gi = both.chunk(2, -1)
    out = lr.gated_diagonal_scan(leaves[0], gr, gi, leaves[3], reset=c.m)
    out.backward(c.g)
    want, _ = c.forward()
    assert torch.equal(out, want)
    for leaf, w in zip(leaves, c.backward(want)):
        assert torch.equal(leaf.grad, w)
    again = c.backward(want)
    for a, b in zip(c.backward(want), again):
        assert torch.equal(a, b)


def test_a_second_derivative_is_refused():
    """Of each differentiable operator: an error, and no gradient without its graph."""
    x = torch.randn(2, 5, 8, device="cuda", requires_grad=True)
    ones = torch.ones(8, device="cuda")
    table = torch.randn(4, 8, device="cuda", requires_grad=True)
    ids = torch.tensor([0, 3, 3], device="cuda")
    for leaf, out in ((x, lr.gated_diagonal_scan(x, x, x, ones)),
                      (x, lr.short_convolution(x, torch.ones(4, 8, device="cuda"), activation="silu")),
                      (table, lr.embedding(ids, table))):
        g, = torch.autograd.grad((out * out).sum(), leaf, create_graph=True)
        with pytest.raises(RuntimeError):
            g.sum().backward()


def test_workspace_streams_and_capture():
    """A caller's workspace gives the library's results; so does a captured call,
    replayed between eager calls; and a call on another stream after its inputs."""
    c = Case(2, 600, 128, "bf16", reset="some", states=True)
    out, last = c.forward()
    grads = c.backward(out)
    ws = torch.zeros(lr.scan_gated_workspace_bytes(2, 600, 128, lr.BF16) // 4 + 64, device="cuda")
    assert torch.equal(c.forward(workspace=ws)[0], out)
    for a, b in zip(c.backward(out, workspace=ws), grads):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o2, _ = c.forward()
        for a, b in zip(c.backward(o2), grads):
            assert torch.equal(a, b)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            o3, l3 = c.forward()
            g3 = c.backward(o3)
    for k in range(3):
        o3.zero_()
        for t in g3:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o3, out) and torch.equal(l3, last)
        for a, b in zip(g3, grads):
            assert torch.equal(a, b)
        with torch.cuda.stream(side):
            c.forward()
        torch.cuda.synchronize()


def test_refusals():
    c = Case(2, 8, 16, "f32")
    with pytest.raises(ValueError):
        lr.gated_scan(c.x, c.gr[:, :4], c.gi, c.decay)
    with pytest.raises(ValueError):
        lr.gated_scan(c.x, c.gr.bfloat16(), c.gi, c.decay)
    with pytest.raises(ValueError):
        lr.gated_scan(c.x.transpose(1, 2), c.gr, c.gi, c.decay)
    with pytest.raises(ValueError):
        lr.gated_scan(c.x, c.gr, c.gi, c.decay[:4])
    with pytest.raises(ValueError):
        lr.gated_scan(c.x, c.gr, c.gi, c.decay, reset=torch.zeros(2, 7, dtype=torch.bool, device="cuda"))
    with pytest.raises(ValueError):
        lr.gated_scan(c.x, c.gr, c.gi, c.decay, h0=torch.zeros(2, 8, device="cuda"))
    with pytest.raises(ValueError):
        lr.gated_scan(c.x, c.gr, c.gi, c.decay, with_last=False, with_out=False)
    with pytest.raises(TypeError):
        lr.gated_scan(c.x.half(), c.gr.half(), c.gi.half(), c.decay)
    with pytest.raises(lr.LRScanError):
        lr.gated_scan(c.x, c.gr, c.gi, c.decay, scale=-1.0)
    with pytest.raises(lr.LRScanError):
        lr.gated_scan(c.x[:, :0], c.gr[:, :0], c.gi[:, :0], c.decay)
    with pytest.raises(lr.LRScanError):
        lr.gated_scan_backward(c.x, c.gr, c.gi, c.decay, c.x, c.g,
                               workspace=torch.zeros(4, device="cuda"))


def test_offsets_past_32_bits():
    """Tensors of more than 2^32 bytes: the last segment of the last row, which
    stands for itself, against the reference."""
    B, T, D, n = 2, 150000, 8192, 200
    bf = torch.bfloat16
    x = torch.zeros(B, T, D, device="cuda", dtype=bf)
    gr, gi = torch.zeros_like(x), torch.zeros_like(x)
    r = np.random.default_rng(0)
    small = [put(r.standard_normal((1, n, D)), "bf16") for _ in range(4)]
    for t, v in zip((x, gr, gi), small):
        t[-1, -n:] = v[0]
    decay = put(r.normal(-4, 0.5, D), "f32")
    m = torch.zeros(B, T, dtype=torch.bool, device="cuda")
    m[-1, -n] = True
    out, last = lr.gated_scan(x, gr, gi, decay, reset=m)
    cols = np.r_[0:16, D - 16:D]
    f = ref.Gated(*(host(t[..., cols]) for t in small[:3]), host(decay[cols]), 8.0, np.arange(n)[None] == 0)
    close("out", out[-1:, -n:, cols], (f.h, f.E), "bf16")
    close("last", last[-1:, cols], (f.h[:, -1], f.E[:, -1]), "f32")
    g = torch.zeros_like(x)
    g[-1, -n:] = small[3][0]
    grads = lr.gated_scan_backward(x, gr, gi, decay, out, g, reset=m)
    want = f.grad(host(out[-1:, -n:, cols]), host(small[3][..., cols]))
    for name, got in zip(("grad_x", "grad_r", "grad_i"), grads):
        close(name, got[-1:, -n:, cols], want[name], "bf16")
        assert not got[0].any() and not got[1, :-n - 1].any()
    close("grad_decay", grads[3][cols], want["grad_decay"], "f32")


def test_a_mask_changed_before_the_backward_is_refused():
    """As any operand changed in place is: an error, and no gradient of another mask's segments."""
    x = torch.randn(2, 9, 8, device="cuda", requires_grad=True)
    ones = torch.ones(8, device="cuda")
    for call in (lambda m: lr.gated_diagonal_scan(x, x, x, ones, reset=m),
                 lambda m: lr.short_convolution(x, torch.ones(4, 8, device="cuda"), reset=m)):
        m = torch.zeros(2, 9, dtype=torch.bool, device="cuda")
        m[:, 4] = True
        torch.autograd.grad(call(m).sum(), x)
        out = call(m).sum()
        m[:, 4] = False
        with pytest.raises(RuntimeError):
            torch.autograd.grad(out, x)
