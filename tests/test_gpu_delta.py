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
    (1, 1700, 2, 1, 64, 32, "some", True),  # from here on walked in parts
    (2, 2000, 1, 1, 130, 20, None, False),
    (1, 4200, 3, 3, 48, 36, "some", False),
    (1, 2600, 2, 2, 200, 17, "edges", True),
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


@pytest.mark.parametrize("shape", [(2, 200, 4, 2, 128, 128, "some", True), (1, 1700, 2, 1, 64, 40, "some", True),
                                   (1, 70, 3, 1, 33, 7, None, False)], ids=str)
def test_outputs_alone_and_the_state_alone(shape):
    """Without the last state a bf16 forward takes fewer parts of its operands; the state alone is the whole call's."""
    B, T, H, HK, K, V, kind, state = shape
    x, reset, h0, _ = _case(B, T, H, HK, K, V, "bf16", kind, state, seed=2)
    ref, f32 = _refs(x, reset, h0, None, 0.25, False)
    args = [x[n].cuda() for n in NAMES]
    more = dict(scale=0.25, h0=None if h0 is None else x["h0"].cuda(), reset=None if reset is None else reset.cuda())
    out, none = lr.delta_scan(*args, **more, with_last=False)
    assert none is None
    # an operand of two parts is off by 2^-18: below a hundredth of the bound's half step of bf16
    D.check("out", out, ref["out"], f32["out"], torch.bfloat16)
    none, last = lr.delta_scan(*args, **more, with_out=False)
    assert none is None and torch.equal(last, lr.delta_scan(*args, **more)[1])


def test_calls_repeat_bit_for_bit():
    x, reset, _, _ = _case(2, 1700, 4, 2, 64, 48, "bf16", "some", seed=3)
    args = [x[n].cuda() for n in NAMES]
    go, r = x["grad_out"].cuda(), reset.cuda()
    first = lr.delta_scan(*args, reset=r) + lr.delta_scan_backward(*args, go, reset=r)[:5]
    for _ in range(3):
        again = lr.delta_scan(*args, reset=r) + lr.delta_scan_backward(*args, go, reset=r)[:5]
        assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("K,V", [(64, 64), (50, 30)])
def test_strided_operands(K, V, dt):
    """Parts of one projection, steps before batch rows, broadcast gates, one head for all."""
    B, T, H, HK = 3, 100, 4, 2
    x = D.inputs(B, T, H, HK, K, V, DT[dt], 4)
    plain = [x[n].cuda() for n in NAMES]
    go = x["grad_out"].cuda()
    whole = torch.cat([plain[i].flatten(2) for i in range(3)], -1)
    q, k, v = (t.unflatten(-1, (n, -1)) for t, n in zip(whole.split([HK * K, HK * K, H * V], -1), (HK, HK, H)))
    turned = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in plain]
    want = lr.delta_scan(*plain) + lr.delta_scan_backward(*plain, go)[:5]
    for args in ((q, k, v, *plain[3:]), turned):
        assert not args[0].is_contiguous()
        got = lr.delta_scan(*args) + lr.delta_scan_backward(*args, go)[:5]
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    g = plain[3][:, :1, :1].expand(B, T, H)
    one = plain[1][:, :, :1].expand(B, T, HK, K)
    got = lr.delta_scan(plain[0], one, plain[2], g, plain[4])
    want = lr.delta_scan(plain[0], one.contiguous(), plain[2], g.contiguous(), plain[4])
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_operands_at_odd_addresses():
    B, T, H, K, V = 1, 90, 2, 64, 64
    x = D.inputs(B, T, H, H, K, V, torch.bfloat16, 5)
    plain = [x[n].cuda() for n in NAMES]
    go = x["grad_out"].cuda()

    def odd(t):
        flat = torch.zeros(t.numel() + 1, dtype=t.dtype, device="cuda")
        flat[1:] = t.flatten()
        return flat[1:].view(t.shape)

    want = lr.delta_scan(*plain) + lr.delta_scan_backward(*plain, go)[:5]
    moved = [odd(t) for t in plain]
    got = lr.delta_scan(*moved) + lr.delta_scan_backward(*moved, odd(go))[:5]
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("T", [150, 1700])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_segments_do_not_reach_each_other(dt, T):
    """Infinities and NaN in one document leave the others' outputs and gradients as they are."""
    x, _, _, _ = _case(1, T, 2, 1, 64, 32, dt, seed=6)
    cuts = [0, 5, 64, 100, 130]
    reset = torch.zeros(1, T, dtype=torch.bool)
    reset[:, cuts] = True
    args = [x[n].cuda() for n in NAMES]
    go, r = x["grad_out"].cuda(), reset.cuda()
    want = lr.delta_scan(*args, reset=r)[:1] + lr.delta_scan_backward(*args, go, reset=r)[:5]
    for lo, hi in zip(cuts, cuts[1:]):
        bad = [t.clone() for t in args]
        bad[0][:, lo] = float("nan")
        bad[1][:, lo:hi] = float("inf")
        bad[2][:, hi - 1] = float("-inf")
        bad[3][:, lo] = float("nan")
        bad[4][:, hi - 1] = float("nan")
        g = go.clone()
        g[:, lo] = float("nan")
        got = lr.delta_scan(*bad, reset=r)[:1] + lr.delta_scan_backward(*bad, g, reset=r)[:5]
        for a, b in zip(want, got):
            assert torch.equal(a[:, :lo], b[:, :lo]) and torch.equal(a[:, hi:], b[:, hi:])
    # nor does a state that is not finite pass a reset
    h0 = torch.full((1, 2, 64, 32), float("nan"), device="cuda")
    assert torch.equal(lr.delta_scan(*args, reset=r, h0=h0)[0], want[0])
    assert not torch.isfinite(lr.delta_scan(*args, h0=h0)[0]).any()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_segments_that_end_in_any_part_do_not_reach_the_next(dt):
    """A long row is walked in parts; segments with infinities and NaN end in, before and behind parts' ends."""
    T = 2100
    x, _, _, _ = _case(1, T, 2, 1, 64, 32, dt, seed=6)
    cuts = list(range(0, 1000, 37)) + [1024, 1200, 1408, 1500, 1900]
    reset = torch.zeros(1, T, dtype=torch.bool)
    reset[:, cuts] = True
    args = [x[n].cuda() for n in NAMES]
    go, r = x["grad_out"].cuda(), reset.cuda()
    want = lr.delta_scan(*args, reset=r)[:1] + lr.delta_scan_backward(*args, go, reset=r)[:5]
    for odd in (0, 1):  # every other segment, the last ones among them
        bad, g = [t.clone() for t in args], go.clone()
        fine = torch.ones(T, dtype=torch.bool)
        for lo, hi in list(zip(cuts, cuts[1:] + [T]))[odd::2]:
            bad[1][:, lo:hi] = float("inf")
            bad[2][:, hi - 1] = float("nan")
            g[:, lo] = float("nan")
            fine[lo:hi] = False
        got = lr.delta_scan(*bad, reset=r)[:1] + lr.delta_scan_backward(*bad, g, reset=r)[:5]
        for a, b in zip(want, got):
            assert torch.equal(a[:, fine], b[:, fine])


def test_gates_at_their_ends():
    """Decays of 0 and 1, of the type's lowest value and minus infinity, strengths of 0 and 1, against the walk."""
    x, _, _, _ = _case(2, 200, 2, 2, 32, 16, "f32", seed=7)
    gen = torch.Generator().manual_seed(8)
    for value in (0.0, -300.0, -60.0, torch.finfo(torch.float32).min, float("-inf")):
        x["log_decay"][torch.rand(x["log_decay"].shape, generator=gen) < 0.1] = value
    for value in (0.0, 1.0):
        x["beta"][torch.rand(x["beta"].shape, generator=gen) < 0.2] = value
    x["beta"][0, 64:128] = 0.0
    x["k"][1, 100:110] = 0.0
    _run(x, None, x["h0"], x["grad_last"], 0.25, True, "f32")


def test_far_decays_keep_the_near_ones():
    """Strong forgetting early in a block does not blur the mild decays behind it."""
    x, _, _, _ = _case(1, 64, 1, 1, 32, 16, "f32", seed=9)
    x["log_decay"][:] = -1e-3
    x["log_decay"][:, :20] = -190.0
    _run(x, None, None, None, 0.25, True, "f32")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,HK,K,V", [(3, 4, 2, 64, 64), (2, 3, 1, 33, 101), (1, 8, 8, 128, 256), (33, 1, 1, 256, 20)])
def test_steps_are_the_scan(B, H, HK, K, V, dt):
    T = 6
    x, reset, h0, _ = _case(B, T, H, HK, K, V, dt, "some", True, seed=10)
    reset = torch.rand(B, T, generator=torch.Generator().manual_seed(11)) < 0.3
    dev = {n: t.cuda() for n, t in x.items()}
    ref, f32 = _refs(x, reset, h0, None, 0.5, False)
    state = dev["h0"].clone()
    for t in range(T):
        args = [dev[n][:, t] for n in NAMES]
        out, new = lr.delta_step(*args, state, scale=0.5, reset=reset[:, t].contiguous().cuda(), out_state=state)
        assert new is state
        D.check("out", out, ref["out"][:, t], f32["out"][:, t], DT[dt])
    D.check("last", state, ref["last"], f32["last"], DT[dt])
    # from nothing, and without an output
    none, first = lr.delta_step(*[dev[n][:, 0] for n in NAMES], with_out=False)
    want = lr.delta_step(*[dev[n][:, 0] for n in NAMES], torch.zeros_like(state))[1]
    assert none is None and torch.allclose(first, want, rtol=1e-6, atol=1e-7)


def test_a_step_drops_a_state_that_is_not_finite():
    x, _, _, _ = _case(2, 1, 2, 1, 32, 16, "f32", seed=12)
    args = [x[n][:, 0].cuda() for n in NAMES]
    args[3][0] = float("nan")
    bad = torch.full((2, 2, 32, 16), float("inf"), device="cuda")
    out, new = lr.delta_step(*args, bad, reset=torch.tensor([True, True], device="cuda"))
    want_out, want = lr.delta_step(*args)
    assert torch.equal(out, want_out) and torch.equal(new, want) and torch.isfinite(new).all()


@pytest.mark.parametrize("T", [130, 1700])
def test_autograd(T):
    x, reset, _, _ = _case(1, T, 4, 2, 64, 32, "f32", "some", seed=13)
    leaves = [x[n].cuda().requires_grad_() for n in NAMES]
    go, r = x["grad_out"].cuda(), reset.cuda()
    y = lr.gated_delta_rule(*leaves, scale=0.3, reset=r)
    got = torch.autograd.grad(y, leaves, go)
    plain = [t.detach() for t in leaves]
    want = lr.delta_scan_backward(*plain, go, scale=0.3, reset=r)[:5]
    assert torch.equal(y, lr.delta_scan(*plain, scale=0.3, reset=r, with_last=False)[0])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    z = lr.gated_delta_rule(*leaves, reset=r)
    r.logical_not_()
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        z.sum().backward()
    r.logical_not_()
    z = lr.gated_delta_rule(*leaves)
    with pytest.raises(RuntimeError):
        (gq,) = torch.autograd.grad(z.sum(), leaves[:1], create_graph=True)
        gq.sum().backward()


@pytest.mark.parametrize("T", [130, 1700])
def test_captured_calls_replay(T):
    """Forward and backward in a graph on a stream of their own, new inputs before each replay."""
    x, reset, _, _ = _case(2, T, 2, 1, 64, 40, "bf16", "some", seed=14)
    args = [x[n].cuda() for n in NAMES]
    go, r = x["grad_out"].cuda(), reset.cuda()
    bytes_ = lr.scan_delta_workspace_bytes(2, T, 2, 1, 64, 40, 1, True)
    ws = torch.empty(bytes_, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        kept = lr.delta_scan(*args, reset=r, workspace=ws)
        kept += lr.delta_scan_backward(*args, go, reset=r, workspace=ws)[:5]
    for seed in range(4):
        y = D.inputs(2, T, 2, 1, 64, 40, torch.bfloat16, 20 + seed)
        for a, n in zip(args, NAMES):
            a.copy_(y[n])
        go.copy_(y["grad_out"])
        r.copy_(_reset(2, T, "some", seed))
        graph.replay()
        want = lr.delta_scan(*args, reset=r) + lr.delta_scan_backward(*args, go, reset=r)[:5]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, want)), seed


def test_a_capture_without_a_workspace_is_refused():
    from test_gpu_graphs_streams import fresh_stream
    x, _, _, _ = _case(1, 70, 1, 1, 32, 16, "f32", seed=15)
    args = [x[n].cuda() for n in NAMES]
    side = fresh_stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        with pytest.raises(lr.LRScanError) as e:
            lr.delta_scan(*args)
        assert e.value.status == -8
        step = lr.delta_step(*[t[:, 0] for t in args])  # needs none
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(step[1], lr.delta_step(*[t[:, 0] for t in args])[1])


def test_two_streams_at_once():
    cases = [_case(2, 600, 4, 2, 64, 64, "bf16", "some", seed=16 + i) for i in range(2)]
    args = [[x[n].cuda() for n in NAMES] for x, *_ in cases]
    go = [x["grad_out"].cuda() for x, *_ in cases]
    want = [lr.delta_scan_backward(*a, g)[:5] for a, g in zip(args, go)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = lr.delta_scan_backward(*args[i], go[i])[:5]
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_workspaces_hold_what_the_call_says():
    """A buffer of exactly the size, with bytes behind it that stay."""
    for B, T, H, HK, K, V in ((2, 100, 4, 2, 33, 20), (1, 1700, 2, 1, 64, 40)):
        for dt, code in (("f32", 0), ("bf16", 1)):
            x, reset, _, _ = _case(B, T, H, HK, K, V, dt, "some", seed=18)
            args = [x[n].cuda() for n in NAMES]
            go, r = x["grad_out"].cuda(), reset.cuda()
            for back in (False, True):
                n = lr.scan_delta_workspace_bytes(B, T, H, HK, K, V, code, back)
                buf = torch.full((n + 4096,), 77, dtype=torch.uint8, device="cuda")
                call = (lambda **w: lr.delta_scan_backward(*args, go, reset=r, **w)[:5]) if back else (
                    lambda **w: lr.delta_scan(*args, reset=r, **w))
                got = call(workspace=buf[:n])
                assert (buf[n:] == 77).all()
                assert all(torch.equal(a, b) for a, b in zip(got, call()))


def test_outputs_end_where_they_end():
    """Rows of a ragged call, written into the middle of a buffer through the C ABI, leave the rest as it was."""
    B, T, H, HK, K, V = 2, 77, 3, 1, 70, 37
    x, reset, h0, _ = _case(B, T, H, HK, K, V, "bf16", "some", True, seed=19)
    d = {n: t.cuda() for n, t in x.items()}
    r = reset.cuda()
    want = lr.delta_scan(*[d[n] for n in NAMES], reset=r) + lr.delta_scan_backward(*[d[n] for n in NAMES], d["grad_out"],
                                                                                reset=r)[:5]
    kinds = [(t.shape, t.dtype) for t in want]
    bufs = [torch.full((t.numel() + 512,), 7.0, dtype=t.dtype, device="cuda") for t in want]
    views = [b[256:256 + t.numel()].view(t.shape) for b, t in zip(bufs, want)]
    p = [d[n].data_ptr() for n in NAMES]
    s = torch.cuda.current_stream().cuda_stream
    opts = lr.make_opts(reset=r)
    lr.scan_delta_fwd(*p, K ** -0.5, views[0].data_ptr(), views[1].data_ptr(), B, T, H, HK, K, V, 1, None, s, opts)
    lr.scan_delta_bwd(*p, K ** -0.5, d["grad_out"].data_ptr(), None, *[v.data_ptr() for v in views[2:]], B, T, H, HK, K, V,
                      1, None, s, opts)
    torch.cuda.synchronize()
    for b, v, t in zip(bufs, views, want):
        assert torch.equal(v, t) and (b[:256] == 7).all() and (b[256 + t.numel():] == 7).all(), kinds


def test_refusals():
    x = D.inputs(2, 5, 4, 2, 16, 8, torch.float32, 0)
    d = {n: t.cuda() for n, t in x.items()}
    args = [d[n] for n in NAMES]

    def call(**more):
        a = {**d, **more}
        return lr.delta_scan(*[a[n] for n in NAMES], **{k: v for k, v in more.items() if k not in NAMES})

    bad = [dict(q=d["q"][..., :8]), dict(k=d["k"].bfloat16()), dict(v=d["v"][:, :4]), dict(v=d["v"][:, :, :3]),
           dict(log_decay=d["log_decay"].double()), dict(beta=d["beta"][:, :, :2]), dict(beta=d["beta"].cpu()),
           dict(k=d["k"].transpose(2, 3)), dict(h0=d["h0"].bfloat16()), dict(h0=d["h0"][:, :2]),
           dict(h0=d["h0"].transpose(2, 3)), dict(reset=torch.zeros(2, 4, dtype=torch.bool, device="cuda")),
           dict(reset=torch.zeros(2, 5, device="cuda")), dict(q=d["q"][0])]
    for more in bad:
        with pytest.raises((ValueError, TypeError)):
            call(**more)
    with pytest.raises(ValueError):
        lr.delta_scan(*args, with_out=False, with_last=False)
    for go in (d["grad_out"].bfloat16(), d["grad_out"][:, :4], d["grad_out"].transpose(0, 1).contiguous().transpose(0, 1)):
        with pytest.raises(ValueError):
            lr.delta_scan_backward(*args, go)
    with pytest.raises(lr.LRScanError) as e:
        lr.delta_scan(torch.zeros(1, 2, 1, 257, device="cuda"), torch.zeros(1, 2, 1, 257, device="cuda"),
                      torch.zeros(1, 2, 1, 8, device="cuda"), torch.zeros(1, 2, 1, device="cuda"),
                      torch.zeros(1, 2, 1, device="cuda"))
    assert e.value.status == -2
    with pytest.raises(lr.LRScanError):
        lr.delta_scan(*[t[:, :0].contiguous() for t in args])
    with pytest.raises(lr.LRScanError) as e:
        lr.delta_scan(*args, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == -5


def test_offsets_past_32_bits():
    """A long row of many heads, over 2^31 values: behind its last reset it gives what a short call gives."""
    T, H, K, V, tail = 560000, 32, 64, 128, 200
    gen = torch.Generator(device="cuda").manual_seed(11)

    def normal(*s):
        return torch.randn(s, generator=gen, device="cuda", dtype=torch.bfloat16)

    q, k = (torch.nn.functional.normalize(normal(1, T, 1, K), dim=-1) for _ in range(2))
    v, go = normal(1, T, H, V), normal(1, T, H, V)
    g = -0.1 * torch.rand(1, T, H, generator=gen, device="cuda")
    beta = torch.rand(1, T, H, generator=gen, device="cuda")
    reset = torch.zeros(1, T, dtype=torch.bool, device="cuda")
    reset[:, [0, 1000, T - tail]] = True
    args = (q, k, v, g, beta)
    out = lr.delta_scan(*args, reset=reset, with_last=False)[0][:, T - tail:].clone()
    grads = [t[:, T - tail:].clone() for t in lr.delta_scan_backward(*args, go, reset=reset)[:5]]
    short = [t[:, T - tail:].contiguous() for t in args]
    assert torch.equal(out, lr.delta_scan(*short, with_last=False)[0])
    first = torch.zeros(1, tail, dtype=torch.bool, device="cuda")
    first[:, 0] = True
    want = lr.delta_scan_backward(*short, go[:, T - tail:].contiguous(), reset=first)[:5]
    assert all(torch.equal(a, b) for a, b in zip(grads, want))
