"""The AdamW update against its definition in 64 bits: states in 32 and 8 bits,
master weights, many tensors, views at odd addresses, device step numbers in
graphs, and the optimizer class.

Bounds (u = 2^-24).  g = scale grad, b1 m and (1 - b1) g, their sum and the two
factors round once each: dm = 5 u (|b1 m| + |(1 - b1) g|).  v has the square too,
and an 8-bit state's decoding three more: dv = 9 u v.  sqrt halves dv and rounds,
and root, its factor, the sum with eps, the step's factor, a product and a
quotient round: the update's relative error is 4.5 u + 8 u beside dm's share, the
decayed weight's 3 u; one more for the difference.  A stored bf16 adds 2^-8 / 2
of itself as half a step.  A code of e4m3 is off by half a step, 2^-4 of the
value, or half the smallest one, 2^-10 of its scale (a root may be raised to the
smallest: 2^-9).
"""
import copy
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import linear_recurrence_sequence_diag_amd as lr  # noqa: E402

U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
E4M3 = torch.float8_e4m3fn


@pytest.fixture(autouse=True, scope="module")
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lr.library()


def _groups(n):
    return -(-n // lr.ADAMW_GROUP)


def _decode(codes, scale):
    c = codes.cpu().float().flatten().double()
    return c * scale.cpu().double().repeat_interleave(lr.ADAMW_GROUP)[:c.numel()]


class Case:
    def __init__(self, sizes, dtype, bits, master, seed=0, offset=0, zero=False):
        gen = torch.Generator().manual_seed(seed)

        def put(x, kind):
            flat = torch.zeros(x.numel() + offset, dtype=kind, device="cuda")
            flat[offset:] = x.to(kind).cuda()
            return flat[offset:]

        def normal(n, sd):
            return torch.randn(n, generator=gen) * sd * (0.0 if zero else 1.0)

        self.sizes, self.bits = sizes, bits
        w = [torch.randn(n, generator=gen) for n in sizes]
        self.params = [put(x, dtype) for x in w]
        self.masters = [put(x, torch.float32) for x in w] if master else None
        self.grads = [put(torch.randn(n, generator=gen) * 10.0 ** (torch.rand(n, generator=gen) * 6 - 5), dtype)
                      for n in sizes]
        m, v = [normal(n, 0.1) for n in sizes], [normal(n, 0.3) ** 2 for n in sizes]
        self.scale = torch.tensor([0.75], device="cuda")
        self.ms = self.vs = None
        if bits == 32:
            self.m, self.v = [put(x, torch.float32) for x in m], [put(x, torch.float32) for x in v]
        else:
            self.m, self.ms, self.v, self.vs = [], [], [], []
            for x, codes, scales in [(x, self.m, self.ms) for x in m] + [(x.sqrt(), self.v, self.vs) for x in v]:
                s = torch.stack([y.abs().max() for y in x.split(lr.ADAMW_GROUP)]) / 448
                c = torch.where(s.repeat_interleave(lr.ADAMW_GROUP)[:x.numel()] > 0,
                                x / s.repeat_interleave(lr.ADAMW_GROUP)[:x.numel()].clamp(min=1e-30), torch.zeros_like(x))
                flat = torch.zeros(x.numel() + offset, dtype=torch.uint8, device="cuda").view(E4M3)
                flat[offset:].copy_(c.cuda().to(E4M3))
                codes.append(flat[offset:])
                scales.append(s.cuda())

    def update(self, step, **more):
        lr.adamw_update(self.params, self.grads, self.m, self.v, step, masters=self.masters, exp_avg_scales=self.ms,
                        exp_avg_sq_scales=self.vs, **more)

    def state(self, i):
        if self.bits == 32:
            return self.m[i].cpu().double(), self.v[i].cpu().double()
        return _decode(self.m[i], self.ms[i]), _decode(self.v[i], self.vs[i]) ** 2

    def expect(self, step, rate=1e-2, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.1, scaled=True):
        out = []
        for i in range(len(self.sizes)):
            m, v = self.state(i)
            w = (self.masters or self.params)[i].cpu().double()
            g = self.grads[i].cpu().double() * (0.75 if scaled else 1.0)
            b1, b2 = betas
            dm = 5 * U * (b1 * m.abs() + (1 - b1) * g.abs())
            m, v = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
            den = (v / (1 - b2 ** step)).sqrt() + eps
            f = rate / (1 - b1 ** step)
            dw = 4 * U * w.abs() + f * dm / den + 13.5 * U * f * m.abs() / den
            w = w * (1 - rate * weight_decay) - f * m / den
            out.append(dict(w=w, dw=dw + U * w.abs(), m=m, dm=dm + U * m.abs(), v=v, dv=9 * U * v))
        return out

    def check(self, want):
        for i, e in enumerate(want):
            what = f"tensor {i} of {self.sizes[i]}"

            def near(got, ref, d, name):
                off = (got.detach().cpu().double() - ref).abs()
                assert (off <= d).all(), (what, name, (off / d.clamp(min=1e-300)).max())

            p = self.params[i]
            half = 0.0 if p.dtype == torch.float32 else torch.finfo(p.dtype).eps / 2
            if self.masters:
                near(self.masters[i], e["w"], e["dw"], "master")
                assert torch.equal(p, self.masters[i].to(p.dtype)), what
            else:
                near(p, e["w"], e["dw"] * (1 + half) + half * e["w"].abs(), "param")
            if self.bits == 32:
                near(self.m[i], e["m"], e["dm"], "exp_avg")
                near(self.v[i], e["v"], e["dv"], "exp_avg_sq")
                continue
            for codes, scale, x, d, least in ((self.m[i], self.ms[i], e["m"], e["dm"], 2.0 ** -10),
                                              (self.v[i], self.vs[i], e["v"].sqrt(), e["dv"].sqrt() * 0 + 5 * U * e["v"].sqrt(), 2.0 ** -9)):
                assert scale.numel() == _groups(x.numel())
                top = torch.stack([y.abs().max() for y in x.split(lr.ADAMW_GROUP)])
                slack = torch.stack([y.max() for y in d.split(lr.ADAMW_GROUP)])
                near(scale * 448, top, slack + 6 * U * top, "scale")
                s = scale.cpu().double().repeat_interleave(lr.ADAMW_GROUP)[:x.numel()]
                near(_decode(codes, scale), x, (2.0 ** -4 + 8 * U) * x.abs() + d * (1 + 2.0 ** -4) + least * s * (1 + 8 * U),
                     "codes")
            root = _decode(self.v[i], self.vs[i])
            assert ((root > 0) == (e["v"] > 0)).all(), what


SIZES = [[1], [255, 256, 257], [4096, 4097, 3, 1000, 16384 + 5], [65 * 256 * 4 + 2]]


@pytest.mark.parametrize("offset", [0, 1, 3])
@pytest.mark.parametrize("master", [False, True])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_update(dt, bits, master, offset):
    for seed, sizes in enumerate(SIZES):
        c = Case(sizes, DT[dt], bits, master, seed, offset)
        for step in (1, 7):
            want = c.expect(step)
            c.update(step, rate=1e-2, betas=(0.9, 0.99), weight_decay=0.1, grad_scale=c.scale)
            c.check(want)


@pytest.mark.parametrize("bits", [32, 8])
def test_from_zero_states_with_zero_gradients(bits):
    c = Case([700, 5], torch.float32, bits, False, zero=True)
    c.grads[0][256:512] = 0  # a group without anything
    c.grads[1].zero_()
    want = c.expect(1, scaled=False, weight_decay=0.0)
    before = [p.clone() for p in c.params]
    c.update(1, rate=1e-2, betas=(0.9, 0.99), weight_decay=0.0)
    c.check(want)
    assert torch.equal(c.params[1], before[1]) and torch.equal(c.params[0][256:512], before[0][256:512])
    if bits == 8:
        assert c.ms[0][1] == 0 and c.vs[0][1] == 0


def test_a_small_root_beside_a_large_one_is_not_lost():
    c = Case([256], torch.float32, 8, False, zero=True)
    c.grads[0].fill_(1e-9)
    c.grads[0][7] = 10.0
    c.update(1, rate=1e-3, betas=(0.9, 0.99), weight_decay=0.0, eps=0.0)
    root = _decode(c.v[0], c.vs[0])
    assert (root > 0).all() and root[7] > 0.9
    before = c.params[0].clone()
    c.grads[0].zero_()
    c.update(2, rate=1e-3, betas=(0.9, 0.99), weight_decay=0.0, eps=0.0)
    # m of the small ones is below its own smallest code, so nothing moves them far
    moved = (c.params[0] - before).abs()
    assert torch.isfinite(moved).all() and moved.max() <= 1e-2


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors(bits):
    sizes = [1 + 37 * i % 1500 for i in range(200)]
    c = Case(sizes, torch.bfloat16, bits, True, 5)
    want = c.expect(3)
    c.update(3, rate=1e-2, betas=(0.9, 0.99), weight_decay=0.1, grad_scale=c.scale)
    c.check(want)


def test_neighbours_of_the_tensors_stay():
    flat = {k: torch.full((3000,), 7.0, device="cuda") for k in ("p", "m", "v", "x")}
    flat["v"].fill_(4.0)
    cut = slice(515, 515 + 1021)
    keep = {k: t.clone() for k, t in flat.items()}
    grads = torch.randn(3000, device="cuda")
    lr.adamw_update([flat["p"][cut]], [grads[cut]], [flat["m"][cut]], [flat["v"][cut]], 2, masters=[flat["x"][cut]])
    for k, t in flat.items():
        assert torch.equal(t[:515], keep[k][:515]) and torch.equal(t[515 + 1021:], keep[k][515 + 1021:]), k
        assert not torch.equal(t[cut], keep[k][cut])


@pytest.mark.parametrize("bits", [32, 8])
def test_a_captured_update_counts_its_steps(bits):
    """The step's number and the gradients' factor on the device: every replay is the eager update of its number."""
    eager = Case([5000, 33, 300], torch.bfloat16, bits, True, 9)
    held = copy.deepcopy(eager)
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        step.add_(1)
        held.update(step, rate=1e-2, grad_scale=held.scale)
    torch.cuda.synchronize()
    for t in range(1, 6):
        for a, b in zip(eager.grads, held.grads):
            a.normal_()
            b.copy_(a)
        eager.scale.fill_(1.0 / t)
        held.scale.fill_(1.0 / t)
        graph.replay()
        # the eager one by a device number too: both form the corrections on the device
        eager.update(torch.tensor([t], device="cuda"), rate=1e-2, grad_scale=eager.scale)
        torch.cuda.synchronize()
        assert int(step) == t
        for name in ("params", "masters", "m", "v"):
            for a, b in zip(getattr(eager, name), getattr(held, name)):
                assert torch.equal(a.float(), b.float()), (t, name)


def test_host_and_device_numbers_agree():
    for t in (1, 2, 1000, 10 ** 6):
        a = Case([3000], torch.float32, 32, False, 2)
        b = copy.deepcopy(a)
        want = a.expect(t)
        a.update(t, rate=1e-2, betas=(0.9, 0.99), weight_decay=0.1, grad_scale=a.scale)
        b.update(torch.tensor([t], device="cuda"), rate=1e-2, betas=(0.9, 0.99), weight_decay=0.1, grad_scale=b.scale)
        a.check(want)
        b.check(want)


def test_on_another_stream():
    c = Case([100000], torch.float32, 32, False, 4)
    want = c.expect(2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.update(2, rate=1e-2, betas=(0.9, 0.99), weight_decay=0.1, grad_scale=c.scale)
    torch.cuda.current_stream().wait_stream(side)
    c.check(want)


@pytest.mark.parametrize("bits,master", [(32, False), (32, True), (8, False), (8, True)])
def test_optimizer(bits, master):
    gen = torch.Generator(device="cuda").manual_seed(0)

    def model():
        torch.manual_seed(3)
        return torch.nn.ModuleList([torch.nn.Linear(70, 33), torch.nn.Linear(33, 5)]).cuda().to(torch.bfloat16)

    a = model()
    opt = lr.AdamW(a.parameters(), rate=1e-2, betas=(0.9, 0.99), weight_decay=0.1, state_bits=bits, master=master)
    ps = list(a.parameters())
    c = Case([p.numel() for p in ps], torch.bfloat16, bits, master, zero=True)
    for i, p in enumerate(ps):
        c.params[i].copy_(p.detach().flatten())
        if master:
            c.masters[i].copy_(p.detach().flatten())
    for t in range(1, 5):
        for i, p in enumerate(ps):
            p.grad = torch.randn(p.shape, generator=gen, device="cuda").to(p.dtype)
            c.grads[i].copy_(p.grad.flatten())
        opt.step(grad_scale=c.scale)
        c.update(t, rate=1e-2, betas=(0.9, 0.99), weight_decay=0.1, grad_scale=c.scale)
        if t == 2:  # saved and loaded: another optimizer goes on alike
            saved = copy.deepcopy(opt.state_dict())
            opt = lr.AdamW(a.parameters(), rate=0.5, state_bits=bits, master=master)
            opt.load_state_dict(saved)
    for i, p in enumerate(ps):
        assert torch.equal(p.detach().flatten(), c.params[i]), i
        s = opt.state[p]
        assert s["step"] == 4 and torch.equal(s["exp_avg"].flatten().float(), c.m[i].float())
        assert s["exp_avg"].dtype == (E4M3 if bits == 8 else torch.float32)
    assert math.isclose(opt.param_groups[0]["lr"], 1e-2)


def test_refusals():
    def tensors(n=10, kind=torch.float32):
        return [torch.zeros(n, device="cuda", dtype=kind)]

    p, g, m, v = (tensors() for _ in range(4))
    e = [torch.zeros(10, device="cuda", dtype=torch.uint8).view(E4M3)]
    s = tensors(1)
    up = lr.adamw_update
    bad = [
        lambda: up([], [], [], [], 1), lambda: up(p, [], m, v, 1), lambda: up(p, g, m, tensors(9), 1),
        lambda: up(p, tensors(10, torch.bfloat16), m, v, 1), lambda: up(p, g, tensors(10, torch.bfloat16), v, 1),
        lambda: up(p, [torch.zeros(20, device="cuda")[::2]], m, v, 1), lambda: up(p, [torch.zeros(10)], m, v, 1),
        lambda: up(p, g, m, v, 1, masters=tensors(10, torch.bfloat16)), lambda: up(p, g, e, e, 1),
        lambda: up(p, g, e, e, 1, exp_avg_scales=s), lambda: up(p, g, m, v, 1, exp_avg_scales=s, exp_avg_sq_scales=tensors(1)),
        lambda: up(p, g, e, e, 1, exp_avg_scales=tensors(2), exp_avg_sq_scales=tensors(2)),
        lambda: up(p + p, g + g, m + tensors(), v + tensors(), 1), lambda: up(p + tensors(), g + g, m + m, v + tensors(), 1),
        lambda: up(p, g, m, v, torch.tensor([1])), lambda: up(p, g, m, v, torch.ones(1, device="cuda")),
        lambda: up(p, g, m, v, 1, grad_scale=2.0), lambda: up(p, g, m, v, 1, grad_scale=torch.ones(2, device="cuda")),
        lambda: lr.AdamW([torch.nn.Parameter(p[0])], state_bits=16),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for more in (dict(rate=math.nan), dict(betas=(1.0, 0.9)), dict(betas=(0.9, -0.1)), dict(eps=-1.0),
                 dict(weight_decay=math.inf)):
        with pytest.raises(lr.LRScanError):
            up(p, g, m, v, 1, **more)
    with pytest.raises(lr.LRScanError):
        up(p, g, m, v, 0)
    with pytest.raises(lr.LRScanError):  # an empty tensor
        up(tensors(0), tensors(0), tensors(0), tensors(0), 1)
