"""The example model with the gated delta rule, the AdamW update and adjusted logits together: gradients against a
64-bit form of the whole model, packed documents, token-by-token decoding, and training and decoding steps captured
in graphs."""
import math
import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

U = 2.0 ** -24


@pytest.fixture(scope="module")
def lm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import recurrent_lm
    return recurrent_lm


def _plain(p, ids, start, heads, width):
    """The model's logits from its formulas on the CPU, a token at a time, in p's precision."""
    B, T = ids.shape
    x = p["table"][ids] * math.sqrt(width)
    K = p["taps"].shape[0]
    hd = width // heads
    S = x.new_zeros(B, heads, hd, hd)
    rows = []
    for t in range(T):
        z = p["taps_bias"].expand(B, width)
        alive = torch.ones(B, 1, dtype=torch.bool)
        for j in range(K):  # the input j tokens ago, unless a document starts in between
            if t - j >= 0:
                z = z + torch.where(alive, x[:, t - j] * p["taps"][K - 1 - j], torch.zeros((), dtype=x.dtype))
                alive = alive & ~start[:, t - j, None]
        c = z * torch.sigmoid(z)
        m = c @ p["gates"]
        q, k, v = m[:, :3 * width].unflatten(-1, (3 * heads, hd)).split(heads, 1)
        q, k = (y / y.norm(dim=-1, keepdim=True) for y in (q, k))
        gate, beta = m[:, 3 * width:].chunk(2, -1)
        a = torch.exp(-torch.nn.functional.softplus(gate + p["decay"]))
        S = torch.where(start[:, t, None, None, None], torch.zeros_like(S), S) * a[..., None, None]
        e = v - (S * k[..., None]).sum(2)
        S = S + k[..., None] * (torch.sigmoid(beta)[..., None] * e)[:, :, None]
        h = (S * q[..., None]).sum(2).flatten(1)
        rows.append((h + x[:, t]) @ p["head"])
    return torch.stack(rows, 1)


def _plain_gradients(model, ids, start, w, dtype):
    p = {n: t.detach().cpu().to(dtype).requires_grad_() for n, t in model.named_parameters()}
    logits = _plain(p, ids, start, model.heads, p["table"].shape[1])
    (logits * w.to(dtype)).sum().backward()
    return {"logits": logits.detach(), **{n: t.grad for n, t in p.items()}}


@pytest.mark.parametrize("T", [1, 37, 70])
def test_gradients_of_the_whole_model(lm, T):
    model = lm.RecurrentLM(vocab=23, width=64, mixer="delta").cuda()
    gen = torch.Generator().manual_seed(T)
    ids = torch.randint(0, 23, (3, T), generator=gen)
    start = torch.rand(3, T, generator=gen) < 0.1
    w = torch.randn(3, T, 23, generator=gen)
    logits = model(ids.cuda(), start.cuda())
    (logits * w.cuda()).sum().backward()
    got = {"logits": logits.detach(), **{n: t.grad for n, t in model.named_parameters()}}
    ref, f32 = (_plain_gradients(model, ids, start, w, d) for d in (torch.float64, torch.float32))
    for n, r in ref.items():
        # another order of the same fp32 sums: a multiple of what fp32 loses on the CPU, and units of the largest
        bound = 8 * (f32[n].double() - r).abs().max() + 64 * U * r.abs().max()
        off = (got[n].double().cpu() - r).abs().max()
        print(f"{n}: {(off / bound).item():.2f} of the bound")
        assert off <= bound, n


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("optimizer", ["adamw", "adamw8"])
def test_training_runs(lm, dtype, optimizer):
    model = lm.RecurrentLM(dtype=dtype, mixer="delta").cuda()
    before = [p.detach().clone() for p in model.parameters()]
    losses = lm.train(model, 5, B=4, T=100, optimizer=optimizer)
    assert len(losses) == 5 and all(math.isfinite(x) for x in losses)
    for p, q in zip(model.parameters(), before):
        assert torch.isfinite(p).all() and not torch.equal(p, q)


def test_documents_do_not_see_each_other(lm):
    model = lm.RecurrentLM(mixer="delta").cuda()
    ids = torch.randint(0, 97, (2, 160), device="cuda")
    start = torch.zeros(2, 160, dtype=torch.bool, device="cuda")
    start[:, [0, 75]] = True
    a = model(ids, start)
    ids[:, :75] = torch.randint(0, 97, (2, 75), device="cuda")
    b = model(ids, start)
    assert torch.equal(a[:, 75:], b[:, 75:]) and not torch.equal(a[:, :75], b[:, :75])


def test_decoding_is_the_whole_row(lm):
    model = lm.RecurrentLM(mixer="delta").cuda()
    prompt = torch.randint(0, 97, (3, 70), device="cuda")
    ids, seen = lm.generate(model, prompt, 10)
    whole = model(ids)[:, 69:].detach()
    # the recurrence in blocks and token by token, sums over widths of 128 in fp32
    assert (seen - whole).abs().max() <= 1e-4 * whole.abs().max()


@pytest.mark.parametrize("mixer", ["gated", "delta"])
def test_penalties_of_a_generated_row(lm, mixer):
    """Every choice is the largest of the step's logits after the penalties' formulas in 64 bits."""
    model = lm.RecurrentLM(vocab=17, width=64, mixer=mixer).cuda()
    prompt = torch.randint(0, 17, (4, 9), device="cuda")
    rep, pres, freq = 1.5, 0.75, 0.25  # exact in fp32, so a choice between near values is all that rounding moves
    ids, seen = lm.generate(model, prompt, 30, rep, pres, freq)
    for i in range(30):
        z = seen[:, i].double().cpu()
        said = torch.nn.functional.one_hot(ids[:, :9 + i].cpu(), 17).sum(1)
        answered = torch.nn.functional.one_hot(ids[:, 9:9 + i].cpu(), 17).sum(1) if i else torch.zeros_like(said)
        z = torch.where(said > 0, torch.where(z > 0, z / rep, z * rep), z) - freq * answered - pres * (answered > 0)
        chosen = z.gather(1, ids[:, 9 + i, None].cpu())[:, 0]
        assert (chosen >= z.amax(1) - 8 * U * seen[:, i].abs().max().item() * rep).all()
    free, _ = lm.generate(model, prompt, 30)
    assert not torch.equal(free, ids)


def test_a_captured_training_step(lm):
    """Forward, backward and the update with its step on the device, in one graph: replays give the eager chain's bits."""
    from test_gpu_graphs_streams import fresh_stream
    lr = lm.lr
    gen = torch.Generator().manual_seed(5)
    B, T, H, K, V = 2, 150, 3, 32, 40

    def normal(*s):
        return torch.randn(s, generator=gen).cuda()

    first = [torch.nn.functional.normalize(normal(B, T, H, K), dim=-1) for _ in range(2)]
    first += [normal(B, T, H, V), -torch.rand(B, T, H, generator=gen).cuda(), torch.rand(B, T, H, generator=gen).cuda()]
    go = normal(B, T, H, V)
    reset = (torch.rand(B, T, generator=gen) < 0.05).cuda()
    params = [t.clone() for t in first]
    m, v = ([torch.zeros_like(t) for t in params] for _ in range(2))
    count = torch.zeros(1, dtype=torch.int64, device="cuda")
    # of the backward, which is the larger one
    ws = torch.empty(lr.scan_delta_workspace_bytes(B, T, H, H, K, V, lr.F32, 1), dtype=torch.uint8, device="cuda")

    def train():
        out, last = lr.delta_scan(*params, reset=reset, workspace=ws)
        grads = lr.delta_scan_backward(*params, go, reset=reset, workspace=ws)[:5]
        count.add_(1)
        lr.adamw_update(params, list(grads), m, v, count, rate=1e-3)
        return out, last

    def chain(one):
        for t, x in zip(params, first):
            t.copy_(x)
        for t in (*m, *v, count):
            t.zero_()
        rows = []
        for _ in range(4):
            rows += [t.clone() for t in (*one(), *params, *m, *v)]
        return rows

    want = chain(train)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=fresh_stream()):
        held = train()

    def replay():
        graph.replay()
        torch.cuda.synchronize()
        return held

    for _ in range(2):
        assert all(torch.equal(a, b) for a, b in zip(chain(replay), want))
        assert all(torch.equal(a, b) for a, b in zip(chain(train), want))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_captured_decode_step(lm, dtype):
    """Lookup, delta step, logits and their adjustment of one token in a graph, the state moved on in place and the
    history grown on the device: every replay, with eager calls between, gives the eager chain's bits."""
    from test_gpu_graphs_streams import fresh_stream
    lr = lm.lr
    gen = torch.Generator().manual_seed(6)
    B, vocab, H, HK, K, V, steps = 5, 131, 4, 2, 24, 40, 6
    width = (2 * HK * K + H * V)
    table = torch.randn(vocab, width, generator=gen).to(dtype).cuda()
    head = torch.randn(H * V, vocab, generator=gen).to(dtype).cuda()
    gate, beta = -torch.rand(B, H, generator=gen).cuda(), torch.rand(B, H, generator=gen).cuda()
    rep, pres = (torch.full((B,), x, device="cuda") for x in (1.25, 0.5))
    allowed = torch.randint(-2 ** 31, 2 ** 31, (B, -(-vocab // 32)), generator=gen, dtype=torch.int64).to(torch.int32).cuda()
    begin = torch.randint(0, vocab, (B,), generator=gen).cuda()
    token, said = begin.clone(), torch.zeros(B, dtype=torch.int64, device="cuda")
    history, state = torch.zeros(B, steps + 2, dtype=torch.int64, device="cuda"), torch.zeros(B, H, K, V, device="cuda")

    def step():
        x = lr.embed(token, table)
        q, k = (y.unflatten(-1, (HK, K)) for y in x[:, :2 * HK * K].chunk(2, -1))
        v = x[:, 2 * HK * K:].unflatten(-1, (H, V))
        h, _ = lr.delta_step(q, k * K ** -0.5, v, gate, beta, state=state, out_state=state)
        z = lr.adjust_logits(h.flatten(1) @ head, history, said, repetition=rep, presence=pres, allowed=allowed)
        token.copy_(z.argmax(-1))
        history.scatter_(1, said[:, None], token[:, None])
        said.add_(1)
        return h, z

    def chain(one):
        token.copy_(begin)
        for t in (said, history, state):
            t.zero_()
        rows = []
        for _ in range(steps):
            rows += [t.clone() for t in (*one(), token, history, state)]
        return rows

    want = chain(step)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=fresh_stream()):
        held = step()

    def replay():
        graph.replay()
        torch.cuda.synchronize()
        return held

    for _ in range(2):
        assert all(torch.equal(a, b) for a, b in zip(chain(replay), want))
        assert all(torch.equal(a, b) for a, b in zip(chain(step), want))


def test_the_optimizer_refuses_capture(lm):
    from test_gpu_graphs_streams import fresh_stream
    w = torch.nn.Parameter(torch.ones(8, device="cuda"))
    opt = lm.lr.AdamW([w])
    w.grad = torch.ones_like(w)
    opt.step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=fresh_stream()):
        kept = w.detach() + 1
        with pytest.raises(RuntimeError, match="captured"):
            opt.step()
    assert kept.numel() == 8


def test_the_model_refuses_other_mixers_and_widths(lm):
    for more in (dict(mixer="other"), dict(mixer="delta", width=72)):
        with pytest.raises(ValueError, match="mixer"):
            lm.RecurrentLM(**more)
