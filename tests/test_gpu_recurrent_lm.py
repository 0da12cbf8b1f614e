"""The example model: its training lowers the loss, packed documents do not see
each other, and token-by-token decoding gives the whole row's logits."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def lm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import recurrent_lm
    return recurrent_lm


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_training_learns_to_count(lm, dtype):
    model = lm.RecurrentLM(dtype=dtype).cuda()
    losses = lm.train(model, 40)
    # from the uniform guess, ln 97 = 4.57, to well below what one token back can tell
    assert losses[0] > 4.0 and losses[-1] < 0.75 * losses[0], losses


def test_documents_do_not_see_each_other(lm):
    model = lm.RecurrentLM().cuda()
    ids = torch.randint(0, 97, (2, 60), device="cuda")
    start = torch.zeros(2, 60, dtype=torch.bool, device="cuda")
    start[:, [0, 25]] = True
    a = model(ids, start)
    ids[:, :25] = torch.randint(0, 97, (2, 25), device="cuda")
    b = model(ids, start)
    assert torch.equal(a[:, 25:], b[:, 25:]) and not torch.equal(a[:, :25], b[:, :25])


def test_decoding_is_the_whole_row(lm):
    model = lm.RecurrentLM().cuda()
    prompt = torch.randint(0, 97, (3, 40), device="cuda")
    ids, seen = lm.generate(model, prompt, 10)
    whole = model(ids)[:, 39:].detach()
    # two orders of the same fp32 sums over a width of 128
    assert (seen - whole).abs().max() <= 1e-4 * whole.abs().max()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_captured_step_replays_to_the_eager_chain(lm, dtype):
    """Lookup, convolution step and gated step of one token in a graph on a stream that has no workspace, the states
    moved on in place: every replay, with eager calls between, gives the eager chain's bits."""
    from test_gpu_graphs_streams import fresh_stream
    lr = lm.lr
    B, V, D, K, steps = 5, 31, 136, 4, 6
    table, gates = torch.randn(V, D, device="cuda").to(dtype), torch.randn(B, 2 * D, device="cuda").to(dtype)
    taps, bias, decay = (torch.randn(*s, device="cuda") for s in ((K, D), (D,), (D,)))
    tokens = torch.randint(0, V, (steps, B), device="cuda")
    starts = torch.rand(steps, B, device="cuda") < 0.2
    ids, reset = tokens[0].clone(), starts[0].clone()
    window, state = torch.zeros(B, K - 1, D, device="cuda", dtype=dtype), torch.zeros(B, D, device="cuda")

    def step():
        c, _ = lr.short_conv_step(lr.embed(ids, table, 2.0), taps, bias, window, reset=reset, activation="silu",
                                  out_state=window)
        return c, lr.gated_step(c, gates[:, :D], gates[:, D:], decay, state, reset=reset, out_state=state)[0]

    def chain(one):
        window.zero_()
        state.zero_()
        rows = []
        for k in range(steps):
            ids.copy_(tokens[k])
            reset.copy_(starts[k])
            rows += [t.clone() for t in (*one(), window, state)]
        return rows

    want = chain(step)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=fresh_stream()):
        out = step()

    def replay():
        graph.replay()
        torch.cuda.synchronize()
        return out

    for _ in range(2):
        assert all(torch.equal(a, b) for a, b in zip(chain(replay), want))
        assert all(torch.equal(a, b) for a, b in zip(chain(step), want))
