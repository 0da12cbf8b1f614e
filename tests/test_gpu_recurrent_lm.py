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
