"""The example model's generated rows."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "recurrent_lm.py")
    spec = importlib.util.spec_from_file_location("recurrent_lm_generate", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("mixer", ["gated", "delta"])
@pytest.mark.parametrize("rules", [{}, dict(repetition=1.3, presence=0.4, frequency=0.1)], ids=["plain", "penalties"])
def test_prompts_of_either_whole_type_give_the_same_rows(lm, mixer, rules):
    """int64, the type of the chosen tokens, whatever the prompt's."""
    model = lm.RecurrentLM(mixer=mixer).cuda()
    prompt = torch.randint(0, 97, (3, 20), device="cuda")
    want, seen = lm.generate(model, prompt, 6, **rules)
    got, again = lm.generate(model, prompt.int(), 6, **rules)
    assert want.dtype == got.dtype == torch.int64 and torch.equal(want, got) and torch.equal(seen, again)
    assert torch.equal(got[:, :20], prompt)
