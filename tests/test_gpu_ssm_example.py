"""The example's stack of mixers: gradients through every operator, training, and single tokens against a pass over
the whole prompt."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "ssm_mixer.py")
    spec = importlib.util.spec_from_file_location("ssm_mixer_example", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_training_lowers_the_loss(ex):
    import math

    import torch

    torch.manual_seed(0)
    model = ex.Model().cuda()
    losses = ex.train(model, torch.Generator().manual_seed(1), 40)
    assert all(math.isfinite(v) for v in losses)
    assert sum(losses[-5:]) / 5 < 0.8 * sum(losses[:5]) / 5
    for name, p in model.named_parameters():
        assert p.grad is not None and bool(p.grad.abs().max() > 0), name


def test_tokens_follow_the_prompt(ex):
    """The last tokens decoded one by one from the state of what is before them give the logits of one pass over all:
    bf16 roundings on two ways of computing the same, through two blocks."""
    import torch

    torch.manual_seed(0)
    model = ex.Model().cuda()
    letters, off, _ = ex.words(torch.Generator().manual_seed(2), 5, "cuda")
    whole, _ = model.prompt(letters, off)
    lens = off.diff().long()
    last = 4
    keep = torch.cat([torch.arange(int(o), int(o + n) - last, device="cuda") for o, n in zip(off[:-1], lens)])
    short = torch.cat([off.new_zeros(1), (lens - last).cumsum(0).to(torch.int32)])
    _, states = model.prompt(letters[keep], short)
    for t in range(last):
        at = off[1:].long() - last + t
        got = model.token(letters[at], states)
        assert float((got - whole[at]).abs().max() / whole.abs().max()) <= 3e-2
