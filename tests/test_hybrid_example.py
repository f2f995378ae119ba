"""The hybrid decoder example: decode steps behind a prompt give what the prompt
call gives over the same tokens."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


def test_decode_steps_agree_with_one_longer_prompt():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_step.py")
    spec = importlib.util.spec_from_file_location("hybrid_step", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    # Both sides end in e4m3, off by up to 2^-4 of a value each: rms 2^-4 / sqrt(3) a side at most.  The layers between
    # round some tens of bf16 operands (2^-8 each), differently in the two forms.
    assert example.main() < 2 * 2.0 ** -4 / 3 ** 0.5 + 16 * 2.0 ** -8


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_step.py")
    spec = importlib.util.spec_from_file_location("hybrid_step", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_a_refused_request_stops_the_step_and_leaves_the_next_one_right():
    import torch

    example = _example()
    x = torch.randn((150, 512), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").to(torch.bfloat16)
    lens = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    model, fresh = (example.HybridDecoder(requests=2, n_pages=4) for _ in range(2))
    with pytest.raises(RuntimeError, match="1 requests refused"):
        model.step(x[:150].repeat(2, 1), lens(20, 280), True)                 # 1 + 5 pages of 4
    for prompts, rows, new in ((True, x[:150], (20, 130)), (False, x[:2], (1, 1))):
        got, want = (m.step(rows, lens(*new), prompts)[2] for m in (model, fresh))
        assert torch.equal(got, want)
    with pytest.raises(ValueError, match="without cached tokens"):
        model.step(x[:10], lens(5, 5), True)
    with pytest.raises(ValueError, match="one token a request"):
        model.step(x[:3], lens(2, 1), False)
    with pytest.raises(RuntimeError, match="refused"):
        for _ in range(64):                                                    # until the pages run out
            model.step(x[:2], lens(1, 1), False)
