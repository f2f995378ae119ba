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
