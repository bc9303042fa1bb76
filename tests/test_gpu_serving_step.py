"""The serving example: the same tokens, batched, chunked and continued in different ways, have the same log
probabilities. Keys, values and outputs are rounded to bf16 (2^-8) and activations to e4m3 (2^-4 of a value, or of a
neighbouring one after a different rounding before it) in two layers; probabilities of 1 / 1024 then move by some
hundredths, and an error in a page or an offset moves them by ones."""
import importlib.util
import os

import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu


def test_the_ways_agree():
    spec = importlib.util.spec_from_file_location("serving_step", os.path.join(ROOT, "examples", "serving_step.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    far = example.main()
    assert set(far) == {"prompts together", "token by token", "continuations", "after packing"}
    for what, value in far.items():
        assert value < 0.1, (what, value)
