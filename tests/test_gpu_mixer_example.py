"""The head-decay mixer layer of examples/decay_mixer.py: it trains, and a prompt
continued token by token gives what one call over all tokens gives."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decay_mixer.py")


def test_example_trains_and_serves():
    spec = importlib.util.spec_from_file_location("decay_mixer", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    first, last, worst = mod.main()
    assert last < 0.9 * first, (first, last)
    # bf16 activations: a dozen roundings of 2^-9 between the two ways
    assert worst < 2e-2, worst
