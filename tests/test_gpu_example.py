"""The example that runs the operators together, as they would be used."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


def test_hybrid_step():
    """A tree of drafts verified at once against its accepted paths token by token.  Both
    sides round the residual stream and the projections to bf16 (2^-8) about a dozen
    times (2 layers, 2 sublayers, 3 roundings), in matrix products of different shapes:
    2^-4 of the largest output, half of that in the states; the first layer's conv
    states hold the same projections of the same inputs."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_step.py")
    spec = importlib.util.spec_from_file_location("hybrid_step", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    worst, size, state, conv = example.main()
    assert worst <= 2.0 ** -4 * size
    assert state <= 2.0 ** -5
    assert conv
