"""The hybrid decode example runs both layer kinds over one page pool and agrees with fp64 attention."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_decode.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("hybrid_decode", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("steps,batch,prompt", [(70, 6, 300), (3, 1, 17)])
def test_hybrid_decode_example(example, steps, batch, prompt):
    # bf16 weights and outputs: 2^-8 of each, as in the decode tests, against the largest value
    worst, h = example.run(steps, batch, prompt)
    assert worst < 2 ** -6 and torch.isfinite(h).all()
