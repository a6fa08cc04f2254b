"""The example layer: decoding continues the prefill, and training descends.

Decode and prefill quantise the same rows in the same way, so they differ where the
recurrences' own roundings move an element across a rounding boundary: bf16 outputs (2^-8),
then e2m1 elements of the out-projection's input, single steps of which (up to a third of an
element) are averaged over more than a thousand products: 5% of the largest output is allowed,
and for the fp32 states, which see only the bf16 projections (equal in both), 1%."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_layer.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("hybrid_layer", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("width,heads,batch,prompt,tokens", [(512, 4, 2, 200, 6), (1024, 8, 1, 65, 3), (256, 2, 5, 1, 4)])
def test_decode_continues_the_prefill(example, width, heads, batch, prompt, tokens):
    out, state = example.prefill_then_decode(width, heads, batch, prompt, tokens, seed=prompt)
    assert out < 5e-2 and state < 1e-2


def test_training_descends(example):
    losses = example.train(steps=20)
    assert losses[-1] < 0.5 * losses[0]
