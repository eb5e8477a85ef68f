"""The example that runs the operators for long contexts as a server would: each flow's last step against attention
in 32 bits over the tokens that it attends to.

Tolerance (relative, 2-norm): the result's rounding to 16 bits, half a step of each element (bf16 2^-8, f16 2^-11),
and as much again for the reference's sums and weights in 32 bits: twice that."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("long_context_example",
                                                  os.path.join(ROOT, "examples", "long_context.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("kw,most", [
    ({}, 2.0 ** -7), (dict(storage="mxfp8", dim=128, dtype="f16"), 2.0 ** -10), (dict(storage="mxfp4", page=8), 2.0 ** -7)])
def test_flows(example, kw, most):
    assert example.shared(**kw) < most
    chosen, whole = example.selected(**kw)
    assert chosen < most
    # every page selected: nothing is left out
    chosen, whole = example.selected(**dict(kw, budget=300))
    assert chosen < most and whole < most
    last, held = example.evicted(**kw)
    assert last < most and held == 64 + (200 - 128) % 64
