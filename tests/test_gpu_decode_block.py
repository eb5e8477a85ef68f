"""The example that runs the operators of a tensor-parallel attention block together: its last step
against the block computed in 32 bits without a cache.

Tolerances (relative, 2-norm of all outputs): q, k, v, the heads and the result are each rounded to
16 bits, 2^-9 (bf16) or 2^-12 (f16) of their norm at most, and what rounds q and k moves the scores
(of magnitude 1) by as much: under 8 such roundings, 2^-6 and 2^-9. A code of 3 bits after the first is
within 2^-4 of its value, uniformly so 2^-4 / sqrt(3) in norm; keys and values each carry one: 2^-3. One bit
after the first: 2^-2 each, 2^-1 together."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("storage,dtype,most", [
    ("16bit", "bf16", 2.0 ** -6), ("16bit", "f16", 2.0 ** -9), ("mxfp8", "bf16", 2.0 ** -3),
    ("mxfp4", "f16", 2.0 ** -1)])
def test_last_step(storage, dtype, most):
    spec = importlib.util.spec_from_file_location(
        "decode_block", os.path.join(ROOT, "examples", "decode_block.py"))
    block = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(block)
    assert block.main(storage, steps=40, dtype=dtype) < most
    assert block.main(storage, steps=5, dtype=dtype, ranks=2, hidden=512, q_heads=6, kv_heads=2,
                      head_dim=128, batch=6, page=8, most=64) < most
