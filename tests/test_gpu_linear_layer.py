"""The per-head-decay linear attention layer of examples/linear_layer.py: prompts followed by single
tokens equal the whole sequences in one call, and a training step's gradients are finite.

Tolerances.  Both ways compute each output from the same bf16 inputs; they differ by the roundings
of o and y (2^-9 each, of values up to about 6 times the rms, plus the norm's common factor): within
2^-5 of the rms.  fp32: 1e-4.  States: 1e-5 in the 2-norm, as in the attention's own tests.
"""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,lengths,heads,d", [("bfloat16", (300, 45, 1024), 4, 128),
                                                   ("float32", (70, 1), 3, 64)])
def test_prompts_then_tokens(dtype, lengths, heads, d):
    import torch
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "linear_layer.py")
    spec = importlib.util.spec_from_file_location("linear_layer", path)
    layer = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(layer)
    off, off_state, grads = layer.demo(lengths, 3, heads, d, getattr(torch, dtype))
    assert off <= (2.0 ** -5 if dtype == "bfloat16" else 1e-4)
    assert off_state <= 1e-5
    T = sum(lengths) + 3 * len(lengths)
    assert grads["dq"].shape == (T, heads, d) and grads["dg"].shape == (T, heads)
    for t in grads.values():
        assert bool(torch.isfinite(t).all())
