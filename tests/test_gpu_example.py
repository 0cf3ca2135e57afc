"""The example's training and serving steps (needs an MI355X)."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_layer.py")


def test_moe_layer_example():
    spec = importlib.util.spec_from_file_location("moe_layer", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    # bf16 values pass through up to four roundings of 2^-9 relative each on the
    # way to a gradient (inputs are exact): 4 * 2^-9 and, as the router's own
    # product and its softmax see rounded logits of size up to 4, 8 * 2^-8 there
    for name, error in example.main().items():
        assert error <= (8 * 2.0 ** -8 if name in ("grad router", "grad x") else 4 * 2.0 ** -8), (name, error)
    for name, error in example.main(tokens=1, experts=4, topk=2).items():
        assert error <= (8 * 2.0 ** -8 if name in ("grad router", "grad x") else 4 * 2.0 ** -8), (name, error)
