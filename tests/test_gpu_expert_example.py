"""The expert layer's example (examples/expert_layer.py) runs its operators
together, served in 8 bits (prompts and single tokens) and trained, and agrees
with fp32 references.

Bounds, from the roundings on the way: serving quantises activations and
weights twice each with 127 steps (about 0.3 / 127 of a row's largest value per
value, largest values being some 3 to 4 deviations: 0.9% a quantisation, four
of them in quadrature 1.8%) and rounds to bf16 (0.2%): below 4%.  Training
rounds rows to bf16 two or three times (0.2% each): below 1%."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("tokens", [5, 700])
def test_example(tokens):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location(
        "expert_layer_example", os.path.join(ROOT, "examples", "expert_layer.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    errors = example.main(tokens=tokens, steps=2)
    assert errors["prompt"] < 0.04 and errors["decoding"] < 0.04, errors
    for name in ("out", "dx", "dweights", "dw"):
        assert errors[name] < 0.01, errors
