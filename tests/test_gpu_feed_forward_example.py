"""The feed-forward block's example (examples/feed_forward.py) runs its
operators together, served in 4 and in 8 bits and trained, and agrees with fp32
references.

Bounds, from the roundings on the way.  4 bits: a block's largest of 16 normal
values is some 2.2 deviations, so that steps are 0.18, 0.37 and 0.73 deviations
wide and a value is off by about 0.09 deviations; gate and up take two such
roundings each (0.13), their product 0.18, the down product two more (0.13): 0.23
in quadrature, up to twice the steps for scales that are powers of two: below 0.4.
Experts in 8 bits: weights twice with 127 steps (0.9% a quantisation, 1.3%) and
bf16 rows (0.2% each): below 3%.  Training rounds rows to bf16 two or three times
(0.2% each): below 1%."""
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
        "feed_forward_example", os.path.join(ROOT, "examples", "feed_forward.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    errors = example.main(tokens=tokens, steps=2)
    for name in ("nv prompt", "nv decoding", "mx prompt", "mx decoding"):
        assert errors[name] < 0.4, errors
    assert errors["experts"] < 0.03, errors
    for name in ("out", "dx", "dnorm", "dw"):
        assert errors[name] < 0.01, errors
