"""The few-token expert layer (sgemm_experts_layer, include/expert_layer.h) near
its largest numbers of tokens, with rows long enough that every warp walks many
steps, and choices that crowd on few experts; bounds as in test_gpu_experts_layer.py."""
import numpy as np
import pytest

from test_gpu_experts_layer import TYPES, WTYPES, Layer, gpu_ready, run  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("wtype", WTYPES)
@pytest.mark.parametrize("type_", TYPES)
@pytest.mark.parametrize("T,k,E,H,F", [(17, 2, 6, 1024, 1024), (33, 2, 6, 1024, 1280),
                                       (64, 2, 5, 1040, 1024), (24, 4, 16, 1500, 1100),
                                       (64, 8, 40, 1024, 200)])
def test_many_tokens_on_long_rows(type_, wtype, T, k, E, H, F):
    rng = np.random.default_rng(T)
    run(Layer(type_, wtype, E, H, F, rng), T, k, rng, drop=0.05)


@pytest.mark.parametrize("wtype", WTYPES)
@pytest.mark.parametrize("T,E,crowd", [(64, 8, 50), (32, 30, 28), (64, 100, 60), (20, 3, 20),
                                       (12, 6, 11)])
def test_choices_that_crowd_on_one_expert(wtype, T, E, crowd):
    """The first `crowd` tokens choose the same expert, first, in the middle or last
    in order; the others spread."""
    rng = np.random.default_rng(E)
    layer = Layer("bf16", wtype, E, 272, 1100, rng)
    for favourite in (0, E // 2, E - 1):
        ids = rng.integers(0, E, (T, 2))
        ids[:crowd, 0] = favourite
        run(layer, T, 2, rng, ids=ids)
