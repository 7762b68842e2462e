"""The router in one workgroup for 17 to 64 tokens (each wave has several) on the
GPU against the float64 oracle: experts, offsets and order equal, weights within
oracle.moe_weight_bound."""
import numpy as np
import pytest

import oracle
from tests.test_gpu_moe import _check_route, _rng, _to

pytestmark = pytest.mark.gpu

# tokens, experts, topk: all in one launch, which tests/test_moe_route_launches.py checks
ROUTES = [(17, 120, 8), (31, 66, 3), (33, 62, 5), (40, 50, 7), (48, 42, 1), (50, 40, 16), (63, 32, 2), (64, 8, 2), (64, 32, 16),
          (64, 1, 1)]


@pytest.fixture(scope="module")
def g(gpu_lib):
    import post_weight_quantization_11_amd as g
    return g


@pytest.mark.parametrize("tokens,experts,k", ROUTES)
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_route_of_several_tokens_a_wave(g, tokens, experts, k, dtype):
    rng = _rng(tokens, experts, k, 71)
    L, L64 = _to(rng.standard_normal((tokens, experts)) * 2, dtype, experts + 5)
    for renormalize in (True, False):
        _check_route(g.gptq_moe_route(L, k, renormalize=renormalize), L64, k, renormalize)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_ties_and_masked_logits_in_every_wave(g, dtype):
    """Rows of few values, of zeros, without any logit, with infinities and NaN, as
    the first to the last token of a wave (tokens go to sixteen waves in turn)."""
    rng = _rng(40, 50)
    T, E, k = 40, 50, 6
    l = rng.integers(-2, 3, size=(T, E)).astype(np.float64)
    for t in range(3, T, 4):
        l[t] = -np.inf
    for t in range(5, T, 7):
        l[t] = np.nan
        l[t, 9:11] = [-1.0, 2.0]
    for t in range(2, T, 9):
        l[t] = 0.0
        l[t, ::2] = -0.0
    for t in range(4, T, 11):
        l[t, [3, 48]] = np.inf
    L, L64 = _to(l, dtype)
    for renormalize in (True, False):
        _check_route(g.gptq_moe_route(L, k, renormalize=renormalize), L64, k, renormalize)


def test_all_tokens_on_one_expert(g):
    rng = _rng(64, 9)
    l = rng.standard_normal((64, 9))
    l[:, 4] = 50.0
    L, L64 = _to(l, "f32")
    _check_route(g.gptq_moe_route(L, 1), L64, 1, True)
    assert oracle.moe_route(L64, 1, True)[2].tolist() == [0] * 5 + [64] * 5
