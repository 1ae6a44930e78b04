"""The statistics of sharq_norm_residual's norms are those of sharq_rmsnorm, to the bit."""
import numpy as np
import pytest
import torch

from tests.gpu_common import require_gpu
from tests.kv_common import bf16

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,k", [(2000, 4096), (200, 4096), (1500, 5120), (400, 32768), (100, 1280), (3000, 256)])
@pytest.mark.parametrize("spread", [0.0, 3.0])
def test_same_bits_as_the_rmsnorm_call(tokens, k, spread):
    """Both take the square sums in float64, whose rounding (2^-53 of the sum a step) reaches the float32
    mean in one row of 2^20 or so: none of these. A sum off by 4e-7 shows in most cases."""
    S = require_gpu()
    rng = np.random.default_rng(tokens + k)
    x, _ = bf16(rng, tokens, k)
    if spread:  # magnitudes from row to row and within a row
        x = (x.float() * torch.from_numpy(np.exp(spread * rng.standard_normal((tokens, k))).astype(np.float32)).cuda()).bfloat16()
    g, _ = bf16(rng, k)
    zero = torch.zeros_like(x)
    want = S.sharq_rmsnorm(x, g)
    r, h = S.sharq_norm_residual(zero, x, pre_gamma=g)
    assert torch.equal(r, x) and torch.equal(h, want)
    r, _ = S.sharq_norm_residual(x, zero, post_gamma=g)
    assert torch.equal(r, want)


@pytest.mark.parametrize("tokens", [3, 700])
def test_not_a_number_infinity_and_zero(tokens):
    S = require_gpu()
    rng = np.random.default_rng(tokens)
    x, _ = bf16(rng, tokens, 1024)
    x[0], x[1, 5], x[2, 1000] = 0, float("inf"), float("nan")
    g, _ = bf16(rng, 1024)
    want = S.sharq_rmsnorm(x, g)
    _, h = S.sharq_norm_residual(torch.zeros_like(x), x, pre_gamma=g)
    assert torch.equal(torch.isnan(h), torch.isnan(want)) and torch.equal(torch.nan_to_num(h), torch.nan_to_num(want))
    assert torch.isnan(h[2]).all() and not h[0].any()
