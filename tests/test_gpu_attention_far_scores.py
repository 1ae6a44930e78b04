"""Scores far beyond the range in which float32 resolves their exponents, in every form of the attention."""
import numpy as np
import pytest
import torch

from oracle import kv as K
from tests.gpu_common import require_gpu
from tests.kv_common import BF16, Setup, bf16, check_attention

pytestmark = pytest.mark.gpu

NEW = [1, 6, 14, 40, 200]  # two query heads per key head: 2, 12, 28 rows, one row tile, two


@pytest.mark.parametrize("new", NEW)
@pytest.mark.parametrize("size,scale", [(1e8, None), (3e9, None), (1e10, -0.3), (1e20, None), (1e30, None)])
def test_scores_beyond_the_float32_steps_of_an_exponent(new, size, scale):
    """Scores so large that neighbouring float32 values lie many powers of two apart: the largest takes
    everything. Scores are off by at most 2^-16 of `dots` (128 float32 sums of exact products, 2^-17, and
    the factor's rounding), so where the second is farther behind than twice that, y is the first's value
    (products by a weight of one and by 1/l = 1 at most: bf16's half step and two of float32)."""
    S = require_gpu()
    rng = np.random.default_rng(new)
    st = Setup(S, rng, [700], 2, 128, "nvfp4", 16).fill(4.0)
    q, x = bf16(rng, new, 4, 128, scale=size)
    y, lse = S.sharq_attention(q, st.cache, st.batch([new]), scale=scale, return_lse=True)
    k, v = st.kv(0, 700)
    f = 128 ** -0.5 if scale is None else scale
    checked = 0
    for i in range(new):
        for h in range(4):
            n = 700 - new + i + 1
            s = k[:n, h // 2] @ x[i, h] * f
            dots = (np.abs(k[:n, h // 2]) @ np.abs(x[i, h])).max() * abs(f)
            first, second = np.argsort(s)[:-3:-1]
            out, l = y[i, h].double().cpu().numpy(), float(lse[i, h])
            assert np.isfinite(out).all() and abs(l - s[first]) <= dots * 2.0 ** -16 + abs(s[first]) * 2.0 ** -22
            if s[first] - s[second] > dots * 2.0 ** -15:
                want = v[first, h // 2]
                assert (np.abs(out - want) <= np.abs(want) * (BF16 + 2.0 ** -22)).all(), (i, h)
                checked += 1
    assert checked > 2 * new


@pytest.mark.parametrize("new", NEW)
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_one_row_with_far_scores_leaves_the_others_right(new, fmt):
    S = require_gpu()
    rng = np.random.default_rng(new)
    st = Setup(S, rng, [300], 2, 64, fmt, 16).fill()
    q, _ = bf16(rng, new, 4, 64)
    q[0, 1] *= 2.0 ** 40
    y, lse = S.sharq_attention(q, st.cache, st.batch([new]), return_lse=True)
    k, v = st.kv(0, 300)
    check_attention(y, lse, K.attention(q.double().cpu().numpy(), k, v, 300 - new, True, 0, 0.125))
