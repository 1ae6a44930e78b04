"""Query elements far below their row's largest, in every form of the attention."""
import numpy as np
import pytest
import torch

from oracle import kv as K
from tests.gpu_common import require_gpu
from tests.kv_common import BF16, Setup, bf16

pytestmark = pytest.mark.gpu

NEW = [1, 6, 14, 40, 200]  # two query heads per key head: 2, 12, 28 rows, one row tile, two


@pytest.mark.parametrize("new", NEW)
def test_queries_of_many_magnitudes_in_one_row(new):
    """An element 2^-n of its row's largest is exact up to n = 29, rounded by at most 2^-37 of the largest
    below that. Keys that are zero in the row's large elements make the small ones count."""
    S = require_gpu()
    rng = np.random.default_rng(new)
    st = Setup(S, rng, [64], 2, 64, "nvfp4", 16)
    qkv, _ = bf16(rng, 64, 6 * 64)
    kv = qkv.view(64, 6, 64)
    kv[:, 2:4, :16] = 0
    S.sharq_kv_append(qkv, st.cache, st.batch([64]), 2)
    batch = st.batch([new])
    k, v = st.kv(0, 64)
    for n in (20, 29, 33):
        q, _ = bf16(rng, new, 4, 64)
        q[..., 16:] *= 2.0 ** -n
        q[..., 0] = 1.0 + 127 / 128  # the largest, with every bit of its significand
        q[..., 1:16] = 0
        scale = 2.0 ** n * 64 ** -0.5
        y, lse = S.sharq_attention(q, st.cache, batch, causal=False, scale=scale, return_lse=True)
        x = q.double().cpu().numpy()
        ry, rl, mass, flat, dots = K.attention(x, k, v, 0, False, 0, scale)
        # each of the 48 small elements may be off by 2^-37 of the largest (below 2): 2^-36 |k| scale
        lost = 2.0 ** -36 * np.abs(k).sum(-1).max() * scale
        ds = dots * 2.0 ** -16 + 2.0 ** -20 + lost
        got = y.double().cpu().numpy()
        tol = np.abs(ry) * BF16 + mass * (2.0 ** -11 + 2 * ds[..., None]) + flat * 2.0 ** -25 + 1e-30
        assert (np.abs(got - ry) <= tol).all(), (n, (np.abs(got - ry) / tol).max())
        assert (np.abs(lse.double().cpu().numpy() - rl) <= ds + np.abs(rl) * 2.0 ** -22 + 2.0 ** -18).all()
