"""Rows of the cache that no query sees may hold anything, in every form of the attention."""
import numpy as np
import pytest
import torch

from oracle import kv as K
from tests.gpu_common import require_gpu
from tests.kv_common import Setup, bf16, check_attention

pytestmark = pytest.mark.gpu

NEW = [1, 6, 14, 40, 200]  # two query heads per key head: 2, 12, 28 rows, one row tile, two


@pytest.mark.parametrize("new", NEW)
@pytest.mark.parametrize("window", [1, 30, 77, 300])
@pytest.mark.parametrize("fmt,d", [("nvfp4", 64), ("nvfp4", 128), ("mxfp4", 64), ("mxfp4", 128)])
def test_bytes_ahead_of_a_window_do_not_matter(new, window, fmt, d):
    """Only what the window reaches was ever written (the tail of an imported prefix); the rest of its
    pages holds NaN scales."""
    S = require_gpu()
    rng = np.random.default_rng(new + window)
    lengths = [901 + new, 640 + new]
    st = Setup(S, rng, lengths, 2, d, fmt, 64)
    st.cache.pages.fill_(0xFF)
    seen = [min(n, window - 1 + new) for n in lengths]
    qkv, _ = bf16(rng, sum(seen), 6 * d)
    S.sharq_kv_append(qkv, st.cache, st.batch(seen), 2)
    q, x = bf16(rng, 2 * new, 4, d)
    y, lse = S.sharq_attention(q, st.cache, st.batch([new, new]), window=window, return_lse=True)
    for b, n in enumerate(lengths):
        k, v = st.kv(b, n)
        k[: n - seen[b]] = v[: n - seen[b]] = 0  # behind the mask
        rows = slice(b * new, (b + 1) * new)
        check_attention(y[rows], lse[rows], K.attention(x[rows], k, v, n - new, True, window, d ** -0.5), f"sequence {b}")
