"""Windows of up to 2^31 - 1 positions, in every form of the attention."""
import numpy as np
import pytest
import torch

from tests.gpu_common import require_gpu
from tests.kv_common import Setup, bf16

pytestmark = pytest.mark.gpu

NEW = [1, 6, 14, 40, 200]  # two query heads per key head: 2, 12, 28 rows, one row tile, two


@pytest.mark.parametrize("new", NEW)
@pytest.mark.parametrize("window", [1 << 30, 2 ** 31 - 300, 2 ** 31 - 4, 2 ** 31 - 1])
def test_a_window_longer_than_every_context_hides_nothing(new, window):
    """Also where a sequence has fewer cached than new tokens, so that positions begin below zero."""
    S = require_gpu()
    rng = np.random.default_rng(new)
    st = Setup(S, rng, [new + 50] * 3, 2, 128, "nvfp4", 16).fill()
    q, _ = bf16(rng, 3 * new, 4, 128)
    batch = st.batch([new] * 3, [new + 50, max(1, new - 5), (new + 1) // 2])
    y, lse = S.sharq_attention(q, st.cache, batch, return_lse=True)
    y2, lse2 = S.sharq_attention(q, st.cache, batch, window=window, return_lse=True)
    assert torch.equal(y, y2) and torch.equal(lse, lse2)
    assert torch.isfinite(lse[3 * new - 1]).all()
