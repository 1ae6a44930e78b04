"""The decode kernel's bounded wait reports that it gave up, and the next call is right. It waits for a
warp's copies of 32 keys, issued at most one such tile before: from DRAM they are not there at once. (Up to
16 query rows, 40 of 40 calls whose cache had left the L2 reported it; the 17-row form works so long on a
tile that only some do, so that it is no case here.)"""
import numpy as np
import pytest
import torch

from oracle import kv as K
from tests.gpu_common import require_gpu
from tests.kv_common import Setup, bf16, check_attention

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new,group", [(1, 4), (3, 4), (2, 8)])
def test_timeout_is_reported_and_the_next_call_is_right(new, group):
    S = require_gpu()
    rng = np.random.default_rng(new)
    lengths = [30000, 20000]
    st = Setup(S, rng, lengths, 2, 128, "nvfp4", 16).fill()
    q, x = bf16(rng, 2 * new, 2 * group, 128)
    batch = st.batch([new, new])
    ws = S.alloc_attention_workspace(st.cache, batch, 2 * group)
    torch.zeros(1 << 28, dtype=torch.uint8, device="cuda").add_(1)  # the cache leaves the L2
    assert S.sharq_device_status() == S.SHARQ_OK
    try:
        S.sharq_set_wait_limit(1)
        S.sharq_attention(q, st.cache, batch, workspace=ws)
        assert S.sharq_device_status() == S.SHARQ_ERR_TIMEOUT
    finally:
        S.sharq_set_wait_limit(0)
    ws.zero_()
    y, lse = S.sharq_attention(q, st.cache, batch, return_lse=True, workspace=ws)
    assert S.sharq_device_status() == S.SHARQ_OK
    for b in range(2):
        k, v = st.kv(b, lengths[b])
        rows = slice(b * new, (b + 1) * new)
        check_attention(y[rows], lse[rows], K.attention(x[rows], k, v, lengths[b] - new, True, 0, 128 ** -0.5))
