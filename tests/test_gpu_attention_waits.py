"""The prompt kernel's bounded waits give up, report a status that the host reads, and leave the
context usable; no data is lost by it but the call's own output. (The decode kernel waits only for
copies issued two tiles before, which are there when it asks: its wait cannot be made to expire.)"""
import numpy as np
import pytest
import torch

from oracle import kv as K
from tests.gpu_common import require_gpu
from tests.kv_common import Setup, bf16, check_attention

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new", [40, 700])
def test_timeout_is_reported_and_the_next_call_is_right(new):
    S = require_gpu()
    rng = np.random.default_rng(new)
    lengths = [4000, 3000]
    st = Setup(S, rng, lengths, 2, 128, "nvfp4", 16).fill()
    q, x = bf16(rng, 2 * new, 8, 128)
    batch = st.batch([new, new])
    ws = S.alloc_attention_workspace(st.cache, batch, 8)
    assert S.sharq_device_status() == S.SHARQ_OK
    try:
        S.sharq_set_wait_limit(1)
        S.sharq_attention(q, st.cache, batch, workspace=ws)
        assert S.sharq_device_status() == S.SHARQ_ERR_TIMEOUT
    finally:
        S.sharq_set_wait_limit(0)
    ws.zero_()  # a call that gave up may leave its counters behind
    y, lse = S.sharq_attention(q, st.cache, batch, return_lse=True, workspace=ws)
    assert S.sharq_device_status() == S.SHARQ_OK
    for b in range(2):
        k, v = st.kv(b, lengths[b])
        rows = slice(b * new, (b + 1) * new)
        check_attention(y[rows], lse[rows], K.attention(x[rows], k, v, lengths[b] - new, True, 0, 128 ** -0.5))


def test_timeout_with_one_row_tile():
    """The two tiles of a block share the rows here, and one hands its sums to the other."""
    test_timeout_is_reported_and_the_next_call_is_right(20)
