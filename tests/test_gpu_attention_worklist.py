"""Batches whose longest sequence, or the bound on it, is far above the others'."""
import numpy as np
import pytest
import torch

from oracle import kv as K
from tests.gpu_common import require_gpu
from tests.kv_common import Setup, bf16, check_attention

pytestmark = pytest.mark.gpu


def test_a_loose_bound_on_the_rows_costs_no_wait():
    """300 single tokens under a bound of 2^18 rows (the call's tensors are that long, the rest is padding).
    The block that walks from one sequence to the next keeps its other warps waiting meanwhile: that
    has to stay far below 100 us, whatever the bound."""
    S = require_gpu()
    rng = np.random.default_rng(5)
    lengths = rng.integers(1, 200, 300).tolist()
    st = Setup(S, rng, lengths, 1, 64, "nvfp4", 16).fill()
    tokens = 1 << 18
    q = torch.zeros(tokens, 4, 64, dtype=torch.bfloat16, device="cuda")
    q[:300], x = bf16(rng, 300, 4, 64)
    batch = st.batch([1] * 300, tokens=tokens, max_q=tokens)
    y = torch.full_like(q, 3.0)
    lse = torch.full((tokens, 4), 9.0, device="cuda")
    ws = S.alloc_attention_workspace(st.cache, batch, 4)
    assert S.sharq_device_status() == S.SHARQ_OK
    try:
        S.sharq_set_wait_limit(100_000)
        S.sharq_attention(q, st.cache, batch, y=y, lse=lse, workspace=ws)
        assert S.sharq_device_status() == S.SHARQ_OK
    finally:
        S.sharq_set_wait_limit(0)
    assert (y[300:] == 3).all() and (lse[300:] == 9).all()
    for b, n in enumerate(lengths):
        k, v = st.kv(b, n)
        check_attention(y[b:b + 1], lse[b:b + 1], K.attention(x[b:b + 1], k, v, n - 1, True, 0, 0.125), f"sequence {b}")


@pytest.mark.parametrize("group,long", [(4, 3000), (1, 2600), (7, 700)])
def test_one_long_prompt_among_single_tokens(group, long):
    """More row tiles times sequences than threads, empty sequences and sequences of every remainder of
    a row tile between them."""
    S = require_gpu()
    rng = np.random.default_rng(long)
    new = [1, 0, 0, 255, 256, 257, 0, 1, 64, 65] + [0, 1, 3] * 30 + [long] + [1] * 40 + [0] * 70 + [511, 512, 513, 1]
    lengths = [n + int(rng.integers(0, 90)) for n in new]
    st = Setup(S, rng, lengths, 1, 64, "mxfp4", 16).fill()
    q, x = bf16(rng, sum(new), group, 64)
    y, lse = S.sharq_attention(q, st.cache, st.batch(new), return_lse=True)
    at = 0
    for b, m in enumerate(new):
        if m:
            k, v = st.kv(b, lengths[b])
            check_attention(y[at:at + m], lse[at:at + m], K.attention(x[at:at + m], k, v, lengths[b] - m, True, 0, 0.125), f"sequence {b}")
        at += m


def test_more_sequences_times_row_tiles_than_an_index_holds():
    """2^20 sequences, all but three of them empty, under a bound of 2^20 rows."""
    S = require_gpu()
    rng = np.random.default_rng(6)
    n, where = 1 << 20, [0, 400_000, (1 << 20) - 1]
    new = np.zeros(n, np.int64)
    new[where] = [300, 1, 700]
    length = np.zeros(n, np.int64)
    length[where] = [340, 60, 700]
    small = Setup(S, rng, [340, 60, 700], 1, 64, "nvfp4", 1024).fill()
    table = np.full((n, 1), -1, np.int32)
    table[where] = small.table
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    q = torch.zeros(n, 1, 64, dtype=torch.bfloat16, device="cuda")
    q[:1001], x = bf16(rng, 1001, 1, 64)
    batch = S.KVBatch(i32(np.concatenate(([0], np.cumsum(new)))), i32(length), i32(table), n, n)
    y, lse = S.sharq_attention(q, small.cache, batch, return_lse=True)
    assert S.sharq_device_status() == S.SHARQ_OK
    at = 0
    for b, (m, c) in enumerate(zip((300, 1, 700), (340, 60, 700))):
        k, v = small.kv(b, c)
        check_attention(y[at:at + m], lse[at:at + m], K.attention(x[at:at + m], k, v, c - m, True, 0, 0.125), f"sequence {b}")
        at += m


@pytest.mark.parametrize("count,first", [(3, 100), (300, 700)])
def test_index_arrays_that_run_past_the_tensors(count, first):
    """Rows behind the call's tensors are left out, the others and the workspace stay right."""
    S = require_gpu()
    rng = np.random.default_rng(count)
    new = [first] + [60] * 2 + [1] * (count - 3)
    lengths = [n + 20 for n in new]
    st = Setup(S, rng, lengths, 1, 64, "nvfp4", 32).fill()
    tokens = first + 90
    q, x = bf16(rng, tokens, 4, 64)
    cut, full = st.batch(new, tokens=tokens), st.batch(new)
    ws = S.alloc_attention_workspace(st.cache, full, 4)
    y, lse = S.sharq_attention(q, st.cache, cut, return_lse=True, workspace=ws)
    for b, rows in ((0, first), (1, 60), (2, 30)):
        at = sum(new[:b])
        k, v = st.kv(b, lengths[b])
        check_attention(y[at:at + rows], lse[at:at + rows], K.attention(x[at:at + rows], k, v, 20, True, 0, 0.125), f"sequence {b}")
    all_q = torch.zeros(sum(new), 4, 64, dtype=torch.bfloat16, device="cuda")
    all_q[:tokens] = q
    y2, lse2 = S.sharq_attention(all_q, st.cache, full, return_lse=True, workspace=ws)
    for b in range(count):
        at = sum(new[:b])
        k, v = st.kv(b, lengths[b])
        rows = slice(at, at + new[b])
        check_attention(y2[rows], lse2[rows], K.attention(all_q[rows].double().cpu().numpy(), k, v, 20, True, 0, 0.125), f"sequence {b}")
