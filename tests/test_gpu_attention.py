"""Attention over the paged FP4 cache against the oracle's float64."""
import math

import numpy as np
import pytest
import torch

from oracle import kv as K
from tests.gpu_common import require_gpu
from tests.kv_common import Setup, bf16, check_attention

pytestmark = pytest.mark.gpu


def run(S, st, new, group, causal=True, window=0, scale=None, q_mul=1.0, lengths=None, workspace=None):
    """Runs one call and checks every row."""
    lengths = st.lengths if lengths is None else lengths
    hq = group * st.heads
    q, x = bf16(st.rng, sum(new), hq, st.d, scale=q_mul)
    y, lse = S.sharq_attention(q, st.cache, st.batch(new, lengths), causal, window, scale, return_lse=True, workspace=workspace)
    check_rows(S, st, x, y, lse, new, lengths, causal, window, scale)
    return q, y, lse


def check_rows(S, st, x, y, lse, new, lengths, causal=True, window=0, scale=None):
    at = 0
    for b, m in enumerate(new):
        k, v = st.kv(b, lengths[b])
        ref = K.attention(x[at:at + m], k, v, lengths[b] - m, causal, window, st.d ** -0.5 if scale is None else scale)
        check_attention(y[at:at + m], lse[at:at + m], ref, f"sequence {b}")
        at += m


LENGTHS = [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129, 255, 257, 777, 1500]


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("d,heads,group,page", [(128, 8, 4, 16), (64, 2, 1, 32), (128, 1, 7, 64), (64, 4, 8, 128), (128, 2, 16, 16)])
def test_single_tokens(fmt, d, heads, group, page):
    S = require_gpu()
    st = Setup(S, np.random.default_rng(d + heads), LENGTHS, heads, d, fmt, page).fill(2.0)
    run(S, st, [1] * len(LENGTHS), group)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("d,heads,group,page,new", [
    (128, 4, 7, 32, 5), (64, 2, 4, 16, 3), (128, 2, 1, 64, 17), (64, 1, 8, 16, 40), (128, 1, 12, 128, 11)])
def test_several_tokens(fmt, d, heads, group, page, new):
    S = require_gpu()
    rng = np.random.default_rng(new)
    lengths = [new, new + 1, 100, 301, 1111]
    st = Setup(S, rng, lengths, heads, d, fmt, page).fill()
    run(S, st, [new, 1, 0, new, max(1, new // 2)], group)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("d,heads,group,lengths,new", [
    (128, 2, 4, [300, 70], [300, 65]), (64, 3, 1, [513, 1], [513, 1]), (128, 1, 5, [900, 257], [129, 257]),
    (64, 1, 8, [1030], [77]), (128, 2, 1, [256, 128, 2], [256, 128, 2])])
def test_prompts(fmt, d, heads, group, lengths, new):
    S = require_gpu()
    st = Setup(S, np.random.default_rng(sum(new)), lengths, heads, d, fmt, 32).fill()
    run(S, st, new, group)
    run(S, st, new, group, window=50)
    run(S, st, new, group, causal=False)


@pytest.mark.parametrize("window", [1, 2, 31, 32, 33, 200, 100000])
@pytest.mark.parametrize("new", [1, 6, 150])
def test_windows(window, new):
    S = require_gpu()
    lengths = [new, new + 5, 400 + new, 1000]
    st = Setup(S, np.random.default_rng(window), lengths, 2, 128, "nvfp4", 16).fill()
    run(S, st, [new] * 4, 4, window=window)


def test_causal_order_is_by_position():
    """Keys behind a query do not reach it: changing them changes nothing before them."""
    S = require_gpu()
    rng = np.random.default_rng(8)
    for new in (4, 140):
        st = Setup(S, rng, [300], 2, 128, "mxfp4", 16).fill()
        q, y, lse = run(S, st, [new], 2)
        half = new // 2
        qkv, _ = bf16(rng, new - half, 6 * 128, scale=30.0)
        S.sharq_kv_append(qkv, st.cache, st.batch([new - half]), 2)
        y2, lse2 = S.sharq_attention(q, st.cache, st.batch([new]), return_lse=True)
        assert torch.equal(y[:half], y2[:half]) and torch.equal(lse[:half], lse2[:half])
        assert not torch.equal(y[half:], y2[half:])


@pytest.mark.parametrize("new", [1, 5, 140])
def test_rows_that_see_nothing(new):
    """No cached token, positions before the start, pages that are not there: y = 0, lse = -inf; and
    what stands in the bytes that nobody may see (NaN scales among it) does not matter."""
    S = require_gpu()
    rng = np.random.default_rng(new)
    lengths = [new + 90, new + 50, new + 3]
    for fmt in ("nvfp4", "mxfp4"):
        st = Setup(S, rng, lengths, 2, 64, fmt, 16)
        st.cache.pages.fill_(0xFF)  # NaN block scales wherever nothing is appended
        st.fill()
        q, x = bf16(rng, 3 * new, 4, 64)
        hole = st.table.copy()
        hole[1, :] = -1
        lens = [new + 90, new + 50, max(0, new - 2)]
        y, lse = S.sharq_attention(q, st.cache, st.batch([new] * 3, lens, table=hole), return_lse=True)
        assert not y[new:2 * new].any() and torch.isneginf(lse[new:2 * new]).all()
        k, v = st.kv(0, lens[0])
        check_attention(y[:new], lse[:new], K.attention(x[:new], k, v, lens[0] - new, True, 0, 64 ** -0.5))
        k, v = st.kv(2, lens[2])
        check_attention(y[2 * new:], lse[2 * new:], K.attention(x[2 * new:], k, v, lens[2] - new, True, 0, 64 ** -0.5))


def test_a_hole_in_the_table_is_skipped():
    S = require_gpu()
    rng = np.random.default_rng(2)
    for new in (1, 100):
        st = Setup(S, rng, [200], 2, 128, "nvfp4", 16).fill()
        table = st.table.copy()
        table[0, 3], table[0, 7] = -1, st.num_pages
        q, x = bf16(rng, new, 4, 128)
        y, lse = S.sharq_attention(q, st.cache, st.batch([new], table=table), return_lse=True)
        k, v = st.kv(0, 200)
        place = ~np.isin(np.arange(200) // 16, (3, 7))
        check_attention(y, lse, K.attention(x, k, v, 200 - new, True, 0, 128 ** -0.5, place))


@pytest.mark.parametrize("new", [1, 7, 130])
def test_padding_rows_and_strided_queries(new):
    S = require_gpu()
    rng = np.random.default_rng(new)
    st = Setup(S, rng, [300, 250, new], 2, 128, "mxfp4", 64).fill()
    total = 2 * new + 5
    wide, _ = bf16(rng, total, 9, 128)
    q = wide[:, 1:7]
    y = torch.full((total, 6, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((total, 6), 9.0, device="cuda")
    out = S.sharq_attention(q, st.cache, st.batch([new, new, 0], tokens=total), y=y, lse=lse)
    assert out[0] is y and out[1] is lse
    assert (y[2 * new:] == 3).all() and (lse[2 * new:] == 9).all()
    check_rows(S, st, q.double().cpu().numpy(), y, lse, [new, new, 0], st.lengths)
    only = S.sharq_attention(q, st.cache, st.batch([new, new, 0], tokens=total))
    assert torch.equal(only[: 2 * new], y[: 2 * new])


@pytest.mark.parametrize("new", [1, 6, 200])
def test_extreme_scores(new):
    """Scores far apart (one key takes everything), tiny and huge queries, a negative scale."""
    S = require_gpu()
    rng = np.random.default_rng(new)
    st = Setup(S, rng, [700], 2, 128, "nvfp4", 16).fill(4.0)
    run(S, st, [new], 2, q_mul=40.0)
    run(S, st, [new], 2, q_mul=1e-20)
    run(S, st, [new], 2, q_mul=1e10, scale=1e-11)
    run(S, st, [new], 2, scale=-0.3)
    run(S, st, [new], 2, scale=0.0)


@pytest.mark.parametrize("new", [1, 6, 140])
def test_nan_stays_in_its_row(new):
    S = require_gpu()
    rng = np.random.default_rng(new)
    st = Setup(S, rng, [300], 2, 128, "nvfp4", 16).fill()
    q, x = bf16(rng, new, 4, 128)
    q[0, 1, 5] = float("nan")
    y, lse = S.sharq_attention(q, st.cache, st.batch([new]), return_lse=True)
    assert torch.isnan(y[0, 1]).all() and torch.isnan(lse[0, 1])
    good = torch.ones(new, 4, dtype=torch.bool, device="cuda")
    good[0, 1] = False
    k, v = st.kv(0, 300)
    ref = K.attention(np.nan_to_num(q.double().cpu().numpy()), k, v, 300 - new, True, 0, 128 ** -0.5)
    y[0, 1], lse[0, 1] = 0, 0
    g = good.cpu().numpy()
    pick = [torch.where(good[..., None], y, 0), torch.where(good, lse, 0)]
    check_attention(pick[0], pick[1], [np.where(g[..., None] if a.ndim == 3 else g, a, 0) for a in ref])


def test_many_sequences_of_uneven_length():
    """More work items than blocks at once, most of them short, one long."""
    S = require_gpu()
    rng = np.random.default_rng(11)
    lengths = rng.integers(0, 90, 300).tolist()
    lengths[17] = 6000
    st = Setup(S, rng, lengths, 2, 64, "mxfp4", 16).fill()
    new = [min(n, 1) for n in lengths]
    run(S, st, new, 2)


# 33 to 128 query rows of a key head: two tiles of a block share them, each with every second step of
# 128 keys, so the number of steps, and which one an item or a cut begins with, matter
@pytest.mark.parametrize("fmt,d", [("nvfp4", 128), ("mxfp4", 64)])
@pytest.mark.parametrize("group,new", [(1, 33), (7, 5), (4, 32), (16, 8), (40, 3), (128, 1)])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 100), (True, 300), (False, 0)])
def test_one_row_tile(fmt, d, group, new, causal, window):
    S = require_gpu()
    lengths = [new, 127 + new, 128 + new, 129 + new, 256 + new, 257 + new, 384 + new, 513 + new, 1700, 5]
    news = [new] * 9 + [min(new, 5)]
    st = Setup(S, np.random.default_rng(group + new), lengths, 2, d, fmt, 32).fill()
    run(S, st, news, group, causal=causal, window=window)


@pytest.mark.parametrize("lengths", [[128 * 300 + 77], [128 * 150 + 1, 40], [60, 128 * 149]])
def test_one_row_tile_cut_between_blocks(lengths):
    S = require_gpu()
    st = Setup(S, np.random.default_rng(3), lengths, 1, 128, "nvfp4", 64).fill()
    run(S, st, [9] * len(lengths), 8)
    run(S, st, [9] * len(lengths), 8, q_mul=30.0)


@pytest.mark.parametrize("group,new,length", [(1, 1, 60011), (4, 1, 9999), (12, 1, 50000), (32, 1, 40000), (7, 5, 50000),
                                              (40, 5, 30000), (4, 3, 2700)])
@pytest.mark.parametrize("heads,d,fmt", [(1, 128, "nvfp4"), (2, 64, "mxfp4")])
def test_items_of_many_parts(group, new, length, heads, d, fmt):
    """One context over all blocks: up to hundreds of parts, joined in two levels; then the same call
    again, with the counters as the first one left them."""
    S = require_gpu()
    st = Setup(S, np.random.default_rng(group), [length], heads, d, fmt, 64).fill()
    ws = S.alloc_attention_workspace(st.cache, st.batch([new]), group * heads)
    q, y, lse = run(S, st, [new], group, workspace=ws)
    y2, lse2 = S.sharq_attention(q, st.cache, st.batch([new]), return_lse=True, workspace=ws)
    assert torch.equal(y, y2) and torch.equal(lse, lse2)


def test_one_row_tile_with_a_row_that_is_not_a_number():
    """Its row alone; and where only one of the two tiles sees keys."""
    S = require_gpu()
    rng = np.random.default_rng(11)
    for length, window in ((100, 0), (400, 0), (400, 60)):
        st = Setup(S, rng, [length], 2, 128, "nvfp4", 16).fill()
        q, x = bf16(rng, 20, 8, 128)
        q[3, 5, 7] = float("nan")
        y, lse = S.sharq_attention(q, st.cache, st.batch([20]), window=window, return_lse=True)
        assert torch.isnan(y[3, 5]).all() and torch.isnan(lse[3, 5])
        k, v = st.kv(0, length)
        ref = K.attention(np.nan_to_num(q.double().cpu().numpy()), k, v, length - 20, True, window, 128 ** -0.5)
        for got, want in ((y, 0), (lse, 1)):
            got[3, 5] = torch.as_tensor(ref[want][3, 5]).to(got)
        check_attention(y, lse, ref)


def test_one_row_tile_across_missing_pages():
    S = require_gpu()
    rng = np.random.default_rng(12)
    st = Setup(S, rng, [700, 300], 2, 64, "mxfp4", 16).fill()
    table = st.table.copy()
    table[0, 8:16] = -1   # the second step of 128 keys and some of the others
    table[0, 20] = table[1, 0] = st.num_pages
    q, x = bf16(rng, 50, 4, 64)
    y, lse = S.sharq_attention(q, st.cache, st.batch([25, 25], table=table), return_lse=True)
    for b, (length, gone) in enumerate(((700, [*range(8, 16), 20]), (300, [0]))):
        k, v = st.kv(b, length)
        place = ~np.isin(np.arange(length) // 16, gone)
        rows = slice(25 * b, 25 * b + 25)
        check_attention(y[rows], lse[rows], K.attention(x[rows], k, v, length - 25, True, 0, 64 ** -0.5, place))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", [1, 3, 70])
def test_buffers_at_their_least_alignment(new, d):
    """Every buffer 16 bytes (lse and indexes 4) off a round address."""
    S = require_gpu()
    rng = np.random.default_rng(19)
    st = Setup(S, rng, [200, 150], 2, d, "nvfp4", 16).fill()

    def off(t, by):
        n = by // t.element_size()
        out = torch.zeros(t.numel() + 2 * n, dtype=t.dtype, device="cuda")[n:n + t.numel()].view(t.shape)
        out.copy_(t)
        assert out.data_ptr() % (2 * by) == by
        return out

    cache = S.KVCache(off(st.cache.pages, 16), st.num_pages, 16, 2, d, "nvfp4", off(st.cache.k_scale, 4), off(st.cache.v_scale, 4))
    q, x = bf16(rng, 2 * new, 8, d)
    q = off(q, 16)
    y, lse = off(torch.zeros_like(q), 16), off(torch.zeros(2 * new, 8, device="cuda"), 4)
    b = st.batch([new, new])
    batch = S.KVBatch(off(b.cu_q, 4), off(b.kv_len, 4), off(b.page_table, 4), new, 2 * new)
    ws = S.alloc_attention_workspace(cache, batch, 8)
    S.sharq_attention(q, cache, batch, y=y, lse=lse, workspace=off(ws, 16))
    check_rows(S, st, x, y, lse, [new, new], st.lengths)
    k, v = S.sharq_kv_read(cache, batch, off(torch.zeros(2 * new, 2, d, device="cuda"), 16),
                           off(torch.zeros(2 * new, 2, d, device="cuda"), 16))
    k2, v2 = S.sharq_kv_read(st.cache, b, out_dtype=torch.float32)
    assert torch.equal(k, k2) and torch.equal(v, v2)


def test_more_entries_than_threads():
    """Many sequences of several row tiles each, uneven and some empty."""
    S = require_gpu()
    rng = np.random.default_rng(13)
    lengths = rng.integers(0, 140, 260).tolist()
    lengths[3], lengths[200] = 700, 1500
    new = [int(min(n, rng.integers(0, 140))) for n in lengths]
    st = Setup(S, rng, lengths, 1, 64, "nvfp4", 16).fill()
    run(S, st, new, 4)


@pytest.mark.parametrize("group,new", [(40, 1), (128, 1), (128, 3), (33, 8)])
def test_large_groups(group, new):
    S = require_gpu()
    st = Setup(S, np.random.default_rng(group), [200, 5, 900], 1, 64, "mxfp4", 32).fill()
    run(S, st, [new, min(new, 5), new], group)


@pytest.mark.parametrize("new", [1, 90])
def test_nothing_but_padding_and_nothing_cached(new):
    S = require_gpu()
    rng = np.random.default_rng(6)
    st = Setup(S, rng, [50, 40], 2, 128, "nvfp4", 16).fill()
    q, x = bf16(rng, new, 4, 128)
    y = torch.full((new, 4, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((new, 4), 9.0, device="cuda")
    S.sharq_attention(q, st.cache, st.batch([0, 0], tokens=new, max_q=new), y=y, lse=lse)
    assert (y == 3).all() and (lse == 9).all()
    S.sharq_attention(q, st.cache, st.batch([new, 0], [0, 0]), causal=False, y=y, lse=lse)
    assert not y.any() and torch.isneginf(lse).all()


@pytest.mark.parametrize("new", [1, 60])
def test_on_a_stream_of_its_own(new):
    """A call given a stream orders its workspace and outputs there, behind that stream's work."""
    S = require_gpu()
    rng = np.random.default_rng(17)
    st = Setup(S, rng, [1200, 900], 2, 128, "nvfp4", 16).fill()
    q, x = bf16(rng, 2 * new, 8, 128)
    batch = st.batch([new, new])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    late = torch.zeros_like(q)
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # about ten milliseconds
        late.copy_(q)
    for handle in (side, side.cuda_stream):
        y, lse = S.sharq_attention(late, st.cache, batch, return_lse=True, stream=handle)
        side.synchronize()
        check_rows(S, st, x, y, lse, [new, new], st.lengths)


@pytest.mark.parametrize("new", [1, 4, 300])
def test_same_inputs_same_bits(new):
    S = require_gpu()
    rng = np.random.default_rng(new)
    st = Setup(S, rng, [5000, 900], 4, 128, "nvfp4", 16).fill()
    q, _ = bf16(rng, 2 * new, 16, 128)
    batch = st.batch([new, new])
    ws = S.alloc_attention_workspace(st.cache, batch, 16)
    first = S.sharq_attention(q, st.cache, batch, return_lse=True, workspace=ws)
    for _ in range(5):
        again = S.sharq_attention(q, st.cache, batch, return_lse=True, workspace=ws)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_one_workspace_serves_calls_of_several_shapes():
    S = require_gpu()
    rng = np.random.default_rng(21)
    st = Setup(S, rng, [3000, 64, 700], 4, 128, "nvfp4", 16).fill()
    plans = [([1, 1, 1], 4), ([200, 64, 130], 8), ([5, 0, 3], 2), ([1, 0, 0], 1)]
    size = max(S.sharq_attention_workspace_size(st.cache, st.batch(n), g * 4) for n, g in plans)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        for new, group in plans:
            run(S, st, new, group, workspace=ws)


def test_captured_calls_follow_the_batch_and_share_no_state():
    """Two captured graphs with a workspace each, replayed together on two streams, at lengths
    that change between replays."""
    S = require_gpu()
    rng = np.random.default_rng(31)
    st = Setup(S, rng, [2000, 1500], 2, 128, "nvfp4", 16).fill()
    made = []
    for new in (1, 3):
        q, x = bf16(rng, 2 * new, 8, 128)
        batch = st.batch([new, new])
        ws = S.alloc_attention_workspace(st.cache, batch, 8)
        y, lse = S.sharq_attention(q, st.cache, batch, return_lse=True, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            S.sharq_attention(q, st.cache, batch, y=y, lse=lse, workspace=ws)
        made.append((new, x, batch, y, lse, g, q))  # the graph reads q at every replay
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for lens in ([2000, 1500], [40, 1499], [333, 7], [1999, 64]):
        for m in made:
            m[2].kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        torch.cuda.synchronize()
        for s, m in zip(streams, made):
            with torch.cuda.stream(s):
                for _ in range(3):
                    m[5].replay()
        torch.cuda.synchronize()
        for new, x, batch, y, lse, *_ in made:
            check_rows(S, st, x, y, lse, [new, new], lens)


def test_a_block_end_to_end():
    """The attention side of a decode step as a served model runs it: QKV projection, append,
    attention, o projection, norms and residual, the next preparation."""
    S = require_gpu()
    rng = np.random.default_rng(41)
    k, hq, h, d = 512, 4, 2, 128
    wq, _ = bf16(rng, (hq + 2 * h) * d, k, scale=0.05)
    wo, _ = bf16(rng, k, hq * d, scale=0.05)
    pq, po = S.sharq_pack_weight(wq), S.sharq_pack_weight(wo)
    one = torch.ones(k, dtype=torch.bfloat16, device="cuda")
    st = Setup(S, rng, [60, 9], h, d, "nvfp4", 16).fill()
    x, _ = bf16(rng, 2, k)
    batch = st.batch([1, 1])
    qkv = S.sharq_linear(S.sharq_prepare(x, one), pq)
    inv = torch.tensor(10000.0 ** (-np.arange(d // 2) / (d // 2)), dtype=torch.float32, device="cuda")
    q = S.sharq_kv_append(qkv, st.cache, batch, hq, inv_freq=inv)
    y, lse = S.sharq_attention(q, st.cache, batch, return_lse=True)
    check_rows(S, st, q.double().cpu().numpy(), y, lse, [1, 1], st.lengths)
    o = S.sharq_linear(S.sharq_prepare(y.view(2, -1)), po)
    r, hid = S.sharq_norm_residual(o, x, pre_gamma=one)
    assert torch.equal(r, (x.float() + o.float()).bfloat16())
    nxt = S.sharq_prepare(hid)
    torch.cuda.synchronize()
    assert nxt.tokens == 2 and S.sharq_device_status() == S.SHARQ_OK
    assert math.isclose(float(hid.float().square().mean()), 1.0, rel_tol=2 ** -6)


def test_refusals():
    S = require_gpu()
    rng = np.random.default_rng(1)
    st = Setup(S, rng, [20], 2, 64, "nvfp4", 16)
    batch = st.batch([2])
    q, _ = bf16(rng, 2, 4, 64)
    for bad in (q.float(), q[:1], q[..., :32], q[:, :3], q.transpose(0, 1).contiguous().transpose(0, 1), q.cpu()):
        with pytest.raises(S.SharqError):
            S.sharq_attention(bad, st.cache, batch)
    for kw in (dict(causal=False, window=3), dict(window=-1), dict(scale=float("nan")), dict(y=q[:1]), dict(y=q), dict(lse=q),
               dict(workspace=torch.zeros(1, dtype=torch.uint8, device="cuda")[:0])):
        with pytest.raises(S.SharqError):
            S.sharq_attention(q, st.cache, batch, **kw)
    qkv, _ = bf16(rng, 2, 8 * 64)
    for kw in (dict(q_heads=3), dict(inv_freq=torch.ones(3, device="cuda")), dict(inv_freq=torch.ones(40, device="cuda")),
               dict(q_gamma=torch.ones(64, device="cuda")), dict(q_out=q[:1])):
        with pytest.raises(S.SharqError):
            S.sharq_kv_append(qkv, st.cache, batch, **{"q_heads": 4, **kw})
    with pytest.raises(S.SharqError):
        S.sharq_kv_append(qkv[:, :-8], st.cache, batch, 4)
    with pytest.raises(S.SharqError):
        S.sharq_kv_read(st.cache, batch, out_dtype=torch.float16)
    with pytest.raises(S.SharqError):
        S.KVCache(st.cache.pages[:-1], st.num_pages, 16, 2, 64)
    with pytest.raises(S.SharqError):
        S.KVCache(st.cache.pages, st.num_pages, 16, 2, 64, "mxfp4", st.cache.k_scale)
    with pytest.raises(S.SharqError):
        S.KVCache(st.cache.pages, st.num_pages, 16, 2, 64, "nvfp4", st.cache.k_scale[:1])
    with pytest.raises(S.SharqError):
        S.KVBatch(batch.cu_q[:1], batch.kv_len, batch.page_table, 1, 1)
    with pytest.raises(S.SharqError):
        S.KVBatch(batch.cu_q.long(), batch.kv_len, batch.page_table, 1, 1)
    empty = S.KVBatch(batch.cu_q, batch.kv_len, batch.page_table, 0, 0)
    y, lse = S.sharq_attention(q[:0], st.cache, empty, return_lse=True)
    assert y.shape == (0, 4, 64) and lse.shape == (0, 4)
