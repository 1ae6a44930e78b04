"""Appending to the paged FP4 cache and reading it back, against the oracle."""
import numpy as np
import pytest
import torch

from oracle import kv as K
from oracle.formats import e2m1_decode
from tests.gpu_common import code_steps, require_gpu
from tests.kv_common import BF16, F32, Setup, bf16

pytestmark = pytest.mark.gpu


def rows_of(new, lengths):
    """Sequence and position of every token row."""
    return [(b, n - m + i) for b, (m, n) in enumerate(zip(new, lengths)) for i in range(m)]


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("d,heads,group,page", [(128, 8, 4, 16), (64, 3, 1, 32), (128, 1, 8, 128), (64, 16, 1, 4096)])
def test_append_without_rotation_is_bit_exact(fmt, d, heads, group, page):
    S = require_gpu()
    rng = np.random.default_rng(d + heads)
    lengths, new = [37, 1, 0, 130, 16], [37, 1, 0, 61, 0]
    st = Setup(S, rng, lengths, heads, d, fmt, page)
    qkv, x = bf16(rng, sum(new), (group + 2) * heads * d)
    q = S.sharq_kv_append(qkv, st.cache, st.batch(new), group * heads)
    x = x.reshape(len(x), -1, d)
    assert torch.equal(q.view(len(x), -1), qkv[:, : group * heads * d])
    kc, kb = K.quantize(x[:, group * heads:group * heads + heads].astype(np.float32), fmt, st.k_scale)
    vc, vb = K.quantize(x[:, group * heads + heads:].astype(np.float32), fmt, st.v_scale)
    k, v = S.sharq_kv_read(st.cache, st.batch(new), out_dtype=torch.float32)
    kh, vh = S.sharq_kv_read(st.cache, st.batch(new))
    at = 0
    for b, m in enumerate(new):
        got = st.raw(b, np.arange(lengths[b] - m, lengths[b]))
        for g, r, name in zip(got, (kc, kb, vc, vb), ("k codes", "k scales", "v codes", "v scales")):
            assert np.array_equal(g, r[at:at + m]), (b, name)
        at += m
    for t, h, c, byte, s in ((k, kh, kc, kb, st.k_scale), (v, vh, vc, vb, st.v_scale)):
        ref = K.values(c, byte, fmt, s)  # two float32 products: code * block scale is exact
        assert (np.abs(t.double().cpu().numpy() - ref) <= np.abs(ref) * F32).all()
        assert torch.equal(h, t.bfloat16())


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("d,rot,inter,norm", [(128, 128, False, False), (128, 64, True, True), (64, 64, True, False),
                                              (64, 16, False, True), (128, 112, False, "k"), (64, 0, False, "q")])
def test_append_with_norm_and_rotation(fmt, d, rot, inter, norm):
    S = require_gpu()
    rng = np.random.default_rng(rot + d)
    heads, hq, eps = 2, 6, 1e-6
    lengths, new = [3, 5000, 40], [3, 29, 17]
    st = Setup(S, rng, lengths, heads, d, fmt, 16)
    wide, _ = bf16(rng, sum(new), (hq + 2 * heads) * d + 24)  # strided rows
    qkv = wide[:, : (hq + 2 * heads) * d]
    x = qkv.double().cpu().numpy().reshape(len(qkv), -1, d)
    inv = (10000.0 ** (-np.arange(rot // 2) / max(1, rot // 2))).astype(np.float32)
    qg, qgv = bf16(rng, d)
    kg, kgv = bf16(rng, d)
    q = S.sharq_kv_append(qkv, st.cache, st.batch(new), hq, inv_freq=torch.from_numpy(inv).cuda() if rot else None,
                          interleaved=inter, q_gamma=qg if norm in (True, "q") else None,
                          k_gamma=kg if norm in (True, "k") else None, eps=eps)
    pos = np.array([p for _, p in rows_of(new, lengths)])
    xq, xk, xv = x[:, :hq], x[:, hq:hq + heads], x[:, hq + heads:]
    if norm in (True, "q"):
        xq = xq * K.rstd(xq, eps) * qgv
    if norm in (True, "k"):
        xk = xk * K.rstd(xk, eps) * kgv
    both = []
    for y in (xq, xk):
        r = K.rotate(y, pos, inv, inter)
        mag = K.rotate(np.abs(y), np.zeros_like(pos), inv, inter)  # |x1| + |x2| bounds a turned pair
        half = rot // 2
        i = np.arange(half)
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + half)
        s = mag[..., a] + mag[..., b]
        mag[..., a], mag[..., b] = s, s
        both.append((r, mag * 2.0 ** -20))  # at most nine rounded float32 steps on the way
    (rq, tq), (rk, tk) = both
    assert (np.abs(q.double().cpu().numpy() - rq) <= np.abs(rq) * BF16 + tq).all()
    vc, vb = K.quantize(xv.astype(np.float32), fmt, st.v_scale)
    kc, kb = K.quantize(rk.astype(np.float32), fmt, st.k_scale)
    at = steps = 0
    for b, m in enumerate(new):
        got = st.raw(b, np.arange(lengths[b] - m, lengths[b]))
        assert np.array_equal(got[2], vc[at:at + m]) and np.array_equal(got[3], vb[at:at + m])
        # a key within float32 rounding of a border may take either side: one step, rarely
        off = code_steps(got[0], kc[at:at + m])
        same = got[1] == kb[at:at + m]
        assert off.max() <= 1
        steps += (off > 0).sum() + (~same).sum()
        at += m
    assert steps <= 2e-3 * kc.size


def test_append_touches_only_its_rows():
    """Padding rows, dropped positions (no page, behind the table, before the start) and every other
    byte of the cache stay as they were."""
    S = require_gpu()
    rng = np.random.default_rng(3)
    lengths = [20, 70, 5]
    st = Setup(S, rng, lengths, 2, 64, "nvfp4", 16).fill()
    before = st.cache.pages.clone()
    table = st.table.copy()
    table[1, 3:] = st.num_pages + 5  # positions 48.. of sequence 1 have no page
    table[0, 1] = -7
    new = [6, 30, 5]
    over = [20, 70 + 40, 2]  # sequence 1 runs behind the table; sequence 2 starts before position 0
    qkv, _ = bf16(rng, sum(new) + 9, 4 * 2 * 64)
    q = torch.full((sum(new) + 9, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    S.sharq_kv_append(qkv, st.cache, st.batch(new, over, tokens=len(qkv), table=table), 4, q_out=q)
    assert torch.equal(q[: sum(new)].view(sum(new), -1), qkv[: sum(new), : 4 * 64])
    assert (q[sum(new):] == 7).all()
    after = st.cache.pages.cpu().numpy()
    changed = set()
    view = (after != before.cpu().numpy()).reshape(st.num_pages, -1)
    changed = set(np.flatnonzero(view.any(1)).tolist())
    # sequence 0 appends at 14, 15 (its page 0); 16..19 dropped. Sequence 2 keeps positions 0, 1.
    assert changed == {int(table[0, 0]), int(table[2, 0])}
    k, v = (torch.full((len(qkv), 2, 64), 5.0, device="cuda") for _ in range(2))
    S.sharq_kv_read(st.cache, st.batch(new, over, tokens=len(qkv), table=table), k, v)
    for t in (k, v):
        assert (t[sum(new):] == 5).all() and not t[2:6].any() and not t[6:6 + 30].any() and not t[36:39].any()
        assert t[39:41].any() and t[0:2].any()


def test_special_values_are_stored_finite():
    S = require_gpu()
    rng = np.random.default_rng(9)
    for fmt in ("nvfp4", "mxfp4"):
        st = Setup(S, rng, [4], 1, 64, fmt, 16)
        qkv, _ = bf16(rng, 4, 3 * 64)
        qkv[0, 64] = float("inf")
        qkv[1, 70] = float("nan")
        qkv[2, 128:] = 0
        qkv[3, 128] = -float("inf")
        S.sharq_kv_append(qkv, st.cache, st.batch([4]), 1)
        k, v = S.sharq_kv_read(st.cache, st.batch([4]), out_dtype=torch.float32)
        assert torch.isfinite(k).all() and torch.isfinite(v).all()
        assert not v[2].any()
        kc = st.raw(0, [1])[0][0, 0]
        assert e2m1_decode(kc[6:7])[0] == 6.0  # the NaN
        fine = np.r_[0:6, 7:16] if fmt == "nvfp4" else np.r_[0:6, 7:32]
        x = qkv[1, 64:128].clone()
        x[6] = 0
        c, _ = K.quantize(x.double().cpu().numpy()[None, None].astype(np.float32), fmt, st.k_scale)
        assert np.array_equal(kc[fine], c[0, 0][fine])


def test_large_cache_offsets_pass_32_bits():
    """Pages beyond 4 GB of the cache."""
    S = require_gpu()
    page_bytes = S.sharq_kv_page_bytes(4096, 8, 128)
    n = (5 << 30) // page_bytes
    pages = torch.empty(n * page_bytes, dtype=torch.uint8, device="cuda")
    cache = S.KVCache(pages, n, 4096, 8, 128)
    rng = np.random.default_rng(1)
    qkv, x = bf16(rng, 3, 3 * 8 * 128)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    batch = S.KVBatch(i32(0, 3), i32(4099), i32(n - 2, n - 1).view(1, 2), 3, 3)
    S.sharq_kv_append(qkv, cache, batch, 8)
    k, v = S.sharq_kv_read(cache, batch, out_dtype=torch.float32)
    c, b = K.quantize(x.reshape(3, 3, 8, 128)[:, 1].astype(np.float32), "nvfp4", None)
    assert np.array_equal(k.double().cpu().numpy(), K.values(c, b, "nvfp4", None))
    tail = pages[(n - 1) * page_bytes:].clone()
    q = qkv.view(3, 3, 8, 128)[:, 0].contiguous()
    y, lse = S.sharq_attention(q, cache, S.KVBatch(i32(0, 3), i32(3), i32(n - 1).view(1, 1), 3, 3), return_lse=True)
    assert torch.equal(pages[(n - 1) * page_bytes:], tail)
    vv = v.double().cpu().numpy()
    kk = k.double().cpu().numpy()
    from tests.kv_common import check_attention
    check_attention(y, lse, K.attention(q.double().cpu().numpy(), kk, vv, 0, True, 0, 128 ** -0.5))


def test_append_on_another_stream_and_in_a_graph():
    """A captured append follows the index tensors' contents at each replay."""
    S = require_gpu()
    rng = np.random.default_rng(4)
    st = Setup(S, rng, [40, 40], 2, 128, "mxfp4", 16)
    st.cache.pages.zero_()
    qkv, x = bf16(rng, 2, 4 * 2 * 128)
    batch = st.batch([1, 1], [1, 1])
    q = torch.empty(2, 4, 128, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        S.sharq_kv_append(qkv, st.cache, batch, 4, q_out=q)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        S.sharq_kv_append(qkv, st.cache, batch, 4, q_out=q)
    codes, byte = K.quantize(x.reshape(2, 8, 128)[:, 4:6].astype(np.float32), "mxfp4", None)
    for n in range(2, 20):
        batch.kv_len.fill_(n)
        g.replay()
    for b in range(2):
        got = st.raw(b, np.arange(20))
        assert np.array_equal(got[0][:19], codes[b][None].repeat(19, 0)) and not got[0][19].any()
        assert np.array_equal(got[1][:19], byte[b][None].repeat(19, 0))
