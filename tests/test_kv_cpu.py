"""The paged FP4 cache and its operators without a GPU: the layout's arithmetic, the oracle's pins,
and the refusals (checked on the host before any launch)."""
import ctypes

import numpy as np
import pytest
import torch

from fp4_activation_sparse_b200 import build as B
from oracle import kv as K
from oracle.formats import E2M1_MAGNITUDES


@pytest.fixture(scope="module")
def S():
    if not B.up_to_date():
        B.build()
    import fp4_activation_sparse_b200 as S
    return S


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("d", [64, 128])
def test_layout_covers_every_byte_once(fmt, d):
    at = np.concatenate([p.reshape(-1) for p in K.places(d, fmt)])
    assert np.array_equal(np.sort(at), np.arange(K.group_bytes(d, fmt)))


def test_page_bytes(S):
    assert S.sharq_kv_page_bytes(16, 8, 128, "nvfp4") == 8 * K.group_bytes(128, "nvfp4") == 8 * 2304
    assert S.sharq_kv_page_bytes(64, 4, 128, "mxfp4") == 4 * 4 * 2176
    assert S.sharq_kv_page_bytes(32, 1, 64, "nvfp4") == 2 * 1152
    assert S.sharq_kv_page_bytes(4096, 3, 64, "mxfp4") == 3 * 256 * 1088


@pytest.mark.parametrize("args", [(8, 1, 128, 0), (48, 1, 128, 0), (8192, 1, 128, 0), (16, 0, 128, 0), (16, 1, 96, 0),
                                  (16, 1, 128, 2), (16, 1, 0, 0)])
def test_page_bytes_refuses(S, args):
    assert S.lib.sharq_kv_page_bytes(*args) == 0
    assert S.last_error()


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_quantizer_takes_the_nearest_value(fmt):
    rng = np.random.default_rng(5)
    x = rng.standard_normal((40, 3, 64)).astype(np.float32)
    x[:, :, 7] *= 30
    scale = np.array([0.01, 0.002, 0.03], np.float32) if fmt == "nvfp4" else None
    codes, byte = K.quantize(x, fmt, scale)
    v = K.values(codes, byte, fmt, scale)
    unit = K.values(np.full_like(codes, 2), byte, fmt, scale)  # what code 1.0 stands for
    u = np.abs(x) / unit
    grid = np.array(E2M1_MAGNITUDES)
    best = np.abs(np.minimum(u, 6)[..., None] - grid).min(-1)
    assert (np.abs(np.minimum(u, 6) - np.abs(v) / unit) <= best + 1e-5).all()
    if fmt == "nvfp4":  # the largest value of a block lands near 6 unless its scale saturates
        assert ((u.reshape(40, 3, -1, 16).max(-1) < 6.4) | (byte == 126)).all()


def test_quantizer_edges():
    x = np.zeros((1, 1, 64), np.float32)
    codes, byte = K.quantize(x, "mxfp4", None)
    assert not codes.any() and (byte == 127 - 23).all()
    x[0, 0, 0], x[0, 0, 40] = 2.0 ** -40, 1e6
    codes, byte = K.quantize(x, "mxfp4", None)
    assert byte.reshape(-1).tolist() == [104, 140]
    assert K.values(codes, byte, "mxfp4", None).reshape(-1)[[0, 40]].tolist() == [0.0, 6 * 2.0 ** 13]


def test_attention_oracle_by_hand():
    q = np.array([[[1.0, 0.0]], [[0.0, 2.0]]])
    k = np.array([[[1.0, 0.0]], [[0.0, 1.0]], [[1.0, 1.0]]])
    v = np.array([[[1.0, 0.0]], [[0.0, 1.0]], [[4.0, 4.0]]])
    y, lse, *_ = K.attention(q, k, v, 1, True, 0, 1.0)
    w = np.exp([1.0, 0.0])
    np.testing.assert_allclose(y[0, 0], w / w.sum())
    np.testing.assert_allclose(lse[1, 0], np.log(1 + 2 * np.exp(2.0)))
    y, lse, *_ = K.attention(q, k, v, 1, True, 1, 1.0)  # a window of one: itself
    np.testing.assert_allclose(y[:, 0], v[1:, 0])
    y, lse, *_ = K.attention(q, k[:0], v[:0], -2, True, 0, 1.0)
    assert not y.any() and np.isneginf(lse).all()


def good(S):
    c = S._KVCache(0x1000, 0x1000, 0x1000, 4, 16, 2, 128, 0)
    b = S._KVBatch(0x1000, 0x1000, 0x1000, 3, 2, 5, 9)
    return c, b


def calls(S, c, b, **kw):
    """The status of each cache operator on these structs (pointers that no launch may reach)."""
    p, z = ctypes.c_void_p(0x1000), ctypes.c_void_p(0)
    a = dict(stride=(4 + 4) * 128, hq=4, rot=128, freq=p, qg=z, kg=z, eps=1e-6, out=p, q=p, qs=4 * 128, causal=1, window=0,
             scale=0.1, lse=z, ws=p, wsn=0, dtype=0, x=p)
    a.update(kw)
    c, b = ctypes.byref(c) if c else None, ctypes.byref(b) if b else None
    return (S.lib.sharq_kv_append(a["x"], a["stride"], a["hq"], c, b, a["qg"], a["kg"], a["eps"], a["freq"], a["rot"], 0, a["out"], z),
            S.lib.sharq_kv_read(c, b, a["out"], a["out"], a["dtype"], z),
            S.lib.sharq_attention(a["q"], a["qs"], a["hq"], c, b, a["causal"], a["window"], a["scale"], a["out"], a["lse"],
                                  a["ws"], a["wsn"], z))


@pytest.mark.parametrize("field,value", [
    ("pages", 0), ("pages", 0x1008), ("num_pages", 0), ("page_size", 24), ("page_size", 8), ("kv_heads", 0), ("fmt", 3),
    ("fmt", 1),  # MXFP4 with second-level scales
    ("k_scale", 0x1002), ("head_dim", 0)])
def test_cache_fields_refused(S, field, value):
    c, b = good(S)
    setattr(c, field, value)
    assert calls(S, c, b) == (S.SHARQ_ERR_INVALID_ARG,) * 3
    assert S.lib.sharq_attention_workspace_size(ctypes.byref(c), ctypes.byref(b), 4) == 0


def test_head_dim_not_executed(S):
    c, b = good(S)
    c.head_dim = 96
    assert calls(S, c, b, stride=8 * 128) == (S.SHARQ_ERR_UNSUPPORTED,) * 3


@pytest.mark.parametrize("field,value", [
    ("cu_q", 0), ("kv_len", 0), ("page_table", 0), ("n_seq", 0), ("max_pages", 0), ("max_pages", 1 << 27), ("max_q", 0),
    ("max_q", -1), ("tokens", -1), ("cu_q", 0x1002)])
def test_batch_fields_refused(S, field, value):
    c, b = good(S)
    setattr(b, field, value)
    assert calls(S, c, b) == (S.SHARQ_ERR_INVALID_ARG,) * 3


def test_null_structs_refused(S):
    c, b = good(S)
    assert calls(S, None, b) == (S.SHARQ_ERR_INVALID_ARG,) * 3
    assert calls(S, c, None) == (S.SHARQ_ERR_INVALID_ARG,) * 3


@pytest.mark.parametrize("kw,which", [
    (dict(hq=3), (0, 2)), (dict(hq=0), (0, 2)), (dict(stride=512), (0,)), (dict(stride=1025), (0,)), (dict(rot=24), (0,)),
    (dict(rot=144), (0,)), (dict(freq=ctypes.c_void_p(0)), (0,)), (dict(qg=ctypes.c_void_p(0x1008)), (0,)),
    (dict(qg=ctypes.c_void_p(0x1000), eps=-1.0), (0,)), (dict(out=ctypes.c_void_p(0)), (0, 1, 2)),
    (dict(out=ctypes.c_void_p(0x1004)), (0, 1, 2)), (dict(dtype=2), (1,)), (dict(window=-1), (2,)),
    (dict(window=4, causal=0), (2,)), (dict(scale=float("nan")), (2,)), (dict(scale=float("inf")), (2,)), (dict(qs=508), (2,)),
    (dict(q=ctypes.c_void_p(0x1002)), (2,)), (dict(lse=ctypes.c_void_p(0x1002)), (2,)), (dict(ws=ctypes.c_void_p(0)), (2,)),
    (dict(wsn=0), (2,)), (dict(x=ctypes.c_void_p(0)), (0,))])
def test_arguments_refused(S, kw, which):
    c, b = good(S)
    # what the case does not aim at is made to fail too, so that nothing of it can launch
    got = calls(S, c, b, **{"x": ctypes.c_void_p(0), "dtype": 9, "wsn": 0, **kw})
    for i in which:
        assert got[i] == S.SHARQ_ERR_INVALID_ARG, (i, S.last_error())


def test_no_tokens_is_no_launch(S):
    c, b = good(S)
    b.tokens = b.max_q = 0
    assert calls(S, c, b) == (S.SHARQ_OK,) * 3


@pytest.mark.parametrize("kw", [dict(k=12), dict(k=0), dict(k=32776), dict(tokens=-1), dict(y=0), dict(r=0), dict(rout=0),
                                dict(h=0), dict(y=0x1008), dict(gate_rows=0), dict(gate_rows=2, rpg=3), dict(rpg=-1),
                                dict(eps=-1.0), dict(alpha=float("inf")), dict(pre=0x1004)])
def test_norm_residual_refuses(S, kw):
    a = dict(y=0x1000, r=0x1000, tokens=7, k=64, post=0x1000, gate=0x1000, gate_rows=7, rpg=1, alpha=1.0, pre=0x1000,
             eps=1e-6, rout=0x1000, h=0x1000)
    a.update(kw)
    P = ctypes.c_void_p
    assert S.lib.sharq_norm_residual(P(a["y"]), P(a["r"]), a["tokens"], a["k"], P(a["post"]), P(a["gate"]), a["gate_rows"],
                                     a["rpg"], a["alpha"], P(a["pre"]), a["eps"], P(a["rout"]), P(a["h"]),
                                     P(0)) == S.SHARQ_ERR_INVALID_ARG
    assert S.last_error()


def test_norm_residual_without_rows(S):
    P = ctypes.c_void_p
    assert S.lib.sharq_norm_residual(P(0), P(0), 0, 64, P(0), P(0), 0, 0, 1.0, P(0), 1e-6, P(0), P(0), P(0)) == S.SHARQ_OK


def test_binding_refuses_host_tensors(S):
    with pytest.raises(S.SharqError) as e:
        S.sharq_norm_residual(torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(2, 64, dtype=torch.bfloat16))
    assert e.value.status == S.SHARQ_ERR_INVALID_ARG
    with pytest.raises(S.SharqError):
        S.KVCache(torch.zeros(1 << 20, dtype=torch.uint8), 1, 16, 8, 128)
    with pytest.raises(S.SharqError):
        z = torch.zeros(2, dtype=torch.int32)
        S.KVBatch(z, z[:1], z.view(1, 2), 1, 1)


def test_binding_refuses_strides_inside_a_row(S):
    t = torch.zeros(4, 6, 128)
    assert S._rows(t, "q") == 768
    assert S._rows(t.view(4, 768)[:, :512], "q") == 768
    assert S._rows(t[:, :4], "q") == 768
    assert S._rows(t[:1, :4], "q") == 512
    with pytest.raises(S.SharqError):
        S._rows(t.transpose(0, 1), "q")
    with pytest.raises(S.SharqError):
        S._rows(t[:, :, ::2], "q")
