"""Norms before and after a block with its gate and residual scale, against the oracle."""
import numpy as np
import pytest
import torch

from oracle import kv as K
from tests.gpu_common import require_gpu
from tests.kv_common import BF16, bf16

pytestmark = pytest.mark.gpu


def check(r, h, y, res, post, gate, rows, alpha, pre):
    ref, mag = K.norm_residual(y, res, post, gate, rows, alpha)
    got = r.double().cpu().numpy()
    # at most eight rounded float32 steps of the two terms, then bf16
    assert (np.abs(got - ref) <= np.abs(ref) * BF16 + mag * 2.0 ** -21 + 1e-38).all()
    if pre is not None:
        want = got * K.rstd(got, 1e-6) * pre  # of the residual stream as stored
        assert (np.abs(h.double().cpu().numpy() - want) <= np.abs(want) * (BF16 + 2.0 ** -21) + 1e-38).all()


@pytest.mark.parametrize("tokens,k", [(1, 8), (1, 264), (3, 4096), (17, 5120), (5, 32768), (2, 32760), (300, 512), (1, 7168)])
@pytest.mark.parametrize("post,gates,pre,alpha", [(True, 0, True, 1.0), (False, 1, True, 0.5), (True, 3, False, 0.87), (False, 0, False, 0.0)])
def test_norm_residual(tokens, k, post, gates, pre, alpha):
    S = require_gpu()
    rng = np.random.default_rng(tokens + k)
    y, yv = bf16(rng, tokens, k)
    r, rv = bf16(rng, tokens, k, scale=3.0)
    pg, pgv = bf16(rng, k) if post else (None, None)
    qg, qgv = bf16(rng, k) if pre else (None, None)
    g, gv = bf16(rng, gates, k) if gates else (None, None)
    rows = -(-tokens // gates) if gates > 1 else 0
    ro, h = S.sharq_norm_residual(y, r, pg, g, rows, alpha, qg)
    assert (h is None) == (not pre)
    check(ro, h, yv, rv, pgv, gv, rows, np.float64(np.float32(alpha)), qgv)
    if gates == 1:  # one gate row may come as a vector
        again, _ = S.sharq_norm_residual(y, r, pg, g[0], 0, alpha, qg)
        assert torch.equal(again, ro)
    # in place
    r2, y2 = r.clone(), y.clone()
    ro2, h2 = S.sharq_norm_residual(y2, r2, pg, g, rows, alpha, qg, residual_out=r2, h_out=y2 if pre else None)
    assert ro2 is r2 and torch.equal(r2, ro)
    assert not pre or torch.equal(h2, h)


def test_zero_and_special_rows():
    S = require_gpu()
    rng = np.random.default_rng(1)
    y, yv = bf16(rng, 4, 1024)
    r, rv = bf16(rng, 4, 1024)
    one = torch.ones(1024, dtype=torch.bfloat16, device="cuda")
    y[0], r[0] = 0, 0
    y[1, 3] = float("inf")
    r[2, 7] = float("nan")
    ro, h = S.sharq_norm_residual(y, r, one, None, 0, 1.0, one)
    assert not ro[0].any() and not h[0].any()
    assert torch.isnan(ro[1, 3]) and torch.isnan(h[1]).all()  # inf * rstd 0
    assert torch.isnan(ro[2, 7]) and torch.isfinite(ro[2, :7]).all() and torch.isnan(h[2]).all()
    check(ro[3:], h[3:], yv[3:], rv[3:], np.ones(1024), None, 0, 1.0, np.ones(1024))
    tiny = torch.full((1, 64), 1e-30, dtype=torch.bfloat16, device="cuda")
    ro, h = S.sharq_norm_residual(tiny, tiny, one[:64], None, 0, 1.0, one[:64])
    assert torch.isfinite(h).all()


@pytest.mark.parametrize("size", [6e18, 1e-18])
def test_rows_whose_squares_leave_float32(size):
    """Eight squares together overflow or lose float32's precision, their mean over the row does not."""
    S = require_gpu()
    rng = np.random.default_rng(7)
    y, yv = bf16(rng, 3, 4096, scale=size)
    z = torch.zeros_like(y)
    y[:, 64:4096 if size > 1 else 64] = 0  # few large values; every small one
    one = torch.ones(4096, dtype=torch.bfloat16, device="cuda")
    got = y.double().cpu().numpy()
    want = got * K.rstd(got, 0.0)
    for r, h in (S.sharq_norm_residual(y, z, pre_gamma=one, eps=0.0), S.sharq_norm_residual(z, y, pre_gamma=one, eps=0.0)):
        assert torch.equal(r, y)
        assert (np.abs(h.double().cpu().numpy() - want) <= np.abs(want) * (BF16 + 2.0 ** -21)).all()
    r, _ = S.sharq_norm_residual(y, z, post_gamma=one, eps=0.0)
    assert (np.abs(r.double().cpu().numpy() - want) <= np.abs(want) * (BF16 + 2.0 ** -21)).all()


def test_other_stream_and_no_rows():
    S = require_gpu()
    rng = np.random.default_rng(2)
    y, yv = bf16(rng, 64, 2048)
    r, rv = bf16(rng, 64, 2048)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ro, _ = S.sharq_norm_residual(y, r, stream=side)
    side.synchronize()
    check(ro, None, yv, rv, None, None, 0, 1.0, None)
    ro, h = S.sharq_norm_residual(y[:0], r[:0], pre_gamma=y[0])
    assert ro.shape == (0, 2048) and h.shape == (0, 2048)


def test_refusals():
    S = require_gpu()
    z = torch.zeros(6, 64, dtype=torch.bfloat16, device="cuda")
    for kw in (dict(residual=z[:5]), dict(residual=z.float()), dict(post_gamma=z[0, :32]), dict(gate=z[:2], rows_per_gate=2),
               dict(gate=z, rows_per_gate=-1), dict(h_out=z), dict(alpha=float("nan")), dict(eps=-1.0, pre_gamma=z[0]),
               dict(residual_out=z[:, :32]), dict(residual_out=z, h_out=z, pre_gamma=z[0])):
        with pytest.raises(S.SharqError):
            S.sharq_norm_residual(z, **{"residual": z, **kw})
    with pytest.raises(S.SharqError):
        S.sharq_norm_residual(z[:, :63], z[:, :63])
    with pytest.raises(S.SharqError):
        S.sharq_norm_residual(z[:, :12].contiguous(), z[:, :12].contiguous())
