"""Every element of the residual / norm / quantiser's outputs is written: NaN (or bits
that no code has) lies in the buffers before the call, and an output that is NaN
fails.  Tolerances as derived in test_gpu_norm."""
import numpy as np
import pytest
import torch

from test_gpu_norm import CASES, F32, QCASES, U, codes_fp32, f32, half_step, hq, inputs, stream64, unpack
from test_gpu_norm_edges import check_x, holes, within

pytestmark = pytest.mark.gpu


def check_h(h, H, Y, w_post, gate, alpha, off, eps):
    want, block = stream64(H, Y, w_post, gate, alpha, off, eps)
    tol = 35 * U * block + U * want.abs()
    within(h, want, tol + half_step(want.abs() + tol, H.dtype))


@pytest.mark.parametrize("M,K,xt,wt,post,gate,alpha,off,pad", CASES)
def test_residual_norm_writes_every_element(M, K, xt, wt, post, gate, alpha, off, pad):
    H, Y, w, w_post, g = inputs(M, K, xt, wt, post, gate, pad, seed=11)
    h, x = hq.hq_residual_norm(H, w, 1e-5, Y=Y, w_post=w_post, gate=g, alpha=alpha, w_offset=off,
                               H_out=holes(M, K, xt, pad), X=holes(M, K, xt))
    check_h(h, H, Y, w_post, g, alpha, off, 1e-5)
    check_x(x, h, w, off, 1e-5)
    # the norm alone, and the stream alone
    x0 = hq.hq_residual_norm(H, w, 1e-5, w_offset=off, X=holes(M, K, xt))[1]
    check_x(x0, H, w, off, 1e-5)
    h0 = hq.hq_residual_norm(H, None, 1e-5, Y=Y, w_post=w_post, gate=g, alpha=alpha, H_out=holes(M, K, xt))[0]
    check_h(h0, H, Y, w_post, g, alpha, 0.0, 1e-5)


@pytest.mark.parametrize("M,K,group,bits,xt,wt,block,gate,alpha,off,signs", QCASES)
def test_norm_rotate_quant_writes_every_element(M, K, group, bits, xt, wt, block, gate, alpha, off, signs):
    H, Y, w, _, g = inputs(M, K, xt, wt, False, gate, 0, seed=12)
    Y, g = (Y, g) if block else (None, None)
    h, x, sx = holes(M, K, xt, 8), holes(M, K, xt), holes(1, M, F32)[0]
    marked = torch.full((M, K), 99, dtype=torch.int8, device="cuda") if bits == 8 else \
        torch.full((M, K // 2), 0x88, dtype=torch.uint8, device="cuda")     # no code has these bits
    Xq, sx, h, x = hq.hq_norm_rotate_quant(H, w, 1e-5, group, Y=Y, gate=g, alpha=alpha, w_offset=off, bits=bits,
                                           H_out=h, X=x, Xq=marked, sx=sx)
    want_h, want_q, _ = codes_fp32(H, Y, g, alpha, w, off, group, None, bits)
    assert np.array_equal(f32(h), want_h) and np.array_equal(unpack(Xq, bits), want_q)
    check_x(x, h, w, off, 1e-5)
    assert sx.isfinite().all() and (sx > 0).all()
