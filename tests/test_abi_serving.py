"""Refusals of the calls between two layers (residual / norm / quantiser, adapter
plan, adapters) that need no GPU: the C ABI rejects bad arguments with the
documented status before anything is enqueued, the Python calls reject tensors
of the wrong device, type or shape."""
import ctypes as ct

import pytest
import torch

P = ct.c_void_p(16)      # non-null, aligned, never dereferenced: the checks come first
ODD = ct.c_void_p(24)    # not 16-byte aligned
F16, BF16, F32 = 0, 1, 2
OK, ARG, ALIGN, UNSUPPORTED = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    from w4a4_bit_gemm_hq_b200 import build_lib
    build_lib.build()
    from w4a4_bit_gemm_hq_b200 import _lib
    return _lib.lib


P2, P3 = ct.c_void_p(32), ct.c_void_p(48)


def norm(lib, H=P, ldh=256, Y=P2, ldy=256, xt=F16, M=4, K=256, wp=None, gate=None, ldg=0, alpha=1.0, w=P, wt=F16,
         off=0.0, eps=1e-5, Ho=P, ldho=256, X=P2, ldx=256):
    return lib.hq_residual_norm(H, ldh, Y, ldy, xt, M, K, wp, gate, ldg, alpha, w, wt, off, eps, Ho, ldho, X, ldx, None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), ARG), (dict(K=0), ARG), (dict(xt=7), ARG), (dict(wt=-1), ARG),
    (dict(eps=-1e-6), ARG), (dict(eps=float("nan")), ARG),
    (dict(ldh=255), ARG), (dict(ldy=248), ARG), (dict(ldho=8), ARG), (dict(ldx=0), ARG),
    (dict(gate=P, ldg=128), ARG),
    (dict(Y=None, gate=P), ARG), (dict(Y=None, wp=P), ARG),
    (dict(Ho=P3, X=P3), ARG), (dict(ldho=264), ARG), (dict(ldx=264), ARG), (dict(Ho=P2, X=P3, ldho=264), ARG),
    (dict(X=P, Ho=P3, ldx=264), ARG),
    (dict(w=None), ARG), (dict(X=None), ARG), (dict(w=None, X=None, Ho=None), ARG), (dict(H=None), ARG),
    (dict(H=ODD), ALIGN), (dict(Y=ODD), ALIGN), (dict(gate=ODD), ALIGN), (dict(wp=ODD), ALIGN), (dict(w=ODD), ALIGN),
    (dict(Ho=ODD), ALIGN), (dict(X=ODD), ALIGN),
    (dict(Ho=P3, ldh=260), ALIGN), (dict(X=P3, ldx=260), ALIGN), (dict(xt=F32, X=P3, ldy=258), ALIGN), (dict(gate=P, ldg=260), ALIGN),
    (dict(K=16385, ldh=16392, ldy=16392, ldho=16392, ldx=16392), UNSUPPORTED), (dict(M=1 << 31), UNSUPPORTED),
    (dict(M=0, H=None, Y=None, w=None, X=None, Ho=None), OK), (dict(M=0), OK),
])
def test_residual_norm_refusals(lib, kw, want):
    assert norm(lib, **kw) == want


def normq(lib, H=P, ldh=256, Y=P2, ldy=256, xt=F16, M=4, K=256, gate=None, ldg=0, w=P, wt=F16, eps=1e-5, group=128,
          d=None, bits=4, Ho=P, ldho=256, X=None, ldx=0, Xq=P, sx=P):
    return lib.hq_norm_rotate_quant(H, ldh, Y, ldy, xt, M, K, gate, ldg, 1.0, w, wt, 0.0, eps, group, d, bits, Ho, ldho,
                                    X, ldx, Xq, sx, None)


@pytest.mark.parametrize("kw,want", [
    (dict(group=3), ARG), (dict(group=4), ARG), (dict(group=8192), ARG), (dict(group=0), ARG), (dict(group=-8), ARG),
    (dict(K=384, ldh=384, ldy=384, ldho=384, group=256), ARG), (dict(K=240, group=16), ARG),
    (dict(bits=5), ARG), (dict(bits=16), ARG), (dict(M=-1), ARG), (dict(wt=3), ARG), (dict(xt=9), ARG),
    (dict(xt=F32), UNSUPPORTED), (dict(K=32768, ldh=32768, ldy=32768, ldho=32768), UNSUPPORTED),
    (dict(w=None), ARG), (dict(Xq=None), ARG), (dict(sx=None), ARG), (dict(H=None), ARG), (dict(Y=None, gate=P), ARG),
    (dict(Xq=ODD), ALIGN), (dict(X=ODD, ldx=256), ALIGN), (dict(X=P3, ldx=128), ARG), (dict(Ho=P3, ldh=260), ALIGN),
    (dict(M=0, H=None, w=None, Xq=None, sx=None), OK),
])
def test_norm_rotate_quant_refusals(lib, kw, want):
    assert normq(lib, **kw) == want


@pytest.mark.parametrize("M,n", [(1, 0), (1, 5), (64, 1), (65, 1), (4096, 64), (130, 1000)])
def test_max_tiles_is_enough_for_any_batch(lib, M, n):
    rows = lib.hq_lora_max_tiles(M, n)
    buckets = min(n + 1, M)
    # the worst batch: every bucket one token over a multiple of 64
    left, tiles = M - buckets, buckets
    tiles += left // 64
    assert tiles <= rows <= M // 64 + buckets
    assert lib.hq_lora_max_tiles(0, n) == 0 and lib.hq_lora_max_tiles(M, -1) == 0


@pytest.mark.parametrize("a,want", [
    ((P, -1, 4, P2, P3), ARG), ((P, 8, -1, P2, P3), ARG), ((None, 8, 4, P2, P3), ARG), ((P, 8, 4, None, P3), ARG),
    ((P, 8, 4, P2, None), ARG), ((P, 8, 1023, P2, P3), UNSUPPORTED), ((P, 1 << 23, 4, P2, P3), UNSUPPORTED),
    ((P, 8, 4, P, P3), ARG), ((P, 8, 4, P2, P), ARG), ((P, 8, 4, P2, P2), ARG),
    ((None, 0, 4, None, None), OK),
])
def test_plan_refusals(lib, a, want):
    assert lib.hq_lora_plan(*a, None) == want


def lora(lib, X=P, xt=F16, M=4, K=256, ldx=256, A=P, B=P, N=128, n=3, r=16, order=P, tiles=P, base=None, ldb=128, Y=P,
         yt=F16, ldy=128, ws=P, bytes=1 << 20):
    return lib.hq_lora_apply(X, xt, M, K, ldx, A, B, N, n, r, None, None, order, tiles, base, ldb, Y, yt, ldy, ws, bytes,
                             None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), ARG), (dict(K=0), ARG), (dict(N=-8), ARG), (dict(n=-1), ARG), (dict(r=0), ARG),
    (dict(xt=5), ARG), (dict(yt=5), ARG), (dict(xt=F32), UNSUPPORTED),
    (dict(ldx=248), ARG), (dict(ldy=120), ARG), (dict(base=P, ldb=120), ARG),
    (dict(base=ct.c_void_p(32), Y=ct.c_void_p(32), ldb=136), ARG),
    (dict(K=252, ldx=256), UNSUPPORTED), (dict(N=100), UNSUPPORTED), (dict(r=12), UNSUPPORTED),
    (dict(r=264), UNSUPPORTED), (dict(n=1023), UNSUPPORTED), (dict(M=1 << 23), UNSUPPORTED),
    (dict(X=None), ARG), (dict(Y=None), ARG), (dict(A=None), ARG), (dict(B=None), ARG), (dict(order=None), ARG),
    (dict(tiles=None), ARG), (dict(ws=None), ARG), (dict(bytes=255), ARG),
    (dict(X=ODD), ALIGN), (dict(A=ODD), ALIGN), (dict(B=ODD), ALIGN), (dict(Y=ODD), ALIGN), (dict(base=ODD), ALIGN),
    (dict(ws=ODD), ALIGN), (dict(ldx=260), ALIGN), (dict(ldy=132), ALIGN), (dict(base=ct.c_void_p(32), ldb=132), ALIGN),
    (dict(M=0, X=None, Y=None, ws=None), OK), (dict(N=0, Y=None), OK),
])
def test_lora_refusals(lib, kw, want):
    assert lora(lib, **kw) == want


def test_python_calls_refuse_host_tensors(lib):
    from w4a4_bit_gemm_hq_b200 import hq
    h = torch.zeros(4, 256, dtype=torch.float16)
    w = torch.zeros(256, dtype=torch.float16)
    with pytest.raises(ValueError):
        hq.hq_residual_norm(h, w, 1e-5)
    with pytest.raises(ValueError):
        hq.hq_norm_rotate_quant(h, w, 1e-5, 128)
    with pytest.raises(ValueError):
        hq.hq_lora_plan(torch.zeros(4, dtype=torch.int32), 2)
    A, B = torch.zeros(2, 8, 256, dtype=torch.float16), torch.zeros(2, 64, 8, dtype=torch.float16)
    order, tiles = torch.zeros(4, dtype=torch.int32), torch.zeros(3, 3, dtype=torch.int32)
    with pytest.raises(ValueError):
        hq.hq_lora_apply(h, A, B, order, tiles)
