"""The residual / norm / quantiser calls at their edges: rows of infinities in any
arrangement, rows whose largest value is too small for the quantiser's reciprocal, the
largest rows the fp32 sum of squares has room for.  Tolerances as derived in
test_gpu_norm."""
import numpy as np
import pytest
import torch

from test_gpu_norm import BF16, F16, F32, U, codes_fp32, f32, half_step, hq, inv_rms, rows, unpack, weights

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


def holes(M, K, dt, pad=0):
    """[M, K] view of a buffer full of NaN, rows on 16 bytes."""
    return torch.full((M, -(-K // 8) * 8 + pad), NAN, dtype=dt, device="cuda")[:, :K]


def within(got, want, tol):
    err = (got.double() - want).abs()
    assert (err <= tol).all(), ((~(err <= tol)).sum(), (err / tol).max())


def check_x(x, h, w, off, eps):
    want = h.double() * (w.double() + off) * inv_rms(h.double(), eps)
    tol = 33 * U * want.abs()
    within(x, want, tol + half_step(want.abs() + tol, h.dtype))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("xt", [F16, BF16])
@pytest.mark.parametrize("K,group", [(128, 128), (1024, 8), (2048, 128), (1536, 512), (4096, 4096)])
def test_scale_of_rows_with_infinities(K, group, xt, bits):
    """NaN whatever the infinities' number, signs and places: those of one group may
    leave only NaN behind the rotation, beside finite groups or with none."""
    M = 12
    H, w = rows(M, K, xt, 3), weights(K, xt, 4)
    d = torch.ones(group, dtype=torch.int8, device="cuda")
    d[2] = -1
    w[K - 3] = 0
    want = hq.hq_norm_rotate_quant(H, w, 1e-5, group, d, bits=bits)
    assert want[1].isfinite().all()
    g = torch.Generator(device="cuda").manual_seed(5)
    H2 = H.clone()
    H2[1, :4] = torch.tensor([INF, INF, INF, -INF])
    H2[2, :4] = torch.tensor([INF, INF, -INF, -INF])
    H2[4] = torch.where(torch.rand(K, generator=g, device="cuda") < 0.5, -INF, INF)
    H2[5, torch.randperm(K, generator=g, device="cuda")[:8]] = INF
    H2[6, torch.randperm(K, generator=g, device="cuda")[:8]] = torch.tensor([INF, -INF] * 4, dtype=xt, device="cuda")
    H2[7, K - 3] = INF                    # on a channel of weight zero
    H2[8] = INF
    H2[9, 0] = NAN
    H2[10, K - 1] = -INF
    bad = [1, 2, 4, 5, 6, 7, 8, 9, 10]
    got = hq.hq_norm_rotate_quant(H2, w, 1e-5, group, d, bits=bits)
    for m in range(M):
        if m in bad:
            assert got[1][m].isnan(), (m, got[1][m])
        else:
            assert torch.equal(got[0][m], want[0][m]) and got[1][m] == want[1][m]
    # the block's infinities, with the gate, are the stream's
    Y = torch.zeros_like(H)
    Y[1, :4] = torch.tensor([INF, INF, INF, -INF])
    Y[3] = INF
    got = hq.hq_norm_rotate_quant(H, w, 1e-5, group, d, Y=Y, gate=weights(K, xt, 6).abs() + 1, bits=bits)
    assert got[1][[1, 3]].isnan().all() and got[1][[0, 2, 4]].isfinite().all()
    # and those of the weights every row's
    w2 = w.clone()
    w2[:4] = torch.tensor([INF, INF, INF, -INF])
    assert hq.hq_norm_rotate_quant(H, w2, 1e-5, group, d, bits=bits)[1].isnan().all()


def tiny_rows(K, group, amaxes):
    H = torch.randn(len(amaxes), K, generator=torch.Generator().manual_seed(7))
    H[:, 0] = 2.0 * group                   # no rotated value of the first group is zero
    H[:, group:2 * group] = 0               # those of the second are, where there is one
    return (H / H.abs().amax(1, keepdim=True) * torch.tensor(amaxes)[:, None] / 2).to(BF16)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("K,group", [(64, 8), (128, 128), (2048, 512), (4096, 4096)])
def test_rows_too_small_for_the_reciprocal(K, group, bits):
    """Where 7 / amax is infinite the clamp decides: the largest code with the value's
    sign, 0 for a zero.  Rows on both sides of that, bf16 subnormals among them."""
    top = 7 if bits == 4 else 127
    amaxes = [3e-40, 1e-39, 1e-38, 2e-38, 3e-38, 1e-37, 3.5e-37, 4e-37, 1e-36]
    H = tiny_rows(K, group, amaxes).cuda()
    w = torch.ones(K, dtype=F32, device="cuda")
    Xq, sx, _, _ = hq.hq_norm_rotate_quant(H, w, 1e-5, group, bits=bits)
    q = unpack(Xq, bits).astype(np.int64)
    u = f32(H)
    s = 1
    while s < group:
        t = u.reshape(len(amaxes), K // (2 * s), 2, s)
        u = np.stack((t[:, :, 0] + t[:, :, 1], t[:, :, 0] - t[:, :, 1]), 2).reshape(len(amaxes), K)
        s *= 2
    amax = np.abs(u).max(1)
    assert u.dtype == np.float32 and (amax > 0).all()
    with np.errstate(over="ignore"):
        inv = np.float32(top) / amax
    assert np.isinf(inv).any() and np.isfinite(inv).any()
    for m in range(len(amaxes)):
        if np.isinf(inv[m]):
            want = np.sign(u[m]).astype(np.int64) * top
        else:
            want = np.clip(np.rint(u[m] * inv[m]), -top, top).astype(np.int64)
        assert np.array_equal(q[m], want), (m, inv[m], q[m][:8], want[:8])
    want = (amax / np.float32(top)).astype(np.float32) * np.float32(1 / np.sqrt(group))
    want = want.astype(np.float64) / np.sqrt(1e-5)
    assert (np.abs(sx.cpu().numpy() - want) <= 34 * U * want + 2.0 ** -149 * 400).all()


@pytest.mark.parametrize("K", [4096, 16384])
@pytest.mark.parametrize("xt", [BF16, F32])
def test_rows_as_large_as_the_sum_of_squares_allows(xt, K):
    """sum v^2 just below the largest fp32 number (3.4028e38)."""
    g = torch.Generator(device="cuda").manual_seed(1)
    size = (0.98 * 3.4028e38 / K) ** 0.5
    H = torch.where(torch.rand(3, K, generator=g, device="cuda") < 0.5, -size, size).to(xt)
    H = torch.where(H.double().abs() > size, H * 0.99, H).to(xt)      # a rounding up of the type taken back
    H[1, ::2] = 0
    assert (H.double().square().sum(1) < 3.4028e38).all()
    w = weights(K, F32, 2)
    x = hq.hq_residual_norm(H, w, 1e-5, X=holes(3, K, xt))[1]
    check_x(x, H, w, 0.0, 1e-5)
    if xt != F32:
        sx = hq.hq_norm_rotate_quant(H, w, 1e-5, 128)[1]
        _, _, amax = codes_fp32(H, None, None, 1.0, w, 0.0, 128, None, 4)
        want = amax.astype(np.float64) / 7 / np.sqrt(128) * inv_rms(H.double(), 1e-5)[:, 0].cpu().numpy()
        assert (np.abs(sx.cpu().numpy() - want) <= 34 * U * want).all()
