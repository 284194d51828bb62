"""The quantiser behind the residual and norm at its edges: rows of infinities in any
arrangement."""
import pytest
import torch

from test_gpu_norm import BF16, F16, hq, rows, weights

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


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
