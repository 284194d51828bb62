"""Rows so small that fl32(7 / amax) (or 127 / amax) is infinite, through every variant of
the rotation and quantiser: the definition's clamp decides, so a value has the
largest code with its sign.  Against the oracle and against that statement."""
import numpy as np
import pytest
import torch

import oracle as O
from test_gpu_parity import dev, host, hq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("M,K,group", [(3, 64, 8), (5, 512, 128), (9, 4096, 4096), (70, 512, 128), (70, 1024, 256),
                                       (70, 4096, 4096), (70, 96, 32)])
def test_codes_of_tiny_rows(M, K, group, bits):
    rng = np.random.default_rng(M + K)
    top = 7 if bits == 4 else 127
    amax = 10.0 ** rng.uniform(-39.5, -36.0, (M, 1))
    x = rng.standard_normal((M, K)).astype(np.float32)
    x[:, ::group] = 3.0 * group                    # keeps every rotated value away from zero
    x = x / np.abs(x).max(1, keepdims=True) * (amax / 2)
    x[M // 2] = rng.standard_normal(K)             # an ordinary row among them
    x[M // 2, ::group] = 3.0 * group
    X = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
    d = np.ones(group, np.int8)
    d[1::3] = -1
    want = (O.rotate_quant if bits == 4 else O.rotate_quant8)(X, "bf16", group, d)
    got = (hq.hq_rotate_quant if bits == 4 else hq.hq_rotate_quant8)(dev(X, "bf16"), group, torch.from_numpy(d).cuda())
    q = host(got[0])
    q = O.unpack_s4(q, K) if bits == 4 else q
    u = O.rotate_rows(X, "bf16", group, d)
    peak = np.abs(u).max(1)
    assert (u != 0).all()
    with np.errstate(over="ignore"):
        small = np.isinf(np.float32(top) / peak)
    assert small.any() and not small.all()
    assert np.array_equal(q[small], (top * np.sign(u[small])).astype(q.dtype))
    assert np.array_equal(host(got[0]), want[0])
    assert np.array_equal(host(got[1]).view(np.uint32), want[1].view(np.uint32))
