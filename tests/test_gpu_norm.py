"""The residual / gate / norm step and its fusion with the rotation and quantiser,
on the GPU against plain implementations in 64 bits (and, for the codes, against
the fp32 sequence that defines them, in numpy).

Tolerances, u = 2^-24 (half a step of fp32):
 * a row's sum of squares: at most 32 sequential fused adds per thread, 5 over
   the lanes and up to 16 over the warps, all terms positive: relative 53 u; the mean's
   division, the added eps, the square root and the reciprocal: 1 / sqrt is off
   by at most (53 + 1 + 1) / 2 + 1 = 28.5 u, taken as 30 u.
 * h: the block term has up to five roundings more (w + off, two products,
   gate, alpha): 35 u of its size, then one of the sum; and half a step of the
   stream's type, eps / 2.
 * x from the stored h: 30 u + 3 u (w + off, two products), and eps / 2.
 * fp16 results below its normal range: half a step there, 2^-25.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

hq = pytest.importorskip("w4a4_bit_gemm_hq_b200.hq") if torch.cuda.is_available() else None

U = 2.0 ** -24
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def rows(M, K, dt, seed, scale=1.0, pad=0):
    """[M, K] view of a wider buffer: rows on 16 bytes, `pad` elements more behind each."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    per = -(-K // 8) * 8 + pad
    return (scale * torch.randn(M, per, generator=g, device="cuda")).to(dt)[:, :K]


def weights(K, dt, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (1 + 0.3 * torch.randn(K, generator=g, device="cuda")).to(dt)


def half_step(v, dt):
    return v.abs() * (torch.finfo(dt).eps / 2) + (2.0 ** -25 if dt == F16 else 0.0)


def inv_rms(v, eps):
    return 1 / (v.square().mean(1, keepdim=True) + eps).sqrt()


def stream64(H, Y, w_post, gate, alpha, off, eps):
    """(h, size of the block term) in 64 bits."""
    p = Y.double()
    if w_post is not None:
        p = p * (w_post.double() + off) * inv_rms(p, eps)
    if gate is not None:
        p = p * gate.double()
    return H.double() + alpha * p, (alpha * p).abs()


def check_stream(h, H, Y, w_post, gate, alpha, off, eps):
    want, block = stream64(H, Y, w_post, gate, alpha, off, eps)
    tol = 35 * U * block + U * want.abs()
    tol = tol + half_step(want.abs() + tol, H.dtype)
    bad = (h.double() - want).abs() > tol
    assert not bad.any(), (bad.sum(), ((h.double() - want).abs() / tol).max())


def check_normed(x, h, w, off, eps):
    want = h.double() * (w.double() + off) * inv_rms(h.double(), eps)
    tol = 33 * U * want.abs()
    tol = tol + half_step(want.abs() + tol, h.dtype)
    bad = (x.double() - want).abs() > tol
    assert not bad.any(), (bad.sum(), ((x.double() - want).abs() / tol).max())


CASES = [
    # M, K, stream, weights, norm after, gate, alpha, offset, pad
    (1, 1, F32, F32, False, None, 1.0, 0.0, 0),
    (2, 7, F16, F32, True, "token", 0.5, 1.0, 0),
    (3, 8, BF16, BF16, True, "channel", 1.0, 0.0, 8),
    (5, 31, F32, F16, True, "token", 0.22, 0.0, 4),
    (1, 256, F16, F16, False, None, 1.0, 0.0, 0),
    (33, 1000, BF16, F32, True, None, 1.0, 1.0, 24),
    (4, 1023, F16, BF16, False, "channel", 1.4, 1.0, 0),
    (7, 1024, F32, F32, True, "channel", 1.0, 0.0, 0),
    (7, 1025, BF16, F16, False, "token", 1.0, 0.0, 8),
    (2, 4096, F16, F16, False, None, 1.0, 0.0, 0),
    (300, 4096, BF16, BF16, True, "token", 1.0, 1.0, 0),
    (17, 5003, F32, BF16, True, "channel", 0.22, 0.0, 0),
    (3, 8192, BF16, F32, False, "channel", 0.5, 0.0, 0),
    (2, 16383, F16, F32, True, "token", 1.0, 0.0, 0),
    (2, 16384, F32, F32, True, "token", 1.0, 0.0, 0),
    # several rows per CTA
    (9001, 100, BF16, F32, True, "token", 1.0, 0.0, 0),
    (6000, 512, F16, BF16, False, "channel", 0.5, 1.0, 8),
    (2500, 6144, BF16, F16, True, "token", 1.0, 0.0, 0),
    (2000, 10000, F16, F32, True, "channel", 1.0, 0.0, 0),
    (3000, 1301, F32, F16, False, None, 1.0, 0.0, 4),
]


def inputs(M, K, xt, wt, post, gate, pad, seed=0):
    H, Y, w = rows(M, K, xt, seed, 2.0, pad), rows(M, K, xt, seed + 1, 0.5, pad), weights(K, wt, seed + 2)
    w_post = weights(K, wt, seed + 3) if post else None
    g = None if gate is None else rows(1, K, xt, seed + 4)[0].contiguous() if gate == "channel" else rows(M, K, xt, seed + 5)
    return H, Y, w, w_post, g


@pytest.mark.parametrize("M,K,xt,wt,post,gate,alpha,off,pad", CASES)
def test_residual_norm(M, K, xt, wt, post, gate, alpha, off, pad):
    H, Y, w, w_post, g = inputs(M, K, xt, wt, post, gate, pad)
    h, x = hq.hq_residual_norm(H, w, 1e-5, Y=Y, w_post=w_post, gate=g, alpha=alpha, w_offset=off)
    check_stream(h, H, Y, w_post, g, alpha, off, 1e-5)
    check_normed(x, h, w, off, 1e-5)


@pytest.mark.parametrize("xt", [F16, BF16, F32])
def test_parts_alone(xt):
    H, Y, w, w_post, g = inputs(9, 520, xt, xt, True, "token", 0)
    h, x = hq.hq_residual_norm(H, w, 1e-6)                       # a norm alone
    assert h is None
    check_normed(x, H, w, 0.0, 1e-6)
    kept = rows(9, 520, xt, 9)
    h, x = hq.hq_residual_norm(H, w, 1e-6, H_out=kept)           # the stream copied along
    assert h is kept and torch.equal(h, H)
    h, x = hq.hq_residual_norm(H, None, 1e-6, Y=Y, w_post=w_post)   # the norm after the block alone
    assert x is None
    check_stream(h, H, Y, w_post, None, 1.0, 0.0, 1e-6)
    h2, _ = hq.hq_residual_norm(H, w, 1e-6, Y=Y, w_post=w_post)
    assert torch.equal(h, h2)


@pytest.mark.parametrize("xt,K", [(F16, 1025), (BF16, 4096), (F32, 333)])
def test_in_place_and_nothing_else_written(xt, K):
    M, pad = 6, 16
    H, Y, w, w_post, g = inputs(M, K, xt, F32, True, "token", pad)
    h, x = hq.hq_residual_norm(H, w, 1e-5, Y=Y, w_post=w_post, gate=g)
    bufs = []
    for t in (H, Y):   # more rows behind the last one, more elements behind each row
        b = torch.full((M + 3, t.stride(0)), 7.0, dtype=xt, device="cuda")
        b[:M, :K] = t
        bufs.append(b)
    hv, yv = bufs[0][:M, :K], bufs[1][:M, :K]
    h2, x2 = hq.hq_residual_norm(hv, w, 1e-5, Y=yv, w_post=w_post, gate=g, H_out=hv, X=yv)
    assert h2 is hv and x2 is yv
    assert torch.equal(hv, h) and torch.equal(yv, x)
    for b in bufs:
        assert (b[:M, K:] == 7).all() and (b[M:] == 7).all()


@pytest.mark.parametrize("xt", [F16, BF16, F32])
def test_rows_do_not_mix(xt):
    M, K = 8, 1100
    H, Y, w, w_post, _ = inputs(M, K, xt, F32, True, None, 0)
    h, x = hq.hq_residual_norm(H, w, 1e-5, Y=Y, w_post=w_post)
    H2, Y2 = inputs(M, K, xt, F32, True, None, 0)[:2]     # the same values (clones would not keep the row stride)
    H2[1, 3] = float("nan")
    Y2[3, 1000] = float("inf")
    Y2[5] = 0
    H2[6] = 0
    Y2[6] = 0
    h2, x2 = hq.hq_residual_norm(H2, w, 1e-5, Y=Y2, w_post=w_post)
    for m in (0, 2, 4, 7):
        assert torch.equal(h2[m], h[m]) and torch.equal(x2[m], x[m])
    assert x2[1].isnan().all() and h2[3].isnan().any() and x2[3].isnan().all()
    assert torch.equal(h2[5], H2[5]) and (h2[6] == 0).all() and (x2[6] == 0).all()


def test_offsets_past_32_bits():
    ld, K = 1 << 30, 256
    big = torch.empty(2 * ld + K, dtype=F16, device="cuda")
    H = big.as_strided((3, K), (ld, 1))
    src = rows(3, K, F16, 1)
    H.copy_(src)
    w = weights(K, F16, 2)
    h, x = hq.hq_residual_norm(H, w, 1e-5, Y=src, H_out=H)
    want_h, want_x = hq.hq_residual_norm(src, w, 1e-5, Y=src)
    assert torch.equal(H, want_h) and torch.equal(x, want_x)
    q = hq.hq_norm_rotate_quant(H, w, 1e-5, 128)
    p = hq.hq_norm_rotate_quant(want_h, w, 1e-5, 128)
    assert torch.equal(q[0], p[0]) and torch.equal(q[1], p[1])


# ------------------------------------------------------- fused with the quantiser
def f32(t):
    return t.float().cpu().numpy()


def codes_fp32(H, Y, gate, alpha, w, off, group, signs, bits):
    """(h, q, amax) by the defining fp32 steps, in numpy."""
    h = f32(H)
    if Y is not None:
        p = f32(Y)
        if gate is not None:
            p = f32(gate) * p
        h = torch.from_numpy(h + np.float32(alpha) * p).to(H.dtype).float().numpy()
    v = h * (f32(w) + np.float32(off))
    M, K = v.shape
    if signs is not None:
        v = v * np.tile(signs.cpu().numpy().astype(np.float32), K // group)
    s = 1
    while s < group:
        t = v.reshape(M, K // (2 * s), 2, s)
        v = np.stack((t[:, :, 0] + t[:, :, 1], t[:, :, 0] - t[:, :, 1]), 2).reshape(M, K)
        s *= 2
    assert v.dtype == np.float32
    amax = np.abs(v).max(1)
    top = np.float32(127 if bits == 8 else 7)
    with np.errstate(divide="ignore"):
        inv = np.where(amax > 0, top / amax, np.float32(0)).astype(np.float32)
    return h, np.rint(v * inv[:, None]).astype(np.int8), amax


def unpack(Xq, bits):
    b = Xq.cpu().numpy()
    if bits == 8:
        return b
    b = b.view(np.int8)
    return np.stack(((b << 4) >> 4, b >> 4), 2).reshape(b.shape[0], -1)


def check_scale(sx, h, w, off, eps, group, amax, bits):
    top = 127 if bits == 8 else 7
    want = amax.astype(np.float64) / top / np.sqrt(group) / np.sqrt((h.astype(np.float64) ** 2).mean(1) + eps)
    # amax is exact; a division, 1/sqrt(g), two products: 4 u more than the row's statistic
    assert (np.abs(sx.cpu().numpy() - want) <= 34 * U * want).all()


QCASES = [
    # M, K, group, bits, stream, weights, block, gate, alpha, offset, signs
    (1, 32, 8, 4, F16, F16, False, None, 1.0, 0.0, False),
    (3, 96, 32, 8, BF16, F32, True, None, 1.0, 0.0, True),
    (2, 1056, 16, 4, BF16, BF16, True, "channel", 0.5, 1.0, True),
    (5, 1088, 64, 4, F16, F32, True, "token", 0.22, 0.0, True),
    (16, 4096, 128, 4, F16, F16, True, None, 1.0, 0.0, True),
    (70, 4096, 128, 8, BF16, BF16, True, None, 1.0, 0.0, False),
    (4, 8448, 256, 4, BF16, F32, True, "channel", 0.5, 0.0, True),
    (3, 1536, 512, 8, F16, F16, True, None, 1.0, 0.0, True),
    (9, 11264, 1024, 4, BF16, F16, False, None, 1.0, 1.0, True),
    (5, 6144, 2048, 4, F16, F32, True, "token", 1.0, 0.0, True),
    (6, 4096, 4096, 8, BF16, BF16, True, None, 1.0, 0.0, True),
    (2, 16384, 4096, 4, F16, F16, True, None, 1.0, 0.0, True),
    # several rows per CTA
    (9001, 96, 32, 4, F16, F16, True, "token", 1.0, 0.0, True),
    (5000, 1024, 8, 8, BF16, F32, False, None, 1.0, 0.0, True),
    (3001, 1536, 512, 4, BF16, BF16, True, "channel", 0.5, 0.0, True),
    (1501, 4096, 2048, 8, F16, F32, True, None, 1.0, 0.0, True),
]


@pytest.mark.parametrize("M,K,group,bits,xt,wt,block,gate,alpha,off,signs", QCASES)
@pytest.mark.parametrize("want_x", [False, True])
def test_norm_rotate_quant(M, K, group, bits, xt, wt, block, gate, alpha, off, signs, want_x):
    H, Y, w, _, g = inputs(M, K, xt, wt, False, gate, 8)
    H[0, K // 3] = 300.0          # an outlier channel
    Y, g = (Y, g) if block else (None, None)
    d = None
    if signs:
        d = (torch.randint(0, 2, (group,), generator=torch.Generator().manual_seed(1)) * 2 - 1).to(torch.int8)
        d[0] = 1
        d = d.cuda()
    Xq, sx, h, x = hq.hq_norm_rotate_quant(H, w, 1e-5, group, d, Y=Y, gate=g, alpha=alpha, w_offset=off, bits=bits,
                                           want_x=want_x)
    want_h, want_q, amax = codes_fp32(H, Y, g, alpha, w, off, group, d, bits)
    if block:
        assert np.array_equal(f32(h), want_h)
        check_stream(h, H, Y, None, g, alpha, off, 1e-5)
    else:
        assert h is None
    assert np.array_equal(unpack(Xq, bits), want_q)
    check_scale(sx, want_h, w, off, 1e-5, group, amax, bits)
    assert (x is not None) == want_x
    if want_x:
        check_normed(x, H if h is None else h, w, off, 1e-5)
    assert hq.hq_last_device_status() == 0
    # and in 64 bits: the codes times their scale are the rotated normed row to half
    # a step, plus the fp32 roundings of log2(group) + 3 stages of sums of up to
    # `group` terms and of the products around the code
    had = np.ones((1, 1))
    while had.shape[0] < group:
        had = np.block([[had, had], [had, -had]])
    v = want_h.astype(np.float64) * (f32(w).astype(np.float64) + off)
    v = v / np.sqrt((want_h.astype(np.float64) ** 2).mean(1, keepdims=True) + 1e-5)
    if d is not None:
        v = v * np.tile(d.cpu().numpy().astype(np.float64), K // group)
    u = (v.reshape(-1, group) @ had).reshape(M, K) / np.sqrt(group)
    step = sx.cpu().numpy().astype(np.float64)[:, None]
    size = np.abs(v).reshape(M, K // group, group).sum(2).repeat(group, 1) / np.sqrt(group)
    tol = 0.5 * step + (np.log2(group) + 3) * U * size + 40 * U * np.abs(u) + 3 * U * step * (127 if bits == 8 else 7)
    assert (np.abs(unpack(Xq, bits) * step - u) <= tol).all()


@pytest.mark.parametrize("gate", ["channel", "token"])
@pytest.mark.parametrize("M,K,group,bits", [(1500, 4096, 256, 4), (700, 8192, 4096, 8)])
def test_quantiser_in_place_over_several_rows_per_cta(M, K, group, bits, gate):
    """The operands of a CTA's next row are read before this row is finished: the rows
    of the block and of the stream that it overwrites are other ones."""
    H, Y, w, _, g = inputs(M, K, BF16, BF16, False, gate, 0)
    want = hq.hq_norm_rotate_quant(H, w, 1e-5, group, Y=Y, gate=g, alpha=0.5, bits=bits, want_x=True)
    want_h, want_q, amax = codes_fp32(H, Y, g, 0.5, w, 0.0, group, None, bits)
    assert np.array_equal(f32(want[2]), want_h) and np.array_equal(unpack(want[0], bits), want_q)
    check_scale(want[1], want_h, w, 0.0, 1e-5, group, amax, bits)
    check_normed(want[3], want[2], w, 0.0, 1e-5)
    got = hq.hq_norm_rotate_quant(H, w, 1e-5, group, Y=Y, gate=g, alpha=0.5, bits=bits, H_out=H, X=Y)
    assert got[2] is H and got[3] is Y
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_quantiser_rows_of_zeros_nan_and_infinity():
    M, K = 6, 2048
    H, w = rows(M, K, BF16, 3), weights(K, BF16, 4)
    a = hq.hq_norm_rotate_quant(H, w, 1e-5, 128)
    H2 = H.clone()
    H2[1] = 0
    H2[3, 5] = float("nan")
    H2[4, 9] = float("-inf")
    b = hq.hq_norm_rotate_quant(H2, w, 1e-5, 128)
    for m in (0, 2, 5):
        assert torch.equal(a[0][m], b[0][m]) and a[1][m] == b[1][m]
    assert (b[0][1] == 0).all() and b[1][1] == 0
    assert b[1][3].isnan() and b[1][4].isnan()
    H2[2] = float("nan")
    assert hq.hq_norm_rotate_quant(H2, w, 1e-5, 2048)[1][2].isnan()


def test_first_sign_must_be_plus_one():
    H, w = rows(2, 256, F16, 3), weights(256, F16, 4)
    d = torch.full((128,), -1, dtype=torch.int8, device="cuda")
    hq.hq_norm_rotate_quant(H, w, 1e-5, 128, d)
    assert hq.hq_last_device_status() == 1
    assert hq.hq_last_device_status() == 0


def test_python_refusals():
    H, Y, w, _, _ = inputs(4, 256, F16, F16, False, None, 0)
    with pytest.raises(ValueError):
        hq.hq_residual_norm(H, w.cpu(), 1e-5)
    with pytest.raises(ValueError):
        hq.hq_residual_norm(H, w[:128], 1e-5)
    with pytest.raises(ValueError):
        hq.hq_residual_norm(H, w, 1e-5, Y=Y.float())
    with pytest.raises(ValueError):
        hq.hq_residual_norm(H, w, 1e-5, Y=Y[:3])
    with pytest.raises(ValueError):
        hq.hq_residual_norm(H, w, 1e-5, Y=Y.t().contiguous().t())
    with pytest.raises(ValueError):
        hq.hq_residual_norm(H, w, 1e-5, Y=Y, w_post=w.float())
    with pytest.raises(hq.HQError):
        hq.hq_residual_norm(H, w, 1e-5, gate=w)        # a gate without a block
    with pytest.raises(ValueError):
        hq.hq_norm_rotate_quant(H, w, 1e-5, 128, Xq=torch.empty(4, 256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        hq.hq_norm_rotate_quant(H, w, 1e-5, 128, torch.ones(64, dtype=torch.int8, device="cuda"))
    with pytest.raises(hq.HQError):
        hq.hq_norm_rotate_quant(H.float(), w, 1e-5, 128)
    h, x = hq.hq_residual_norm(H[:0], w, 1e-5)
    assert x.shape == (0, 256)


# ------------------------------------------------------------- streams and graphs
def test_other_stream_and_captured_graph():
    H, Y, w, w_post, g = inputs(20, 4096, BF16, BF16, True, "token", 0)
    want = hq.hq_residual_norm(H, w, 1e-5, Y=Y, w_post=w_post, gate=g)
    want_q = hq.hq_norm_rotate_quant(H, w, 1e-5, 128, Y=Y)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = hq.hq_residual_norm(H, w, 1e-5, Y=Y, w_post=w_post, gate=g)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    Hs, Ys = torch.zeros_like(H), torch.zeros_like(Y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = hq.hq_residual_norm(Hs, w, 1e-5, Y=Ys, w_post=w_post, gate=g)
        outq = hq.hq_norm_rotate_quant(Hs, w, 1e-5, 128, Y=Ys)
    for k in range(2):
        Hs.copy_(H if k else H.flip(0))
        Ys.copy_(Y if k else Y.flip(0))
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    assert all(torch.equal(p, q) for p, q in zip(outq[:3], want_q[:3]))


# ------------------------------------------------------------------- with the layer
@pytest.mark.parametrize("M", [1, 16, 200])
@pytest.mark.parametrize("kind", ["w4a4", "w4a8", "offq", "post"])
def test_layer_on_the_stream(M, kind):
    K, N, r = 1024, 256, 16
    H, Y, w, w_post, _ = inputs(M, K, BF16, BF16, kind == "post", None, 0)
    W = 0.05 * rows(N, K, F32, 7)
    layer = hq.W4A4Linear.prepare(W, 128, 128, r, X_calib=rows(64, K, BF16, 8), act_bits=8 if kind == "w4a8" else 4,
                                  offq=kind == "offq")
    out, h = layer.forward_normed(H, w, 1e-5, block=Y, w_post=w_post, alpha=0.5)
    if kind in ("offq", "post"):
        want_h, x = hq.hq_residual_norm(H, w, 1e-5, Y=Y, w_post=w_post, alpha=0.5)
        want = layer(x)
    else:
        Xq, sx, want_h, _ = hq.hq_norm_rotate_quant(H, w, 1e-5, 128, Y=Y, alpha=0.5, bits=8 if kind == "w4a8" else 4)
        gemm = hq.w4a8_linear if kind == "w4a8" else hq.w4a4_linear
        want = gemm(Xq, sx, layer.Wq, layer.sw, layer.zw, 128, layer.Rq, layer.sr, layer.sal_idx)
    assert torch.equal(h, want_h) and torch.equal(out, want)
    # the quantised layer of the normed rows stays near the product it stands for: 4-bit
    # codes of 4-sigma rows have steps of about 0.5 sigma (an rms error of 0.15), the
    # weight groups' 15 steps over 5.5 sigma one of 0.11: together 0.18 of the product
    x = stream64(H, Y, w_post, None, 0.5, 0.0, 1e-5)[0]
    x = x * w.double() * inv_rms(x, 1e-5)
    ref = x @ W.double().T
    assert (out.double() - ref).norm() < 0.25 * ref.norm()
    alone, same = layer.forward_normed(H, w, 1e-5)
    assert same is H and alone.shape == (M, N)
