"""The adapter plan and the low-rank adapters beside a layer, on the GPU against
plain implementations (the plan exactly, the product in 64 bits).

Tolerance of the product, S = sum_k |x_k a_k| and D = sum_j |t_j b_j|:
 * t: an MMA adds 16 exact products to the accumulator with at most 17
   truncations of 2^-23 of S; a warp does at most one per slab of 64 channels (a
   block has all of K or a part of it), then 4 warps and up to 8 blocks are
   added: (17 slabs + 12) 2^-23 S, and the scale's product 2^-24;
 * t b: with 16-bit Y t is two bf16 terms (a nearest bf16 is off by 2^-9, twice:
   2^-18 of t) and an fp16 b two exact ones, whose product of both second terms
   (2^-18) is left out: 2^-17 D.  With fp32 Y t is three terms (2^-27) and the
   product left out 2^-27: 2^-26 D.  At most 5 such MMAs of 17 truncations per
   16 rank positions: 85 ceil(r / 16) 2^-23 D;
 * the sum with the base row one rounding (2^-24 of its size), the result half a
   step of its type.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

hq = pytest.importorskip("w4a4_bit_gemm_hq_b200.hq") if torch.cuda.is_available() else None

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


# ------------------------------------------------------------------------- the plan
def plan_plain(ids, n):
    ids = np.where((ids < -1) | (ids >= n), -1, ids)
    order = np.argsort(ids, kind="stable").astype(np.int32)
    M = len(ids)
    tiles = np.tile(np.array([-1, 0, 0], np.int32), (M // 64 + min(n + 1, M), 1))
    t = at = 0
    for a in range(-1, n):
        c = int((ids == a).sum())
        for s in range(0, c, 64):
            tiles[t] = (a, at + s, min(64, c - s))
            t += 1
        at += c
    return order, tiles


@pytest.mark.parametrize("M,n,kind", [
    (1, 0, "random"), (1, 1, "random"), (1, 1022, "random"), (2, 3, "none"), (16, 64, "random"), (31, 2, "random"),
    (32, 1, "one"), (33, 5, "random"), (64, 4, "one"), (65, 4, "one"), (127, 7, "runs"), (1000, 1022, "random"),
    (1024, 31, "random"), (1025, 32, "runs"), (4096, 8, "runs"), (4099, 3, "none"), (8192, 1, "one"),
    (20000, 300, "random"), (100003, 511, "runs"), (300000, 2, "random"),
])
def test_plan(M, n, kind):
    rng = np.random.default_rng(M + n)
    if kind == "none":
        ids = np.full(M, -1)
    elif kind == "one":
        ids = np.full(M, n - 1)
    elif kind == "runs":
        ids = np.repeat(rng.integers(-1, n, M // 37 + 1), 37)[:M]
    else:
        ids = rng.integers(-1, n, M)
    ids = ids.astype(np.int32)
    order, tiles = hq.hq_lora_plan(torch.from_numpy(ids).cuda(), n)
    want = plan_plain(ids, n)
    assert np.array_equal(order.cpu().numpy(), want[0])
    assert np.array_equal(tiles.cpu().numpy(), want[1])
    assert hq.hq_last_device_status() == 0


def test_plan_of_bad_ids():
    ids = np.array([3, -1, 4, -2, 0, 2 ** 31 - 1, 0, -2 ** 31], np.int32)
    order, tiles = hq.hq_lora_plan(torch.from_numpy(ids).cuda(), 4)
    want = plan_plain(ids, 4)
    assert np.array_equal(order.cpu().numpy(), want[0]) and np.array_equal(tiles.cpu().numpy(), want[1])
    assert hq.hq_last_device_status() == 1
    assert hq.hq_last_device_status() == 0


def test_plan_of_nothing():
    order, tiles = hq.hq_lora_plan(torch.empty(0, dtype=torch.int32, device="cuda"), 4)
    assert order.shape == (0,) and tiles.shape == (0, 3)


# --------------------------------------------------------------------- the adapters
def randn(shape, dt, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn(*shape, generator=g, device="cuda")).to(dt)


def batch(M, K, N, n, r, xt, yt, seed=0, ragged=True, runs=1, bare=True):
    rng = np.random.default_rng(seed)
    ids = np.repeat(rng.integers(-1 if bare else 0, n, -(-M // runs)), runs)[:M].astype(np.int32)
    d = {"yt": yt, "ids": torch.from_numpy(ids).cuda(), "X": randn((M, K), xt, seed), "A": randn((n, r, K), xt, seed + 1, K ** -0.5),
         "B": randn((n, N, r), xt, seed + 2, 0.3), "base": randn((M, N), yt, seed + 3),
         "scales": 0.5 + torch.rand(n, generator=torch.Generator().manual_seed(seed)).cuda(), "ranks": None}
    if ragged:
        ranks = rng.integers(0, r + 1, n).astype(np.int32)
        d["ranks"] = torch.from_numpy(ranks).cuda()
        for a in range(n):   # what lies behind an adapter's rank is not to be used
            d["A"][a, ranks[a]:] = float("nan")
            d["B"][a, :, ranks[a]:] = float("nan")
    for a in range(n):       # nor is an adapter that no token has
        if not (ids == a).any():
            d["A"][a] = float("nan")
            d["B"][a] = float("nan")
    return d


def reference(d, base=True):
    """(Y, bound of the error before the last rounding) in 64 bits."""
    X, A, B, ids = d["X"].double(), d["A"], d["B"], d["ids"]
    M, K = X.shape
    N = B.shape[1]
    y = d["base"].double().clone() if base else torch.zeros(M, N, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(y)
    slabs = -(-K // 64)
    steps = 17 * slabs + 12
    split = 2.0 ** -26 if d["yt"] == F32 else 2.0 ** -17
    for a in range(A.shape[0]):
        rows = (ids == a).nonzero().flatten()
        k = A.shape[1] if d["ranks"] is None else int(d["ranks"][a])
        if not rows.numel() or not k:
            continue
        s = float(d["scales"][a]) if d["scales"] is not None else 1.0
        At, Bt = A[a, :k].double().T, B[a, :, :k].double().T
        t = s * (X[rows] @ At)
        et = steps * 2.0 ** -23 * s * (X[rows].abs() @ At.abs()) + 2.0 ** -24 * t.abs()
        y[rows] += t @ Bt
        tol[rows] = et @ Bt.abs() + (split + 85 * -(-k // 16) * 2.0 ** -23) * (t.abs() + et) @ Bt.abs()
    return y, tol + 2.0 ** -24 * y.abs()


def check(Y, d, base=True):
    want, tol = reference(d, base)
    dt = Y.dtype
    tol = tol + (want.abs() + tol) * (torch.finfo(dt).eps / 2) + (2.0 ** -25 if dt == F16 else 0.0)
    err = (Y.double() - want).abs()
    assert not Y.isnan().any() and (err <= tol).all(), (err / tol).max()


def apply(d, plan=None, **kw):
    order, tiles = hq.hq_lora_plan(d["ids"], d["A"].shape[0]) if plan is None else plan
    kw = {"ranks": d["ranks"], "scales": d["scales"], "base": d["base"], **kw}
    return hq.hq_lora_apply(d["X"], d["A"], d["B"], order, tiles, **kw)


@pytest.mark.parametrize("M,K,N,n,r,xt,yt,ragged,runs", [
    (1, 8, 8, 1, 8, F16, F16, False, 1),
    (1, 4096, 11008, 3, 16, F16, F16, False, 1),
    (3, 24, 24, 2, 8, BF16, F32, True, 1),
    (16, 4096, 1032, 64, 32, F16, F32, True, 1),
    (17, 72, 264, 5, 24, BF16, BF16, True, 1),
    (64, 520, 256, 1, 16, BF16, BF16, False, 64),
    (65, 512, 296, 1, 40, F16, BF16, True, 65),
    (200, 1000, 512, 4, 64, F16, F32, True, 50),
    (333, 2048, 4096, 7, 72, BF16, F16, True, 11),
    (500, 136, 88, 30, 128, F16, F16, True, 1),
    (1000, 4096, 1024, 3, 256, BF16, F32, True, 100),
    (2048, 11008, 512, 8, 32, BF16, BF16, False, 256),
    # whole tiles: odd and even numbers of them per adapter, last ones not full, every rank class
    (700, 256, 8, 2, 8, BF16, BF16, False, 100),
    (1111, 128, 72, 3, 24, F16, F16, True, 193),
    (900, 64, 200, 2, 56, BF16, F32, True, 320),
    (1500, 384, 136, 4, 96, F16, BF16, True, 130),
    (640, 200, 640, 1, 128, BF16, F16, True, 640),
    (700, 128, 320, 2, 192, BF16, F32, True, 70),
    (800, 128, 192, 1, 200, F16, F32, True, 800),
    (513, 128, 264, 2, 256, BF16, BF16, True, 171),
    (513, 128, 264, 2, 256, F16, F32, True, 171),
])
def test_apply(M, K, N, n, r, xt, yt, ragged, runs):
    d = batch(M, K, N, n, r, xt, yt, seed=M + K, ragged=ragged, runs=runs)
    Y = apply(d)
    check(Y, d)
    bare = d["ids"] < 0
    assert torch.equal(Y[bare], d["base"][bare])
    assert hq.hq_last_device_status() == 0
    assert torch.equal(apply(d), Y)          # the same bits every time
    assert torch.equal(apply(d, Y=d["base"]), Y) and torch.equal(d["base"], Y)   # in place


@pytest.mark.parametrize("M,K,N,n,r,xt,yt,ragged,runs", [
    (2100, 96, 1320, 3, 24, F16, F32, True, 150),
    (2100, 96, 1320, 3, 24, BF16, F32, False, 150),
    (2100, 128, 1320, 3, 72, BF16, BF16, False, 150),
    (2500, 64, 2056, 2, 200, F16, F16, True, 1),
    (2100, 64, 1320, 3, 192, BF16, F32, False, 90),
])
def test_apply_with_ctas_for_the_whole_gpu(M, K, N, n, r, xt, yt, ragged, runs):
    """Two CTAs per SM with fewer base rows asked for ahead, or one round of larger CTAs."""
    test_apply(M, K, N, n, r, xt, yt, ragged, runs)


@pytest.mark.parametrize("xt", [F16, BF16])
def test_fp32_rows_between_sectors(xt):
    """Rows of Y and base that start on 16-byte boundaries only, and columns that end inside a block."""
    M, N = 700, 328
    d = batch(M, 128, N, 2, 24, xt, F32, seed=9, ragged=True, runs=100)
    want = apply(d)
    check(want, d)
    base = torch.full((M, N + 4), 7.0, device="cuda")
    base[:, :N] = d["base"]
    Y = torch.full((M, N + 12), 7.0, device="cuda")
    assert torch.equal(apply(d, base=base[:, :N], Y=Y[:, 4:N + 4]), want)
    assert (Y[:, :4] == 7).all() and (Y[:, N + 4:] == 7).all()
    assert torch.equal(apply(d, base=base[:, :N], Y=base[:, :N]), want) and (base[:, N:] == 7).all()


@pytest.mark.parametrize("M,runs", [(130, 13), (5, 1)])
@pytest.mark.parametrize("yt", [F16, BF16, F32])
def test_no_base_no_ranks_no_scales(yt, M, runs):
    d = batch(M, 256, 136, 3, 16, BF16, yt, ragged=False, runs=runs)
    d["scales"] = None
    Y = apply(d, base=None, out_dtype=yt)
    check(Y, d, base=False)
    assert (Y[d["ids"] < 0] == 0).all()


@pytest.mark.parametrize("n,bare", [(0, True), (4, True)])
def test_no_token_has_an_adapter(n, bare):
    M, K, N = 70, 64, 72
    ids = torch.full((M,), -1, dtype=torch.int32, device="cuda")
    X, base = randn((M, K), F16, 1), randn((M, N), F16, 2)
    A, B = randn((n, 8, K), F16, 3), randn((n, N, 8), F16, 4)
    order, tiles = hq.hq_lora_plan(ids, n)
    assert torch.equal(hq.hq_lora_apply(X, A, B, order, tiles, base=base), base)
    assert (hq.hq_lora_apply(X, A, B, order, tiles) == 0).all()


def test_strided_rows_and_nothing_else_written():
    d = batch(77, 200, 136, 3, 24, F16, F16, runs=7)
    want = apply(d)
    xbuf = torch.full((80, 264), 9.0, dtype=F16, device="cuda")
    xbuf[:77, :200] = d["X"]
    ybuf = torch.full((80, 160), 9.0, dtype=F16, device="cuda")
    bbuf = torch.full((80, 144), 9.0, dtype=F16, device="cuda")
    bbuf[:77, :136] = d["base"]
    d["X"], d["base"] = xbuf[:77, :200], bbuf[:77, :136]
    work = torch.full((77 * 24 + 40,), 5.0, dtype=F32, device="cuda")
    Y = apply(d, Y=ybuf[:77, :136], workspace=work)
    assert torch.equal(Y, want)
    assert (ybuf[77:] == 9).all() and (ybuf[:, 136:] == 9).all() and (work[77 * 24:] == 5).all()


@pytest.mark.parametrize("M,xt", [(50, BF16), (50, F16), (400, BF16), (400, F16)])
def test_values_of_one_token_stay_with_it(M, xt):
    d = batch(M, 192, 64, 3, 16, xt, BF16, runs=M // 10)
    want = apply(d)
    ids = d["ids"].tolist()
    odd = [m for m in range(M) if ids[m] >= 0][:2] + [m for m in range(M) if ids[m] < 0][:1]
    d["X"][odd[0], 7] = float("nan")
    d["X"][odd[1], 100] = float("inf")
    d["X"][odd[2]] = float("nan")             # a token without an adapter: its input is not used
    got = apply(d)
    for m in range(M):
        if m not in odd[:2]:
            assert torch.equal(got[m], want[m])
    if d["ranks"][ids[odd[0]]] > 0:
        assert got[odd[0]].isnan().all()
    if d["ranks"][ids[odd[1]]] > 0:
        assert not got[odd[1]].isfinite().any()


def test_offsets_past_32_bits():
    # one adapter behind 2^31 elements of A and of B, rows of X and Y 2^30 elements apart
    M, K, N, r, n = 3, 131072, 131072, 64, 300
    A = torch.empty(n, r, K, dtype=F16, device="cuda")
    B = torch.empty(n, N, r, dtype=F16, device="cuda")
    A[-1], B[-1] = randn((r, K), F16, 1, K ** -0.5), randn((N, r), F16, 2, 0.3)
    ids = torch.tensor([n - 1, -1, n - 1], dtype=torch.int32, device="cuda")
    big = torch.empty(2 * (1 << 30) + K, dtype=F16, device="cuda")
    X = big.as_strided((M, K), (1 << 30, 1))
    src = randn((M, K), F16, 3)
    X.copy_(src)
    order, tiles = hq.hq_lora_plan(ids, n)
    Y = hq.hq_lora_apply(X, A, B, order, tiles, Y=X)      # K = N: the result over the input's rows
    d = {"X": src, "A": A[-1:], "B": B[-1:], "ids": torch.where(ids < 0, -1, 0), "ranks": None, "scales": None, "yt": F16}
    check(Y, d, base=False)


def test_bad_plans_are_not_read_through():
    d = batch(40, 128, 64, 3, 16, F16, F16, ragged=False, runs=4, bare=False)
    order, tiles = hq.hq_lora_plan(d["ids"], 3)
    want = apply(d, (order, tiles))
    bad = order.clone()
    bad[0], bad[1] = -5, 1 << 30
    out = torch.full((40, 64), 9.0, dtype=F16, device="cuda")
    apply(d, (bad, tiles), Y=out)
    assert hq.hq_last_device_status() == 1
    skipped = order[:2].long()
    keep = torch.ones(40, dtype=torch.bool, device="cuda")
    keep[skipped] = False
    assert torch.equal(out[keep], want[keep]) and (out[skipped] == 9).all()
    for entry in ([7, 0, 40], [0, 39, 2], [0, -1, 4], [1, 0, 65], [1, 5, -3]):
        bad = tiles.clone()
        bad[0] = torch.tensor(entry, dtype=torch.int32)
        out.fill_(9)
        apply(d, (order, bad), Y=out)
        assert hq.hq_last_device_status() == 1, entry
        first = order[:int(tiles[0, 2])].long()
        assert (out[first] == 9).all()


def test_bad_plans_of_whole_tiles():
    M = 400
    d = batch(M, 128, 72, 3, 16, F16, F16, ragged=False, runs=40, bare=False)
    order, tiles = hq.hq_lora_plan(d["ids"], 3)
    want = apply(d, (order, tiles))
    bad = order.clone()
    bad[0], bad[M - 1] = -5, 1 << 30
    out = torch.full((M, 72), 9.0, dtype=F16, device="cuda")
    apply(d, (bad, tiles), Y=out)
    assert hq.hq_last_device_status() == 1
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    keep[order[0].long()] = keep[order[M - 1].long()] = False
    assert torch.equal(out[keep], want[keep]) and (out[~keep] == 9).all()
    others = d["ids"] != int(tiles[0, 0])
    for entry in ([7, 0, 64], [0, M - 1, 2], [0, -1, 4], [1, 0, 65], [1, 5, -3], [2, 2 ** 31 - 1, 64]):
        bad = tiles.clone()
        bad[0] = torch.tensor(entry, dtype=torch.int32)
        apply(d, (order, bad), Y=out)
        assert hq.hq_last_device_status() == 1, entry
        assert torch.equal(out[others], want[others])


@pytest.mark.parametrize("M", [20, 300])
def test_ranks_outside_are_clamped_and_reported(M):
    d = batch(M, 64, 64, 2, 8, F16, F16, ragged=False, bare=False)
    want = apply(d)
    d["ranks"] = torch.tensor([100, 8], dtype=torch.int32, device="cuda")
    assert torch.equal(apply(d), want)
    assert hq.hq_last_device_status() == 1
    d["ranks"] = torch.tensor([-3, 8], dtype=torch.int32, device="cuda")
    got = apply(d)
    assert hq.hq_last_device_status() == 1
    zero = d["ids"] == 0
    assert torch.equal(got[zero], d["base"][zero]) and torch.equal(got[~zero], want[~zero])


def test_two_streams_and_captured_graph():
    d, e = batch(300, 512, 256, 4, 32, BF16, BF16, seed=1, runs=10), batch(90, 512, 256, 4, 16, BF16, BF16, seed=2)
    want = apply(d), apply(e)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s):
            a = apply(d)
        with torch.cuda.stream(t):
            b = apply(e)
    torch.cuda.synchronize()
    assert torch.equal(a, want[0]) and torch.equal(b, want[1])
    ids = d["ids"].clone()
    cap = {**d, "ids": ids.fill_(-1)}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = apply(cap)
    graph.replay()
    assert torch.equal(out, d["base"])
    ids.copy_(d["ids"])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0])


def test_python_refusals():
    d = batch(10, 64, 64, 2, 8, F16, F16)
    plan = hq.hq_lora_plan(d["ids"], 2)
    with pytest.raises(ValueError):
        hq.hq_lora_plan(d["ids"].long(), 2)
    with pytest.raises(ValueError):
        apply(d, hq.hq_lora_plan(d["ids"], 3))            # the plan of another number of adapters
    with pytest.raises(ValueError):
        apply({**d, "A": d["A"].bfloat16()}, plan)
    with pytest.raises(ValueError):
        apply({**d, "B": d["B"][:, :56]}, plan)
    with pytest.raises(ValueError):
        apply({**d, "base": d["base"].float()}, plan, Y=torch.empty_like(d["base"]))
    with pytest.raises(ValueError):
        apply({**d, "ranks": torch.zeros(2, dtype=torch.int64, device="cuda")}, plan)
    with pytest.raises(ValueError):
        apply({**d, "scales": d["scales"].cpu()}, plan)
    with pytest.raises(hq.HQError):
        apply(d, plan, workspace=torch.empty(10, dtype=F32, device="cuda"))
    with pytest.raises(hq.HQError):
        apply({**d, "X": randn((10, 64), F32, 1), "A": d["A"].float(), "B": d["B"].float(), "base": d["base"]}, plan)
    assert apply({**d, "X": d["X"][:0], "base": d["base"][:0], "ids": d["ids"][:0]}).shape == (0, 64)


# ------------------------------------------------------------------- with the layer
@pytest.mark.parametrize("kind", ["w4a4", "w4a8", "offq"])
@pytest.mark.parametrize("M", [1, 16, 150])
def test_layer_with_adapters(kind, M):
    K, N, n, r = 512, 256, 3, 16
    d = batch(M, K, N, n, r, BF16, BF16, seed=5, bare=M > 1)
    layer = hq.W4A4Linear.prepare(randn((N, K), F32, 9, 0.05), 128, 128, 0, act_bits=8 if kind == "w4a8" else 4,
                                  offq=kind == "offq")
    plan = hq.hq_lora_plan(d["ids"], n)
    with pytest.raises(ValueError):
        layer(d["X"], plan=plan)
    with pytest.raises(ValueError):
        layer.set_adapters(d["A"], d["B"][:, :-8])
    layer.set_adapters(d["A"], d["B"], d["ranks"], d["scales"])
    d["base"] = layer(d["X"])
    Y = layer(d["X"], plan=plan)
    assert torch.equal(Y, apply(d, plan))
    check(Y, d)
    # from the residual stream: the adapters take the normed rows
    H, w = randn((M, K), BF16, 11, 2.0), randn((K,), BF16, 12)
    Y2, _ = layer.forward_normed(H, w, 1e-5, block=d["X"], plan=plan)
    base2, h2 = layer.forward_normed(H, w, 1e-5, block=d["X"])
    _, x2 = hq.hq_residual_norm(H, w, 1e-5, Y=d["X"])
    assert torch.equal(Y2, apply({**d, "X": x2, "base": base2}, plan))
    layer.set_adapters(None, None)
    assert torch.equal(layer(d["X"]), d["base"])


def test_a_decoder_step_captured():
    """Plan, norm + quantiser + layer + adapters, and the next layer's norm on the
    updated stream, as one captured step: replays with other tokens and other
    adapters give what the calls give one by one."""
    M, K, n, r = 24, 1024, 4, 16
    d = batch(M, K, K, n, r, BF16, BF16, seed=3)
    up = hq.W4A4Linear.prepare(randn((K, K), F32, 20, 0.03), 128, 128, 16, X_calib=randn((64, K), BF16, 21))
    down = hq.W4A4Linear.prepare(randn((K, K), F32, 22, 0.03), 128, 128, 16, X_calib=randn((64, K), BF16, 23), act_bits=8)
    up.set_adapters(d["A"], d["B"], d["ranks"], d["scales"])
    down.set_adapters(d["A"], d["B"], d["ranks"], d["scales"])
    w1, w2, w3 = (1 + randn((K,), BF16, 24 + k, 0.2) for k in range(3))

    def step(H, block, ids):
        plan = hq.hq_lora_plan(ids, n)
        y, h = up.forward_normed(H, w1, 1e-5, block=block, plan=plan)
        z, h = down.forward_normed(h, w2, 1e-5, block=y, alpha=0.5, plan=plan)
        return hq.hq_residual_norm(h, w3, 1e-5, Y=z, w_post=w1)

    H, block, ids = torch.zeros(M, K, dtype=BF16, device="cuda"), torch.zeros(M, K, dtype=BF16, device="cuda"), d["ids"].clone()
    step(H, block, ids)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(H, block, ids)
    for seed in range(3):
        H.copy_(randn((M, K), BF16, 30 + seed, 2.0))
        block.copy_(randn((M, K), BF16, 40 + seed))
        ids.copy_(torch.randint(-1, n, (M,), generator=torch.Generator().manual_seed(seed)).to(torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = step(H, block, ids)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert got[1].isfinite().all()
    assert hq.hq_last_device_status() == 0
