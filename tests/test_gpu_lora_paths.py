"""The adapters' kernels one by one: every class of ranks and pair of types in the
whole-tile and in the few-token form, with tokens that have adapters and tiles of
more than 32 tokens; the 16-bit terms that t is split into; and plans with tiles
that are refused or out of order, where every other tile is still done.
Tolerances as derived in test_gpu_lora unless stated."""
import numpy as np
import pytest
import torch

from test_gpu_lora import BF16, F16, F32, apply, batch, check, hq, randn

pytestmark = pytest.mark.gpu

TYPES = [(xt, yt) for xt in (F16, BF16) for yt in (F16, BF16, F32)]


def max_tiles(M, n):
    return M // 64 + min(n + 1, M)


def run(d, few):
    """apply() over rows that hold NaN before the call, so that an unwritten one fails."""
    M, n, N = d["X"].shape[0], d["A"].shape[0], d["B"].shape[1]
    assert (M < 16 * max_tiles(M, n)) == few          # which of the two forms the call takes
    Y = apply(d, Y=torch.full((M, N), float("nan"), dtype=d["yt"], device="cuda"))
    check(Y, d)
    bare = d["ids"] < 0
    assert torch.equal(Y[bare], d["base"][bare])
    assert hq.hq_last_device_status() == 0
    assert torch.equal(apply(d, Y=d["base"]), Y) and torch.equal(d["base"], Y)   # in place


@pytest.mark.parametrize("M,K,N,n,r,xt,yt,runs", [
    (1, 8, 8, 1, 8, F16, F16, 1),
    (1, 4096, 11008, 3, 16, F16, F16, 1),
    (64, 520, 256, 1, 16, BF16, BF16, 64),
    (65, 512, 296, 1, 40, F16, BF16, 65),
    (640, 200, 640, 1, 128, BF16, F16, 640),
    (800, 128, 192, 1, 200, F16, F32, 800),
])
@pytest.mark.parametrize("ragged", [False, True])
def test_batches_of_one_run(M, K, N, n, r, xt, yt, runs, ragged):
    d = batch(M, K, N, n, r, xt, yt, seed=M + K, ragged=ragged, runs=runs, bare=False)
    if ragged:   # a rank of its own, but one that does something
        d = batch(M, K, N, n, r, xt, yt, seed=M + K, ragged=False, runs=runs, bare=False)
        k = r - 3
        d["ranks"] = torch.full((n,), k, dtype=torch.int32, device="cuda")
        d["A"][:, k:] = float("nan")
        d["B"][:, :, k:] = float("nan")
    assert (d["ids"] >= 0).all()
    run(d, few=M < 16 * max_tiles(M, n))


@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("r", [8, 16, 24, 32, 40, 64, 96, 128, 256])
def test_whole_tiles_of_every_kind(r, xt, yt):
    # 2 adapters, runs that end inside a tile and inside a pair of tiles, K and N that end inside a stage and a block
    d = batch(730, 328, 200, 2, r, xt, yt, seed=r, ragged=False, runs=146)
    ids = d["ids"]
    assert (ids >= 0).sum() >= 146
    run(d, few=False)
    d = batch(730, 328, 200, 2, r, xt, yt, seed=r, ragged=False, runs=146, bare=False)
    d["ranks"] = torch.tensor([r - 5, (r + 1) // 2], dtype=torch.int32, device="cuda")
    for a, k in enumerate(d["ranks"].tolist()):
        d["A"][a, k:] = float("nan")
        d["B"][a, :, k:] = float("nan")
    run(d, few=False)


@pytest.mark.parametrize("xt,yt", TYPES)
@pytest.mark.parametrize("r", [8, 16, 24, 32, 40, 64, 96])
def test_few_token_form_with_full_tiles(r, xt, yt):
    # many adapters resident, runs of 64, 50, 33 and 17 tokens of a few of them
    M, K, N, n = 300, 328, 264, 40
    d = batch(M, K, N, n, r, xt, yt, seed=r, ragged=False)
    lens, slots = [64, 50, 33, 64, 17, 1, 64, 7], [3, 7, 11, 39, 0, 20, 3, -1]
    ids = np.repeat(slots, lens).astype(np.int32)
    assert len(ids) == M
    rng = np.random.default_rng(r)
    d = {**d, "ids": torch.from_numpy(ids).cuda(), "A": randn((n, r, K), xt, r, K ** -0.5), "B": randn((n, N, r), xt, r + 1, 0.3)}
    run(d, few=True)
    d["ids"] = torch.from_numpy(rng.permutation(ids)).cuda()     # the same, the tokens of a tile scattered
    d["ranks"] = torch.from_numpy(rng.integers(1, r + 1, n).astype(np.int32)).cuda()
    for a, k in enumerate(d["ranks"].tolist()):
        d["A"][a, k:] = float("nan")
        d["B"][a, :, k:] = float("nan")
    run(d, few=True)


def bf16_terms(t, n):
    """The sum of t's first n bf16 terms."""
    left, total = t.clone(), torch.zeros_like(t)
    for _ in range(n):
        term = left.bfloat16().float()
        total, left = total + term.double(), left - term
    return total


@pytest.mark.parametrize("xt", [BF16, F16])
@pytest.mark.parametrize("r", [16, 48, 96])
def test_terms_of_t_in_an_fp32_result(r, xt):
    """X and B with one non-zero per row: t = fl32(scale * a) and Y = t times a power
    of two, so that nothing but the terms of t and the accumulator's last bits
    can be off.  Three bf16 terms hold t exactly (3 x 8 bits), two fp16 ones to
    2^-22 of t; a product adds one non-zero to the accumulator, at most two
    truncations of 2^-23 for each of the three (two) terms."""
    M, K, N = 700, 64, 128
    rng = np.random.default_rng(r)
    X = torch.zeros(M, K)
    j = torch.from_numpy(rng.integers(0, K, M))
    X[torch.arange(M), j] = 1.0
    A = torch.randn(1, r, K, generator=torch.Generator().manual_seed(r)).to(xt)
    B = torch.zeros(1, N, r)
    i, e = torch.arange(N) % r, torch.from_numpy(rng.integers(-3, 4, N))
    B[0, torch.arange(N), i] = torch.exp2(e.float())
    scale = torch.tensor([1.2345678], dtype=F32)
    t = (A[0].float() * scale)[:, j].T.contiguous()                # [M, r]; fp32 products, rounded once
    want = (t.double()[:, i] * torch.exp2(e.double())).cuda()
    ids = torch.zeros(M, dtype=torch.int32, device="cuda")
    order, tiles = hq.hq_lora_plan(ids, 1)
    Y = hq.hq_lora_apply(X.to(xt).cuda(), A.cuda(), B.to(xt).cuda(), order, tiles, scales=scale.cuda(), out_dtype=F32)
    tol = 6 * 2.0 ** -23 if xt == BF16 else 2.0 ** -22 + 4 * 2.0 ** -23
    err = (Y.double() - want).abs()
    # fp16 terms of a row share one power of two: what is left below the second one's spacing
    top = t.abs().max(1).values.double().cuda()[:, None] * torch.exp2(e.double()).cuda()
    floor = 0.0 if xt == BF16 else 2.0 ** -37 * top
    assert (err <= tol * want.abs() + floor).all(), (err / want.abs()).max()
    if xt == BF16:   # the bound notices a missing term, and three terms are enough
        assert torch.equal(bf16_terms(t, 3), t.double())
        two = (bf16_terms(t, 2) - t.double()).abs()
        assert (two > 2 * tol * t.abs()).any()


@pytest.mark.parametrize("M,n,r", [(300, 40, 32), (300, 40, 96), (700, 2, 32), (700, 2, 128)])
def test_over_the_input(M, n, r):
    """K = N and the result written over X, in every form."""
    d = batch(M, 264, 264, n, r, BF16, BF16, seed=4, ragged=True, runs=50)
    d["base"] = None
    want = apply(d, out_dtype=BF16)
    check(want, d, base=False)
    X = torch.full((M + 2, 272), 9.0, dtype=BF16, device="cuda")
    X[:M, :264] = d["X"]
    d["X"] = X[:M, :264]
    assert apply(d, Y=d["X"]) is d["X"]
    assert torch.equal(d["X"], want) and (X[M:] == 9).all() and (X[:, 264:] == 9).all()
