"""Adapter plans with tiles that are refused or stand out of order: every other tile is
still done.  The rows hold a mark before each call, so that one left out shows."""
import numpy as np
import pytest
import torch

from test_gpu_lora import BF16, F16, F32, apply, batch, hq

pytestmark = pytest.mark.gpu

SENTINEL = 9.0


def positions_done(tiles, bad):
    """Positions in the order of all tiles but those in `bad`."""
    pos = []
    for k, (a, s, c) in enumerate(tiles):
        if c and k not in bad:
            pos += range(s, s + c)
    return pos


@pytest.mark.parametrize("yt", [F16, F32])
@pytest.mark.parametrize("M,n,runs", [(400, 3, 40), (500, 1, 500), (1500, 2, 500)])
def test_a_refused_tile_takes_no_other_with_it(M, n, runs, yt):
    d = batch(M, 128, 72, n, 16, F16, yt, ragged=False, runs=runs, bare=False)
    order, tiles = hq.hq_lora_plan(d["ids"], n)
    want = apply(d, (order, tiles))
    rows = tiles.tolist()
    used = sum(c > 0 for _, _, c in rows)
    for k in sorted({0, 1, 2, used // 2, used - 1}):
        for entry in ([n, 0, 64], [0, M - 1, 2], [0, -1, 4], [n - 1, 0, 65], [rows[k][0], rows[k][1], 65],
                      [n - 1, 5, -3], [n - 1, 2 ** 31 - 1, 64]):
            bad = tiles.clone()
            bad[k] = torch.tensor(entry, dtype=torch.int32)
            out = torch.full((M, 72), SENTINEL, dtype=yt, device="cuda")
            apply(d, (order, bad), Y=out)
            assert hq.hq_last_device_status() == 1, entry
            done = torch.zeros(M, dtype=torch.bool, device="cuda")
            done[order[positions_done(rows, {k})].long()] = True
            assert torch.equal(out[done], want[done]), (k, entry)
            assert (out[~done] == SENTINEL).all(), (k, entry)


@pytest.mark.parametrize("yt", [BF16, F32])
def test_tiles_in_any_order(yt):
    """Every tile is done wherever it stands: swapped, reversed, with unused entries between."""
    M, n = 1500, 2
    d = batch(M, 128, 72, n, 16, BF16, yt, ragged=False, runs=300, bare=False)
    order, tiles = hq.hq_lora_plan(d["ids"], n)
    want = apply(d, (order, tiles))
    used = int((tiles[:, 2] > 0).sum())
    rng = np.random.default_rng(0)
    orders = [torch.arange(len(tiles)).flip(0)] + [torch.from_numpy(rng.permutation(len(tiles))) for _ in range(4)]
    swapped = torch.arange(len(tiles))
    swapped[2], swapped[3] = 3, 2
    assert used > 20
    for p in orders + [swapped]:
        out = torch.full((M, 72), SENTINEL, dtype=yt, device="cuda")
        apply(d, (order, tiles[p.cuda()].contiguous()), Y=out)
        assert torch.equal(out, want)
    assert hq.hq_last_device_status() == 0
    # and a token that stands in no tile keeps its row
    part = tiles.clone()
    part[1] = torch.tensor([-1, 0, 0], dtype=torch.int32)
    out = torch.full((M, 72), SENTINEL, dtype=yt, device="cuda")
    apply(d, (order, part), Y=out)
    left = order[64:128].long()
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    keep[left] = False
    assert torch.equal(out[keep], want[keep]) and (out[left] == SENTINEL).all()
