"""Shared prefixes that give every CTA of the prefix kernels many 128-key tiles: the rings of K and V tiles come
round several times, row tiles end in the middle of a CTA's run (its query rows are loaded anew), and the maxima
grow along the keys, so that the output in tensor memory and the sums are scaled again and again.  The tolerance is
test_paged_attention_gpu's, counted from the formula."""
import pytest

import epilogue_chains_gb300 as fc
from test_paged_attention_gpu import check, make

pytestmark = pytest.mark.gpu
CTAS = 152


def tiles(batch, group, hk, D, prefix):
    """128-key tiles of all row tiles of a call."""
    rows = 256 if batch * group > 128 and D <= 128 else 128
    return hk * -(-batch * group // rows) * -(-prefix // 128)


def grow(p):
    """Scale the prefix's keys by 1, 1.75, ... 6.25 from tile to tile, eight tiles over: a row's scores spread as
    far as its keys are long, so its maximum rises by several powers of two at most steps."""
    page = p["k"].shape[2]
    ids = p["ptable"].long()
    k = p["k"][ids].transpose(0, 1).reshape(p["k"].shape[1], -1, p["k"].shape[3])
    import torch
    at = torch.arange(k.shape[1], device="cuda")
    k = (k.float() * (1 + 0.75 * (at // 128 % 8))[:, None]).to(k.dtype)
    p["k"][ids] = k.view(k.shape[0], len(ids), page, -1).transpose(0, 1)
    return p


def rises(p):
    """The largest rise, in powers of two, of a row's maximum over the keys before a tile to that of the tile, as
    seen by a run of tiles that starts eight before."""
    import torch
    ids = p["ptable"].long()
    hk, D = p["k"].shape[1], p["k"].shape[3]
    k = p["k"][ids].transpose(0, 1).reshape(hk, -1, D)[:, :p["prefix"] // 128 * 128].float()
    q = p["q"][0].view(hk, -1, D).float()
    s = (q @ k.transpose(1, 2) * p["scale"] * 1.4427).view(hk, q.shape[1], -1, 128).amax(3)
    seen = s[:, :, 0:8].cummax(2).values
    return float((s[:, :, 1:8] - seen[:, :, :7]).max())


# rows per key/value head: up to 128 (one row tile), or more (two at a time where D <= 128)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("batch", [3, 40, 70])
def test_many_tiles_per_cta(cuda_device, dtype, D, batch):
    hq, hk, prefix = 32, 8, 16384 - 37
    n = tiles(batch, hq // hk, hk, D, prefix)
    assert n > 6 * CTAS and n % CTAS                       # runs of several tiles, and row tiles that end inside one
    p = grow(make([(41 * b) % 200 for b in range(batch)], hq, hk, D, 64, dtype, prefix=prefix, seed=batch + D))
    assert rises(p) > 8                                    # past the 2^8 by which a maximum may grow before a rescale
    check(p)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_runs_across_row_tiles(cuda_device, dtype, D):
    """Short items: a CTA's run holds parts of several heads and row tiles."""
    hq, hk, prefix = 64, 16, 600
    for batch in (65, 130):                                # 260 and 520 rows per head
        assert tiles(batch, hq // hk, hk, D, prefix) > CTAS
        check(grow(make([b % 3 for b in range(batch)], hq, hk, D, 16, dtype, prefix=prefix, seed=batch + D)))
