"""Values that are not finite, at keys in use: the mask keeps them from the rows that do not see them.  Each column of V has one
such value, at a key of its own.  A row that sees it has it in that column: an infinity or NaN times a positive weight.  Every
other output is what the formula gives with a zero in its place, within the tolerance of reference(), or, where a sequence has
no such value, the same bits as without them in the batch."""
import math

import pytest

import epilogue_chains_gb300 as fc
from test_prompt_attention_gpu import make, reference, run

pytestmark = pytest.mark.gpu


def check(seqs, hq, hk, D, page, dtype, seed=0, std=1.0, room=0):
    """Of every sequence and head each column gets a value that is not finite, at keys that are spread over the sequence, near
    the ends of blocks and of tiles and over all of its new tokens."""
    import torch
    p = make(seqs, hq, hk, D, page, dtype, seed=seed, std=std)
    if room > p["table"].shape[1] * page:        # a wider table
        p["table"] = torch.nn.functional.pad(p["table"], (0, room // page - p["table"].shape[1]), value=1 << 30)
    poison = [math.inf, -math.inf, math.nan]
    dirty, expect = p["v"].clone(), []
    for b, (L, n) in enumerate(seqs):
        if not L:
            continue
        keys = [L - 1, max(L - n, 0), max(L - n + 1, 0), L // 2, 0]
        keys += [k for k in range(max(L - n, 0), L) if k % 128 in (0, 1, 63, 64, 127)][:D // 2]
        keys += [max(L - 1 - (7 * i) % max(n, 1), 0) for i in range(D)]
        pages = p["table"][b].tolist()
        for h in range(hk):
            for c in range(D):
                j, x = min(keys[(c + 11 * h) % len(keys)], L - 1), poison[(c + h) % 3]
                dirty[pages[j // page], h, j % page, c] = x
                p["v"][pages[j // page], h, j % page, c] = 0.0
                expect.append((b, h, c, j, x))
    want, tol = reference(p)
    first = [int(x) for x in p["cu"]]
    for b, h, c, j, x in expect:
        L, n = seqs[b]
        i = max(j - (L - n), 0)                        # the first row that sees key j
        if i < n:
            g = hq // hk
            want[first[b] + i:first[b] + n, h * g:(h + 1) * g, c] = x
    got = run({**p, "v": dirty}).double()
    near = torch.where(want.isfinite(), (got - want).abs() <= tol, (got == want) | (got.isnan() & want.isnan()))
    assert bool(near.all()), [(r, float(got[tuple(r)]), float(want[tuple(r)])) for r in (~near).nonzero()[:6].tolist()]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("hq,hk", [(2, 2), (8, 2), (7, 1)])
@pytest.mark.parametrize("seqs", [[(300, 300)], [(1, 1), (0, 3), (700, 200), (5, 9), (129, 129)], [(2000, 150), (17, 17), (640, 1)]])
def test_values_that_a_row_does_not_see(cuda_device, dtype, D, hq, hk, seqs):
    check(seqs, hq, hk, D, 16 if D == 128 else 64, dtype, seed=D + hq)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,page", [(64, 32), (128, 256), (256, 128)])
def test_parts_that_several_ctas_share(cuda_device, dtype, D, page):
    check([(20000, 130)], 4, 1, D, page, dtype, seed=3)
    check([(9000, 300), (600, 600)], 3, 3, D, page, dtype, seed=4, std=2.0)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("room", [0, 8192])
def test_one_block_of_keys(cuda_device, dtype, D, room):
    """Nothing to join, by the table's width or by the sequences' alone."""
    check([(17, 17), (128, 128), (1, 1), (100, 3), (3, 6)], 8, 2, D, 16, dtype, seed=8, room=room)
    check([(33, 33)], 5, 1, D, 16, dtype, seed=9, room=room)
    check([(64, 64)] * 40, 2, 1, D, 64, dtype, seed=10, room=room)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_long_prompts(cuda_device, D):
    check([(3500, 3500)], 2, 1, D, 64, "bf16", seed=5)


@pytest.mark.parametrize("hq,hk,D", [(32, 8, 128), (8, 8, 256), (8, 1, 64)])
def test_every_value_from_a_key_on(cuda_device, hq, hk, D):
    """A long prompt whose every value from some key on is not a number, next to one without: rows before that key are what they
    are with zeros there, and the other prompt's have the same bits."""
    import torch
    p = make([(8000, 8000), (500, 400)], hq, hk, D, 64, "bf16", seed=6)
    at = 333
    pages = p["table"][0, :125].long()
    rows = torch.arange(8000, device="cuda").view(125, 1, 64, 1) >= at
    dirty = p["v"].clone()
    dirty[pages] = torch.where(rows, torch.full_like(dirty[pages], math.nan), dirty[pages])
    p["v"][pages] = torch.where(rows, torch.zeros_like(p["v"][pages]), p["v"][pages])
    clean = run(p)
    want, tol = reference(p)
    got = run({**p, "v": dirty})
    assert bool(((got.double() - want).abs() <= tol)[:at].all()) and torch.equal(got[8000:], clean[8000:])
    assert bool(got[at:8000].isnan().all())


def test_pages_out_of_range_next_to_them(cuda_device):
    """A page index out of range counts as a page of zeros here too."""
    import torch
    p = make([(200, 200)], 4, 2, 128, 16, "bf16", seed=7)
    p["table"][0, 11] = -3
    zero = {**p, "v": p["v"].clone()}
    last = int(p["table"][0, 12])
    zero["v"][last, :, 7, 5] = 0.0
    p["v"][last, :, 7, 5] = math.inf
    out = []
    for x in (zero, p):
        o = torch.full_like(x["q"], 7.0)
        fc.fuse_prompt_attention(x["q"], x["k"], x["v"], x["table"], x["cu"], x["lens"], o, x["scale"])
        assert fc.fuse_check() == fc.FUSE_EINDEX
        out.append(o)
    assert bool((out[1][199, :, 5] == math.inf).all())
    out[1][199, :, 5] = out[0][199, :, 5]
    u = 2.0 ** -8                   # each is off by less than 2 u (|o| + E) and the scores' part, for weights that sum to 1 and |v| < 6
    assert bool(((out[0].double() - out[1].double()).abs() <= 4 * u * (out[0].double().abs() + 1.0)).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hq,hk,D", [(8, 2, 128), (4, 4, 256), (8, 1, 64)])
@pytest.mark.parametrize("seqs", [[(3000, 3000), (700, 700)], [(2600, 500), (9, 9)], [(100, 100), (33, 20)]])
def test_columns_of_infinities(cuda_device, dtype, hq, hk, D, seqs):
    """One column infinite from a key on, one of minus infinities from another on, one of both signs (NaN where a row sees both) and
    one that has a single infinity far back: the first sequence's, the others stay as they are."""
    import torch
    p = make(seqs, hq, hk, D, 16, dtype, seed=11)
    (L, n), inf = seqs[0], math.inf
    a, b, c, e = L - n + 7, L - 1 - n // 3, L - n // 2, (L - n) // 2
    pages = p["table"][0, :-(-L // 16)].long()
    pos = torch.arange(len(pages) * 16, device="cuda").view(-1, 1, 16)
    dirty = p["v"].clone()
    part, zero = dirty[pages], p["v"][pages]
    live = pos < L
    for x, where, value in ((3, pos >= a, inf), (7, pos >= b, -inf), (D - 1, pos >= c, inf), (D - 1, (pos >= c) & (pos % 5 == 2), -inf), (20, pos == e, inf)):
        hit = (where & live).expand(-1, hk, -1)
        part[..., x] = torch.where(hit, torch.full_like(part[..., x], value), part[..., x])
        zero[..., x] = torch.where(hit, torch.zeros_like(zero[..., x]), zero[..., x])
    dirty[pages], p["v"][pages] = part, zero
    clean = run(p)
    want, tol = reference(p)
    seen = L - n + 1 + torch.arange(n, device="cuda")                      # keys that a row of the first sequence sees
    two = next(k for k in range(c, L + 5) if k % 5 == 2)                   # the last column's first -inf, and its first inf
    one = next(k for k in range(c, L + 5) if k % 5 != 2)
    w = want[:n].clone()
    w[seen > a, :, 3] = inf
    w[seen > b, :, 7] = -inf
    w[(seen > one) & (seen <= two), :, D - 1] = inf
    w[(seen > two) & (seen <= one), :, D - 1] = -inf
    w[(seen > one) & (seen > two), :, D - 1] = math.nan
    w[seen > e, :, 20] = inf
    got = run({**p, "v": dirty})
    near = torch.where(w.isfinite(), (got[:n].double() - w).abs() <= tol[:n], (got[:n].double() == w) | (got[:n].isnan() & w.isnan()))
    assert bool(near.all()), [(r, float(got[tuple(r)]), float(w[tuple(r)])) for r in (~near).nonzero()[:6].tolist()]
    assert torch.equal(got[n:], clean[n:])
