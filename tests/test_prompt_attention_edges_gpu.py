"""Causal attention of packed prompts where every key counts: with keys of zero all weights of a row are equal, and with values
that are one in the column of the key's position (mod D) and zero elsewhere an output is the number of visible keys of that
column over the number of all.  One key that is lost, doubled or taken for another changes an output by 1 / n.

Scores are exactly 0 and the weights a power of two, off by 2^-22 at most (the exponential) before they are rounded to the
type, which makes them exact.  What is rounded besides is 1 / n, its product with the sum (2^-24 each; all of these together
stay below 2^-21) and the result (u = eps / 2 of the type, fp16 2^-25 below its normal range).  The smallest change 1 / n is told from that where the column's count is below 1 / (2 u): 128 in bf16, 1024 in fp16."""
import math

import pytest

import epilogue_chains_gb300 as fc

pytestmark = pytest.mark.gpu
DT = {"bf16": "bfloat16", "f16": "float16"}


def check(seqs, hq, hk, D, page, dtype, seed=0, room=0):
    """seqs: (keys, new tokens) of each sequence; room: keys that the table has entries for, if more."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = getattr(torch, DT[dtype])
    counts = [-(-k // page) for k, _ in seqs]
    pages = sum(counts) + 2
    assert all(-(-k // D) <= (128 if dtype == "bf16" else 1024) for k, _ in seqs)
    kc = torch.full((pages, hk, page, D), math.nan, dtype=dt, device="cuda")
    vc = kc.clone()
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(seqs), max(*counts, -(-room // page))), 1 << 30, dtype=torch.int32, device="cuda")
    at = 0
    for b, (n, _) in enumerate(seqs):
        ids = order[at:at + counts[b]]
        at += counts[b]
        table[b, :counts[b]] = ids
        pos = torch.arange(counts[b] * page, device="cuda")
        one = torch.zeros(counts[b] * page, D, device="cuda", dtype=dt)
        one[pos, pos % D] = 1.0
        one[n:] = math.nan
        zero = torch.zeros_like(one)
        zero[n:] = math.nan
        kc[ids.long()] = zero.view(counts[b], 1, page, D).expand(-1, hk, -1, -1)
        vc[ids.long()] = one.view(counts[b], 1, page, D).expand(-1, hk, -1, -1)
    starts = [0]
    for _, n in seqs:
        starts.append(starts[-1] + n)
    T = starts[-1]
    q = torch.randn(T, hq, D, generator=g, device="cuda").to(dt)
    o = torch.full((T, hq, D), 7.0, dtype=dt, device="cuda")
    fc.fuse_prompt_attention(q, kc, vc, table, torch.tensor(starts, dtype=torch.int32, device="cuda"),
                             torch.tensor([k for k, _ in seqs], dtype=torch.int32, device="cuda"), o, 1.0 / math.sqrt(D))
    assert fc.fuse_check() == fc.FUSE_OK
    u = torch.finfo(dt).eps / 2
    col = torch.arange(D, device="cuda")
    for b, (L, n) in enumerate(seqs):
        seen = L - n + 1 + torch.arange(n, device="cuda")[:, None].double()                # keys that a token sees
        want = torch.where(seen > 0, torch.clamp(torch.floor((seen - 1 - col) / D) + 1, min=0) / seen.clamp(min=1), torch.zeros_like(seen))
        got = o[starts[b]:starts[b + 1]].double()
        err = (got - want[:, None]).abs()
        bound = (u * (1 + 2.0 ** -20) + 2.0 ** -21) * want + (2.0 ** -25 if dtype == "f16" else 0.0)
        bad = (err > bound[:, None]).nonzero()
        assert not len(bad), (b, bad[:4].tolist(), got[tuple(bad[0])], want[bad[0][0], bad[0][2]])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_every_key_counts_once(cuda_device, dtype, D):
    top = 128 * D if dtype == "bf16" else 30000
    top = min(top, 30000)
    check([(top, 33)], 8, 1, D, 64, dtype, 1)                                     # one item over every CTA
    check([(top - 1, 1), (min(top, 9001), 200), (1, 1)], 8, 2, D, 16, dtype, 2)
    check([(min(top, 4500), 4300)], 4, 2, D, 128, dtype, 3)
    check([(2500, 2500), (3, 9), (129, 128)], 6, 2, D, 32, dtype, 4)
    check([(1 + (37 * i) % 611, 1 + min((37 * i) % 611, (11 * i) % 97)) for i in range(70)], 8, 2, D, 16, dtype, 5)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("hq,hk", [(3, 3), (7, 1), (24, 3), (100, 1)])
def test_every_key_counts_once_in_every_head_layout(cuda_device, hq, hk, D):
    check([(300, 300), (1500, 77), (4000, 3), (2, 2)], hq, hk, D, 256, "f16", hq)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_tables_wider_than_the_sequences(cuda_device, dtype, D):
    """As a server's are: a table as wide as its longest context, sequences of one block of keys and less among those of several."""
    check([(17, 17)], 8, 2, D, 16, dtype, 6, room=8192)
    check([(128, 100), (1, 1), (60, 3), (128, 128)], 8, 8, D, 64, dtype, 7, room=20000)
    check([(300, 300), (2, 5), (129, 1)], 6, 2, D, 32, dtype, 8, room=100000)
