"""Log probabilities of rows in which every logit counts: sums of equal terms are exact, so one that is left out or read
twice, at whichever boundary of vectors, threads or CTAs, shows.

Of c equal logits among others of -inf every exponential is 1 and the sum c (below 2^24) is exact: the log probability is
-ln c and the entropy ln c, off by the logarithm's own error only, of which 2^-22 of its value is an upper bound (CUDA's
logf is within 1 ulp)."""
import math

import pytest

import epilogue_chains_gb300 as fc

pytestmark = pytest.mark.gpu
DT = {"bf16": "bfloat16", "f16": "float16", "f32": "float32"}


def check(x, where, top=32):
    """Rows of x have equal logits at `where` (ascending) and -inf elsewhere."""
    import torch
    R, V = x.shape
    c = len(where)
    top = min(top, V)
    tokens = torch.tensor([where[(7 * r) % c] for r in range(R)], dtype=torch.int32, device="cuda")
    lp, H = torch.full((R,), 7.0, device="cuda"), torch.full((R,), 7.0, device="cuda")
    tl, ti = torch.full((R, top), 7.0, device="cuda"), torch.full((R, top), 7, dtype=torch.int32, device="cuda")
    fc.fuse_token_logprobs(x, tokens, lp, entropy=H, top_logprob=tl, top_index=ti)
    assert fc.fuse_check() == fc.FUSE_OK
    ln = math.log(c)
    n = min(top, c)
    for got in (-lp.double(), H.double(), -tl.double()[:, :n]):
        assert bool(((got - ln).abs() <= 2.0 ** -22 * ln).all()), (float(got.min()), float(got.max()), ln)
    assert bool((tl[:, n:] == -math.inf).all())
    first = list(where[:top])
    first += [i for i in range(top) if i not in first][:top - n]                  # then the first of the others
    assert ti.tolist() == [first] * R


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,vocab", [(1, 128000), (3, 32771), (40, 50257), (90, 9000), (350, 5003), (1, 4095), (2, 31)])
def test_every_logit_counts_once(cuda_device, dtype, rows, vocab):
    import torch
    x = torch.full((rows, vocab), 1.5, dtype=getattr(torch, DT[dtype]), device="cuda")
    check(x, range(vocab))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("off", range(16))
def test_boundaries_at_every_start(cuda_device, dtype, off):
    """Rows that begin at every place within a 32-byte vector; equal logits around every place where vectors, the shares of 2,
    4 or 8 CTAs, and what lies before and behind the whole vectors can meet."""
    import torch
    for rows, vocab in ((1, 40003), (80, 16411), (200, 9001), (320, 2477)):
        wide = torch.full((rows, vocab + 48 - vocab % 16), 3.0, dtype=getattr(torch, DT[dtype]), device="cuda")
        x = wide[:, off:off + vocab]
        x.fill_(-math.inf)
        at = {i for i in range(40)} | {vocab - 1 - i for i in range(40)}
        for share in range(1, 8):
            mid = vocab * share // 8
            at |= set(range(mid - 80, mid + 80, 3)) | {mid - 1, mid, mid + 1}
        where = sorted(i for i in at if 0 <= i < vocab)
        x[:, where] = 3.0
        check(x, where)


def test_alternatives_of_two_widths(cuda_device):
    """Widths that differ are refused, a width of 0 among them, whichever of the two it is."""
    import torch
    x = torch.randn(4, 100, device="cuda")
    t = torch.zeros(4, dtype=torch.int32, device="cuda")
    lp = torch.empty(4, device="cuda")
    for a, b in ((0, 5), (5, 0), (3, 5)):
        v, i = torch.full((4, a), 7.0, device="cuda"), torch.full((4, b), 7, dtype=torch.int32, device="cuda")
        with pytest.raises(ValueError):
            fc.fuse_token_logprobs(x, t, lp, top_logprob=v, top_index=i)
    fc.fuse_token_logprobs(x, t, lp, top_logprob=torch.empty(4, 0, device="cuda"), top_index=torch.empty(4, 0, dtype=torch.int32, device="cuda"))
    assert fc.fuse_check() == fc.FUSE_OK
