"""Log probabilities of tokens, entropy and alternatives against their formulas in 64 bits.

Tolerance, with d_j = |x_j - max| scale, E d and E d^2 its moments under the row's probabilities: an exponential is off by
2^-21 of itself and, through its argument (two roundings and that of scale log2(e)), by d 2^-22; a sum runs over at most
n = vocab / 256 + 64 terms (a thread's, then the joins), each step off by half a step of fp32.  So ln S is off by
s = n 2^-24 + 2^-21 + 2^-22 E d + 2^-23 |ln S|, a log probability by s + 2^-22 d + 2^-23 |log p|, and the entropy
ln S + E d by s + E d (2 n 2^-24 + 2^-20) + 2^-22 E d^2 + 2^-22 H."""
import math

import pytest

import epilogue_chains_gb300 as fc

pytestmark = pytest.mark.gpu
DT = {"bf16": "bfloat16", "f16": "float16", "f32": "float32"}


def logits(rows, vocab, dtype, seed=0, std=3.0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (std * torch.randn(rows, vocab, generator=g, device="cuda")).to(getattr(torch, DT[dtype]))


def call(x, tokens, top, scale=1.0, **kw):
    """(logprob, entropy, top_logprob, top_index) with guards around each."""
    import torch
    R = x.shape[0]
    bufs = [torch.full((n + 32,), 7, dtype=dt, device="cuda") for n, dt in
            ((R, torch.float32), (R, torch.float32), (R * top, torch.float32), (R * top, torch.int32))]
    out = [b[16:b.numel() - 16] for b in bufs]
    out[2], out[3] = out[2].view(R, top), out[3].view(R, top)
    fc.fuse_token_logprobs(x, tokens, out[0], entropy=out[1], top_logprob=out[2] if top else None,
                           top_index=out[3] if top else None, scale=scale, **kw)
    assert fc.fuse_check() == fc.FUSE_OK
    assert all(bool((b[:16] == 7).all()) and bool((b[-16:] == 7).all()) for b in bufs)
    return out


def check(x, tokens, top, scale=1.0, **kw):
    import torch
    got = call(x, tokens, top, scale, **kw)
    z = x.double() * scale
    V = x.shape[1]
    M = z.amax(1, keepdim=True)
    dead = M[:, 0] == -math.inf
    d = torch.where(z > -math.inf, M - z, torch.zeros_like(z))
    p = torch.where(z > -math.inf, torch.exp(-d), torch.zeros_like(z))
    S = p.sum(1, keepdim=True)
    p = p / S.clamp(min=1e-300)
    lnS = S.clamp(min=1e-300).log()
    Ed, Ed2 = (p * d).sum(1, keepdim=True), (p * d * d).sum(1, keepdim=True)
    n = V / 256 + 64
    s = n * 2.0 ** -24 + 2.0 ** -21 + 2.0 ** -22 * Ed + 2.0 ** -23 * lnS.abs()
    lp = torch.where(z > -math.inf, -d - lnS, torch.full_like(z, -math.inf))
    lp[dead] = -math.inf
    tol = s + 2.0 ** -22 * d + 2.0 ** -23 * (d + lnS)
    H = torch.where(dead, torch.zeros_like(Ed[:, 0]), (lnS + Ed)[:, 0])
    tolH = (s + Ed * (2 * n * 2.0 ** -24 + 2.0 ** -20) + 2.0 ** -22 * Ed2)[:, 0] + 2.0 ** -22 * H

    def near(a, b, t):
        fin = torch.isfinite(b)
        assert torch.equal(a.double()[~fin], b[~fin])
        err = (a.double() - b).abs()[fin]
        assert bool((err <= t.expand_as(b)[fin]).all()), float((err / t.expand_as(b)[fin]).max())

    if tokens is not None:
        at = tokens.clamp(min=0).long()[:, None]
        want = torch.where(tokens >= 0, lp.gather(1, at)[:, 0], torch.zeros_like(H))
        near(got[0], want, torch.where(tokens >= 0, tol.gather(1, at)[:, 0], torch.zeros_like(H)))
    near(got[1], H, tolH)
    if top:
        best = torch.sort(x.float(), dim=1, descending=True, stable=True).indices[:, :top]
        assert torch.equal(got[3].long(), best)
        near(got[2], lp.gather(1, best), tol.gather(1, best))
    return got


def tokens_for(x, seed=1, padded=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.randint(0, x.shape[1], (x.shape[0],), generator=g, device="cuda", dtype=torch.int32)
    t[:padded] = -1
    return t


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,vocab,top", [(1, 1, 1), (1, 7, 3), (3, 33, 32), (2, 255, 5), (5, 1000, 20), (1, 128000, 20),
                                            (7, 50257, 8), (40, 16385, 1), (100, 32000, 0), (700, 5001, 32)])
def test_sizes(cuda_device, dtype, rows, vocab, top):
    x = logits(rows, vocab, dtype, seed=vocab)
    check(x, tokens_for(x, padded=rows // 4), top)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("off", range(8))
def test_rows_of_any_alignment(cuda_device, dtype, off):
    """Rows of a wider tensor that start and end inside 16-byte vectors."""
    x = logits(5, 3001 + 16, dtype, seed=off)[:, off:off + 2990 + off]
    check(x, tokens_for(x), 10)
    x = logits(3, 20001 + 16, dtype, seed=off)[:, off:off + 19999]
    check(x, tokens_for(x), 4)


@pytest.mark.parametrize("rows,vocab", [(1, 70000), (60, 70000), (130, 9001), (400, 700)])
@pytest.mark.parametrize("scale", [0.25, 1.0, 7.5])
def test_scales(cuda_device, rows, vocab, scale):
    x = logits(rows, vocab, "bf16", seed=rows)
    check(x, tokens_for(x), 6, scale)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,vocab", [(2, 40000), (400, 3000)])
def test_masked_rows(cuda_device, dtype, rows, vocab):
    """Most logits -inf; rows with fewer allowed tokens than alternatives, one, and none."""
    import torch
    x = logits(rows, vocab, dtype, seed=3)
    x[:, torch.rand(vocab, device="cuda") < 0.97] = -math.inf
    t = tokens_for(x)
    check(x, t, 8)
    few = x.clone()
    few[0] = -math.inf
    few[1] = -math.inf
    few[1, vocab - 1] = -2.0
    few[-1] = -math.inf
    few[-1, [0, 2, vocab // 2]] = torch.tensor([1.0, 3.0, 1.0], device="cuda").to(few.dtype)
    check(few, t, 8)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_equal_logits(cuda_device, dtype):
    """Of equal logits the lower index comes first: constant rows, few levels, zeros of both signs."""
    import torch
    x = logits(4, 30000, dtype, seed=5)
    x[0] = 1.5
    x[1] = x[1].round()
    x[2] = torch.where(x[2] > 0, torch.full_like(x[2], 0.0), torch.full_like(x[2], -0.0))
    x[3, :] = torch.where(torch.arange(30000, device="cuda") % 100 == 99, 2.0, 1.0).to(x.dtype)
    check(x, tokens_for(x), 32)
    check(x.repeat(100, 1)[:, :2000], tokens_for(x.repeat(100, 1)[:, :2000]), 32)


def test_large_logits_and_the_lowest_value(cuda_device):
    """Logits near the type's limits, and the type's lowest value as a mask."""
    import torch
    x = logits(3, 9000, "f32", seed=7) + 3.0e4
    check(x, tokens_for(x), 5)
    x = logits(3, 9000, "f32", seed=8)
    x[:, 1000:] = torch.finfo(torch.float32).min
    x[2] = torch.finfo(torch.float32).max
    check(x, tokens_for(x[:, :1000]), 5)
    x = logits(3, 9000, "bf16", seed=9)
    x[:, :8000] = torch.finfo(torch.bfloat16).min
    check(x, tokens_for(x) % 1000 + 8000, 5)


def test_a_sure_token(cuda_device):
    """One logit far above the others: entropy and log probability close to zero, not lost."""
    x = logits(2, 100000, "f32", seed=10, std=1.0)
    x[:, 777] = 40.0
    got = check(x, tokens_for(x) * 0 + 777, 3)
    assert bool((got[0] <= 0).all()) and bool((got[1] >= 0).all())


@pytest.mark.parametrize("rows", [1, 500])
def test_not_a_number(cuda_device, rows):
    import torch
    x = logits(rows, 6000, "bf16", seed=11)
    x[0, 4321] = math.nan
    x[-1, 0] = math.nan
    got = call(x, tokens_for(x), 5)
    for r in (0, rows - 1):
        assert math.isnan(float(got[0][r])) and math.isnan(float(got[1][r])) and bool(got[2][r].isnan().all())
        y = x[r].float().nan_to_num(nan=-math.inf)
        assert torch.equal(got[3][r].long(), torch.sort(y, descending=True, stable=True).indices[:5])
    x = logits(2, 6000, "f32", seed=12)
    x[0, 17] = math.inf
    got = call(x, tokens_for(x), 5)
    assert math.isnan(float(got[0][0])) and math.isnan(float(got[1][0])) and int(got[3][0, 0]) == 17
    assert bool(got[0][1:].isfinite().all())


def test_tokens_out_of_range(cuda_device):
    import torch
    x = logits(4, 1000, "f32", seed=13)
    t = torch.tensor([5, 1000, -7, 999], dtype=torch.int32, device="cuda")
    lp = torch.empty(4, device="cuda")
    fc.fuse_token_logprobs(x, t, lp)
    assert fc.fuse_check() == fc.FUSE_EINDEX and fc.fuse_check() == fc.FUSE_OK
    assert bool(lp[1].isnan()) and float(lp[2]) == 0.0 and bool(lp[[0, 3]].isfinite().all())


def test_outputs_that_are_left_out(cuda_device):
    import torch
    x = logits(6, 40000, "bf16", seed=14)
    t = tokens_for(x)
    want = call(x, t, 5)
    lp, H = torch.empty(6, device="cuda"), torch.empty(6, device="cuda")
    tl, ti = torch.empty(6, 5, device="cuda"), torch.empty(6, 5, dtype=torch.int32, device="cuda")
    fc.fuse_token_logprobs(x, t, lp)
    fc.fuse_token_logprobs(x, None, None, entropy=H)
    fc.fuse_token_logprobs(x, None, None, top_logprob=tl)
    fc.fuse_token_logprobs(x, None, None, top_index=ti)
    for a, b in zip((lp, H, tl, ti), want):
        assert torch.equal(a, b)


def test_captured_and_on_another_stream(cuda_device):
    import torch
    x = logits(3, 60000, "bf16", seed=15)
    t = tokens_for(x)
    want = [w.clone() for w in call(x, t, 5)]
    s = torch.cuda.Stream()
    out = [torch.zeros_like(w) for w in want]
    s.wait_stream(torch.cuda.current_stream())
    fc.fuse_graph_begin(s)
    fc.fuse_token_logprobs(x, t, out[0], entropy=out[1], top_logprob=out[2], top_index=out[3], stream=s)
    g = fc.fuse_graph_end(s)
    assert fc.fuse_graph_kernel_count(g) == 1
    for _ in range(2):
        for o in out:
            o.zero_()
        s.wait_stream(torch.cuda.current_stream())
        fc.fuse_graph_launch(g, s)
        assert fc.fuse_check(s) == fc.FUSE_OK
        assert all(torch.equal(o, w) for o, w in zip(out, want))
    fc.fuse_graph_destroy(g)


def test_refusals(cuda_device):
    import torch
    x = logits(4, 100, "f32")
    t = tokens_for(x)
    lp = torch.empty(4, device="cuda")
    for bad in (dict(top_index=torch.empty(4, 5, device="cuda")), dict(entropy=torch.empty(5, device="cuda")),
                dict(top_logprob=torch.empty(4, 5, device="cuda"), top_index=torch.empty(4, 6, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            fc.fuse_token_logprobs(x, t, lp, **bad)
    with pytest.raises(ValueError):
        fc.fuse_token_logprobs(x.t(), t, lp)
    with pytest.raises(ValueError):
        fc.fuse_token_logprobs(x, t.long(), lp)
    with pytest.raises(fc.FuseError):
        fc.fuse_token_logprobs(x, t, lp, scale=0.0)
    with pytest.raises(fc.FuseError):
        fc.fuse_token_logprobs(x, t, lp, top_logprob=torch.empty(4, 33, device="cuda"))
