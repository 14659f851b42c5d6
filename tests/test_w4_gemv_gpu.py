"""The 4-bit projection against its formula in 64 bits.

Tolerance: (q - z) and its products with x are exact; the fp32 sums run over a group (G terms), the
groups and the parts of a split (K / G and at most 64), each step off by at most 2^-23 (an accumulator
that truncates) of the sum of magnitudes S = sum |x| |w|, twice that with the products by the scale:
(G + K / G + 64) 2^-22 S.  GELU has a slope of at most 1.13 and its approximation is off by 2^-21 of its
value; bias and residual add a rounding each (in the 64 above); the result is rounded once (u = eps / 2)."""
import math

import pytest

import epilogue_chains_gb300 as fc

pytestmark = pytest.mark.gpu
DT = {"bf16": "bfloat16", "f16": "float16"}


def make(M, N, K, G, dtype, zeros=False, bias=False, residual=False, seed=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = getattr(torch, DT[dtype])
    x = torch.randn(M, K, generator=g, device="cuda").to(dt)
    wq = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = ((0.5 + torch.rand(N, K // G, generator=g, device="cuda")) * 0.2 / math.sqrt(K)).to(dt)
    z = torch.randint(0, 16, (N, K // G), generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    b = torch.randn(N, generator=g, device="cuda").to(dt) if bias else None
    r = torch.randn(M, N, generator=g, device="cuda").to(dt) if residual else None
    return x, wq, s, z, b, r


def weights(wq, s, z):
    import torch
    N, K = wq.shape[0], 2 * wq.shape[1]
    G = K // s.shape[1]
    w = torch.stack([wq & 15, wq >> 4], -1).view(N, K).double()
    w -= 8.0 if z is None else z.double().repeat_interleave(G, 1)
    return w * s.double().repeat_interleave(G, 1), G


def check(x, wq, s, z, b, r, gelu=False, **kw):
    import torch
    w, G = weights(wq, s, z)
    K, N, M = x.shape[1], wq.shape[0], x.shape[0]
    y = x.double() @ w.t()
    tol = (G + K / G + 64) * 2.0 ** -22 * (x.double().abs() @ w.abs().t() + (b.double().abs() if b is not None else 0))
    if b is not None:
        y = y + b.double()
    if gelu:
        y = 0.5 * y * torch.special.erfc(-y * math.sqrt(0.5))
        tol = 1.13 * tol + 2.0 ** -21 * y.abs()
    if r is not None:
        y = y + r.double()
        tol = tol + 2.0 ** -23 * y.abs()
    buf = torch.full((M * N + 64,), 7.0, dtype=x.dtype, device="cuda")       # guards around the output
    out = buf[32:32 + M * N].view(M, N)
    fc.fuse_w4_gemv(x, wq, s, out, zeros=z, bias=b, residual=r, gelu=gelu, **kw)
    assert fc.fuse_check() == fc.FUSE_OK
    u = torch.finfo(x.dtype).eps / 2
    err = (out.double() - y).abs()
    tiny = 2.0 ** -25 if x.dtype is torch.float16 else 0.0
    bound = u * y.abs() + (1 + u) * tol + tiny
    assert bool((err <= bound).all()), (float((err / bound).max()), [int(i) for i in (err / bound).argmax().view(1)])
    assert bool((buf[:32] == 7).all()) and bool((buf[32 + M * N:] == 7).all())
    return out


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 32, 33, 64])
def test_tokens_and_groups(cuda_device, dtype, G, M):
    check(*make(M, 200, 1024, G, dtype, zeros=M % 2 == 0, bias=True, residual=M % 3 == 0, seed=M), gelu=M % 4 == 1)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("N,K,G", [(1, 32, 32), (3, 64, 32), (17, 96, 32), (16, 64, 64), (129, 192, 64), (5, 128, 128),
                                   (31, 160, 32), (1000, 320, 64), (15, 2176, 128), (4097, 224, 32), (64, 14336, 128),
                                   (130, 6400, 64), (7, 11008, 32)])
@pytest.mark.parametrize("M", [1, 5, 12, 40])
def test_odd_sizes(cuda_device, dtype, N, K, G, M):
    """Rows that do not fill a tile, a K that ends inside a 128-chunk, fewer chunks than warps, splits."""
    check(*make(M, N, K, G, dtype, zeros=N % 2 == 1, residual=True, seed=N + K))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("G", [32, 64, 128])
def test_few_tokens_many_rows(cuda_device, dtype, G):
    """9 to 16 tokens and more row tiles than SMs, the last one ragged."""
    for M in (9, 16):
        check(*make(M, 24604, 2048, G, dtype, zeros=M == 9, residual=True, seed=G + M))


@pytest.mark.parametrize("M,N,K,G,zeros", [(40, 130, 11264, 128, False), (17, 130, 12288, 128, True),
                                           (64, 300, 5120, 64, True), (33, 129, 5376, 32, False)])
def test_splits_inside_a_block_of_scales(cuda_device, M, N, K, G, zeros):
    check(*make(M, N, K, G, "bf16", zeros=zeros, bias=True, seed=K), gelu=True)


@pytest.mark.parametrize("M,N,K,G,dtype", [(1, 4096, 4096, 128, "bf16"), (5, 4096, 14336, 32, "f16"),
                                           (64, 28672, 4096, 64, "bf16"), (16, 4096, 4096, 128, "f16")])
def test_full_sizes(cuda_device, M, N, K, G, dtype):
    check(*make(M, N, K, G, dtype, zeros=dtype == "f16", bias=True, residual=True), gelu=True)


@pytest.mark.parametrize("K,G", [(320, 64), (288, 32), (2432, 128)])
def test_infinite_scale_in_the_last_groups(cuda_device, K, G):
    """A scale is multiplied with its own group's sum only: an infinite one in the inputs past the last whole
    chunk makes its row infinite, not NaN, and no other row."""
    import torch
    x, wq, s, _, _, _ = make(3, 40, K, G, "bf16", seed=K)
    x = x.abs() + 0.5
    wq |= 0x88                                    # q - 8 in 0 .. 7
    wq[5] = 0xFF
    s[5, -1] = float("inf")
    out = torch.empty(3, 40, dtype=x.dtype, device="cuda")
    fc.fuse_w4_gemv(x, wq, s, out)
    assert bool((out[:, 5] == float("inf")).all())
    keep = [n for n in range(40) if n != 5]
    assert bool(torch.isfinite(out[:, keep]).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_integer_inputs_are_exact(cuda_device, dtype):
    """Integers and scales that are powers of two leave nothing to round: every bit of Y is fixed, so a
    wrong nibble, zero point, scale or column shows whatever the tolerance."""
    import torch
    for M, N, K, G in ((1, 77, 512, 32), (6, 64, 1152, 128), (23, 160, 448, 64), (64, 144, 256, 32)):
        x, wq, s, z, _, _ = make(M, N, K, G, dtype, zeros=True, seed=M)
        x = torch.randint(-1, 2, x.shape, device="cuda").to(x.dtype)
        x[:, K // 3:] = 0                                       # sums stay within 2^8 / 2^11 of exactness
        x[:, :K // 3][:, 20:] = 0
        x[:, -1] = 1
        s = torch.randint(-2, 1, s.shape, device="cuda").double().exp2().to(x.dtype)
        w, _ = weights(wq, s, z)
        y = x.double() @ w.t()
        out = torch.empty(M, N, dtype=x.dtype, device="cuda")
        fc.fuse_w4_gemv(x, wq, s, out, zeros=z)
        assert torch.equal(out, y.to(x.dtype))


def test_repeats_are_equal_bits_and_rows_independent(cuda_device):
    import torch
    x, wq, s, z, b, r = make(24, 512, 4096, 128, "bf16", zeros=True, residual=True)
    a, c = check(x, wq, s, z, b, r), check(x, wq, s, z, b, r)
    assert torch.equal(a, c)
    x2 = x.clone()
    x2[3] = float("nan")                                        # one bad token leaves the others alone
    out = torch.empty_like(a)
    fc.fuse_w4_gemv(x2, wq, s, out, zeros=z, residual=r)
    keep = torch.arange(24, device="cuda") != 3
    assert torch.equal(out[keep], a[keep]) and bool(out[3].isnan().all())


def test_graph_replay_and_side_stream(cuda_device):
    import torch
    x, wq, s, z, b, r = make(3, 768, 2048, 64, "f16", bias=True)
    st = torch.cuda.Stream()
    y = torch.empty(3, 768, dtype=x.dtype, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        fc.fuse_graph_begin(st)
        fc.fuse_w4_gemv(x, wq, s, y, bias=b, stream=st)
        g = fc.fuse_graph_end(st)
    for seed in (1, 2):
        x.copy_(make(3, 768, 2048, 64, "f16", seed=seed)[0])
        torch.cuda.synchronize()
        fc.fuse_graph_launch(g, st)
        st.synchronize()
        assert torch.equal(y, check(x, wq, s, z, b, r))
    fc.fuse_graph_destroy(g)


def test_wrapper_refusals(cuda_device):
    import torch
    x, wq, s, z, b, r = make(3, 64, 256, 64, "bf16", zeros=True, bias=True, residual=True)
    y = torch.empty(3, 64, dtype=x.dtype, device="cuda")
    for bad in (dict(x=x.half()), dict(wq=wq.to(torch.int8)), dict(wq=wq[:, :-16].contiguous()), dict(s=s.float()),
                dict(y=y[:2]), dict(zeros=z[:, :2].contiguous()), dict(bias=b[:5]), dict(residual=r[:2]),
                dict(x=x.t().contiguous().t()), dict(x=x.cpu())):
        p = dict(x=x, wq=wq, s=s, y=y, zeros=z, bias=b, residual=r)
        p.update(bad)
        with pytest.raises(ValueError):
            fc.fuse_w4_gemv(p["x"], p["wq"], p["s"], p["y"], zeros=p["zeros"], bias=p["bias"], residual=p["residual"])
    big = make(65, 64, 256, 64, "bf16")
    with pytest.raises(fc.FuseError):
        fc.fuse_w4_gemv(big[0], big[1], big[2], torch.empty(65, 64, dtype=x.dtype, device="cuda"))
