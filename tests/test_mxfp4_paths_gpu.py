"""The microscaled product at the ends of its sizes, and on the path for many tokens (256 by 256 tiles on pairs of CTAs,
taken from about 40 tiles on): every remainder of K, both types, all epilogues, odd and few weights, scales and values that
are not numbers.  Tolerances are those of check_gemm(); where operands are built of codes whose sums are exact, results are
compared for equality."""
import math

import pytest

import epilogue_chains_gb300 as fc
from test_mxfp4_gpu import check_gemm, operands, quantize, whole

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N", [(3, 5), (70, 2)])
def test_longest_rows(cuda_device, M, N):
    """K = 2^29 - 32, zeros but for ones at chosen values, among them the first and last and those on both sides of where a
    count of bytes or of values passes a power of two, and where the CTAs of a cluster share K: each output is the number of ones that meet."""
    import torch
    K = (1 << 29) - 32
    at = sorted({0, 31, 32, 255, 256, K - 1, K - 32, K - 33, K - 256} | {(1 << e) + d for e in (24, 27, 28) for d in (-1, 0, 255, 256)}
                | {(i << 26) + d for i in range(1, 8) for d in (-1, 0)})
    pick = {r: [k for i, k in enumerate(at) if (i + r) % (2 + r % 3) == 0 or k == K - 1] for r in range(8)}

    def operand(rows, shift):
        q = torch.zeros(rows, K // 2, dtype=torch.uint8, device="cuda")
        s = torch.zeros(fc.fuse_mxfp4_scale_bytes(rows, K), dtype=torch.uint8, device="cuda")
        tiles = -(-K // 128)
        for r in range(rows):
            for k in pick[(r + shift) % 8]:
                q[r, k // 2] += 2 if k % 2 == 0 else 32                      # 1.0
                b = k // 32
                s[((r // 128) * tiles + b // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + b % 4] = 127
        return q, s

    xq, xs = operand(M, 0)
    wq, ws = operand(N, 3)
    y = torch.full((M, N), 7.0, dtype=torch.float16, device="cuda")
    fc.fuse_mxfp4_gemm(xq, xs, wq, ws, y)
    assert fc.fuse_check() == fc.FUSE_OK
    want = [[len(set(pick[m % 8]) & set(pick[(n + 3) % 8])) for n in range(N)] for m in range(M)]
    assert y.tolist() == want


MANY = [(2100, 1283), (10000, 1), (10000, 100), (300, 5300)]      # tokens and weights of at least 40 tiles


def on_pairs(M, N):
    return -(-M // 256) * -(-N // 256) >= 40


@pytest.mark.parametrize("K", [32, 64, 96, 128, 160, 224, 256, 288, 416, 544, 1184, 2592])
def test_pairs_lengths(cuda_device, K):
    """Products of one to four steps in the last stage, a lone block of 32 values, an odd number of scale tiles, and both
    parities of the number of stages."""
    for i, (M, N) in enumerate(MANY):
        assert on_pairs(M, N)
        check_gemm(M, N, K, ("bf16", "f16")[(i + K // 32) % 2], seed=K)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", [(2100, 1283, 544), (2305, 1284, 1024), (10000, 100, 160)])
def test_pairs_epilogues(cuda_device, dtype, M, N, K):
    assert on_pairs(M, N)
    for bias in (False, True):
        for gelu in (False, True):
            for residual in (False, True):
                check_gemm(M, N, K, dtype, bias, gelu, residual, seed=5)


@pytest.mark.parametrize("M,N,K", [(2100, 1283, 288), (10000, 100, 96)])
def test_pairs_whole_numbers(cuda_device, M, N, K):
    """Sums of at most 288 products of at most 36 are exact in fp32; up to 2^8 the bf16 result is too."""
    import torch
    out = check_gemm(M, N, K, make=whole)
    x, w, _, _ = whole(M, N, K)
    want = x.double() @ w.double().t()
    small = want.abs() <= 256
    assert bool(small.any()) and torch.equal(out.double()[small], want[small])


@pytest.mark.parametrize("M,N,K", [(2100, 1283, 1184), (10000, 130, 288)])
def test_pairs_one_scale_at_a_time(cuda_device, M, N, K):
    """Every row's and every block's scale its own: a scale taken for another's shows."""
    import torch

    def make(M, N, K, seed, dtype, bias, residual):
        x = torch.ones(M, K, device="cuda", dtype=torch.bfloat16)
        w = torch.ones(N, K, device="cuda", dtype=torch.bfloat16)
        i, j, k = (torch.arange(n, device="cuda") for n in (M, N, K // 32))
        x *= torch.exp2(((i[:, None] * 7 + k[None] * 3) % 11).float()).repeat_interleave(32, 1).to(x.dtype)
        w *= torch.exp2(-((j[:, None] * 5 + k[None] * 2) % 13).float()).repeat_interleave(32, 1).to(x.dtype)
        return x, w, None, None
    check_gemm(M, N, K, make=make)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_pairs_a_value_that_is_not_finite_stays_in_its_row(cuda_device, dtype):
    import torch
    M, N, K = 2100, 1283, 320
    x, w, _, _ = operands(M, N, K, dtype=dtype)
    rows, cols = [3, 255, 256, 1290, 2099], [0, 127, 128, 700, 1282]
    for n, r in enumerate(rows):
        x[r, (70 * n) % K] = math.nan if n % 2 else math.inf
    for n, c in enumerate(cols):
        w[c, (319 * n) % K] = -math.inf if n % 2 else math.nan
    xq, xs = quantize(x)
    wq, ws = quantize(w)
    y = torch.zeros(M, N, dtype=x.dtype, device="cuda")
    fc.fuse_mxfp4_gemm(xq, xs, wq, ws, y)
    assert fc.fuse_check() == fc.FUSE_OK
    want = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    want[rows], want[:, cols] = True, True
    assert torch.equal(y.isnan(), want)


def test_pairs_captured_next_to_another_call(cuda_device):
    """Replays on one stream while calls of other sizes run on another."""
    import torch
    x, w, b, r = operands(2100, 1283, 544, bias=True, residual=True)
    xq, xs = quantize(x)
    wq, ws = quantize(w)
    want = torch.empty(2100, 1283, dtype=x.dtype, device="cuda")
    fc.fuse_mxfp4_gemm(xq, xs, wq, ws, want, bias=b, residual=r, gelu=True)
    small = torch.empty(40, 1283, dtype=x.dtype, device="cuda")
    fc.fuse_mxfp4_gemm(xq[:40], xs, wq, ws, small)
    want_small = small.clone()
    s = torch.cuda.Stream()
    y = torch.zeros_like(want)
    s.wait_stream(torch.cuda.current_stream())
    fc.fuse_graph_begin(s)
    fc.fuse_mxfp4_gemm(xq, xs, wq, ws, y, bias=b, residual=r, gelu=True, stream=s)
    g = fc.fuse_graph_end(s)
    for _ in range(20):
        fc.fuse_graph_launch(g, s)
        fc.fuse_mxfp4_gemm(xq[:40], xs, wq, ws, small)
    assert fc.fuse_check(s) == fc.FUSE_OK and fc.fuse_check() == fc.FUSE_OK
    assert torch.equal(y, want) and torch.equal(small, want_small)
    fc.fuse_graph_destroy(g)
