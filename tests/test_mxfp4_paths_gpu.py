"""The microscaled product at the ends of its sizes.  Operands are built from codes whose products and sums are exact, so
results are compared for equality."""
import pytest

import epilogue_chains_gb300 as fc

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
