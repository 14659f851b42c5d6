"""Limits of the prompt operators' sizes: calls that would count past 32 bits, or past a bounded wait, are refused on
the host, before anything is enqueued."""
import pytest

import epilogue_chains_gb300 as fc

A, B, C, D_, E = (0x100000000000 + (i << 40) for i in range(5))   # far apart, never read


@pytest.mark.parametrize("M,N", [(1, 1), (65, 1), (3, 4096)])
@pytest.mark.parametrize("K", [1 << 29, (1 << 29) + 32, 1 << 30, (1 << 31) - 32])
def test_product_refuses_rows_whose_scales_32_bits_do_not_count(M, N, K):
    """A row's scale tiles of 2^21 stages are 2^31 bytes."""
    assert fc._load().fuse_mxfp4_gemm(A, B, C, D_, None, None, E, M, N, K, 0, fc.FUSE_BF16, None) == fc.FUSE_EUNSUPPORTED
