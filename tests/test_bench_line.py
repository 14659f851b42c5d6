"""The benchmark's line carries the report of the kernels that its rows launch, not of every kernel of the
library: the line is read whole by whoever runs the benchmark, and has to stay short."""
import json
import os
import re

import pytest

import bench
import epilogue_chains_gb300 as fc

CSRC = os.path.join(os.path.dirname(os.path.abspath(fc.__file__)), "csrc")


class Reports:
    """Stands for the library: a report of every kernel that the sources define, several variants each."""

    def __init__(self):
        self.names = []
        for f in sorted(os.listdir(CSRC)):
            if f.endswith(".cu"):
                with open(os.path.join(CSRC, f), encoding="utf-8") as src:
                    names = re.findall(r'"(\w+_kernel)\b[^"]*"', src.read())
                self.names += [n + "<variant>" for n in names]

    def fuse_kernel_count(self):
        return len(self.names)

    def fuse_kernel_report(self, i):
        return dict.fromkeys(bench.REPORT_FIELDS, 0) | {"name": self.names[i], "symbol": "left out"}


def test_the_report_is_of_the_rows_kernels():
    lib = Reports()
    kinds = {n.split("_kernel")[0] for n in lib.names}
    assert {"chain_fused", "gemm_decode", "attn_persist", "paged_own", "rope_append", "w4_gemv", "w4_tile"} <= kinds
    got = bench.kernel_report(lib)
    left = [n for n in lib.names if n not in {r["name"] for r in got}]
    assert left and all(n.startswith(("paged_", "rope_", "w4_")) for n in left)
    assert all(set(r) == set(bench.REPORT_FIELDS) for r in got)


@pytest.mark.gpu
def test_the_report_stays_short(cuda_device):
    got = bench.kernel_report(fc)
    assert 19 <= len(got) < 30 < fc.fuse_kernel_count()
    assert len(json.dumps(got)) < 10_000
