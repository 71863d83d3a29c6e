"""The traffic table's guard: a figure holds for the sources that its kernel was captured with, and for those alone."""
from __future__ import annotations

import os
import shutil
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import bench  # noqa: E402

CSRC = os.path.join(ROOT, "nvfp4_quantization_group_b200", "csrc")


@pytest.mark.parametrize("workload,kernels,other", [("grouped_moe", "hq_nvfp4.cu", "hq_fp8.cu"),
                                                    ("dense_nvfp4", "hq_nvfp4.cu", "hq_fp8.cu"),
                                                    ("dsa_indexer_nvfp4", "hq_fp8.cu", "hq_nvfp4.cu"),
                                                    ("qmoe_swiglu", "hq_fp8.cu", "hq_nvfp4.cu")])
def test_a_figure_goes_by_its_kernels_sources(tmp_path, workload, kernels, other):
    csrc = str(tmp_path / "csrc")
    shutil.copytree(CSRC, csrc)
    sha = bench.kernel_source_sha(workload, csrc)
    assert sha == bench.kernel_source_sha(workload)
    for name in os.listdir(csrc):
        path = os.path.join(csrc, name)
        before = open(path, "rb").read()
        with open(path, "ab") as f:
            f.write(b"// another state\n")
        changed = name in (kernels, "hq_device.cuh", "hq_internal.h", "hq_api.cu")
        assert (bench.kernel_source_sha(workload, csrc) != sha) == changed, name
        with open(path, "wb") as f:
            f.write(before)
    assert kernels in bench.kernel_sources(workload) and other not in bench.kernel_sources(workload)
    # what those files include is among them (the C header apart)
    for name in bench.kernel_sources(workload):
        for line in open(os.path.join(csrc, name)):
            if line.startswith('#include "') and "hq.h" not in line:
                assert line.split('"')[1] in bench.kernel_sources(workload), (name, line)
