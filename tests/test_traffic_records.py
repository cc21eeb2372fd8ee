"""The benchmark's DRAM traffic of a launch comes from a committed capture, and only while the kernel's
sources are those that were captured: the records of the workloads that it runs by name belong to the
present sources."""
import pytest

import bench


@pytest.mark.parametrize("kernel,workload,T", [
    ("grouped_gemm_kernel<gate_up>", "131k_skewed", 131072),
    ("grouped_gemm_kernel<gate_up>", "20b_prefill", 8192),
    ("expert_tile_kernel<0>", "20b_decode", 16),
    ("stream_gate_up_kernel", "20b_decode", 16),
    ("stream_gate_up_mx_kernel", "20b_decode_mxfp4", 16),
])
def test_records_belong_to_the_present_sources(kernel, workload, T):
    assert bench.ncu_traffic(kernel, workload, T) is not None
