"""The HBM counters that bench.py reports belong to the GEMM sources they were taken on."""

import bench


def test_recorded_counters_are_of_the_current_gemm_sources():
    assert bench.gemm_sources_sha256() == bench.TRAFFIC_COUNTERS["gemm_sources_sha256"]
