"""The recorded DRAM traffic of the headline GEMM belongs to the sources as they are
(bench.py reports none otherwise)."""
import bench


def test_the_recorded_traffic_is_of_the_current_sources():
    b = bench.recorded_traffic("tc_gemm_kernel", "sq4096")
    assert b is not None, "profiles/traffic.json was taken on other sources: take it again with the command it names"
    assert b >= 3 * 4096 * 4096 * 2  # A, B and C once
