"""The bench's stored DRAM traffic belongs to the grouped-GEMM sources as they are. A change to one of them makes the figure
unmeasured (null in the bench's line): capture it again with the change, or keep what the GEMMs do not use out of their
sources."""
import bench


def test_stored_traffic_is_of_the_present_sources():
    for workload in bench.GEMM_TRAFFIC:
        assert bench.gemm_traffic(workload) is not None, (workload, bench.gemm_source_digest())
