"""The recorded HBM traffic belongs to the sources as they are, so that the benchmark reports it."""
import pytest

import bench


@pytest.mark.parametrize("kernel,workload", [("pack", "C2"), ("stage2", "C2"), ("pack", "C3"), ("decode", "C3"), ("pack", "C5"), ("stage2", "C5")])
def test_traffic_is_recorded(kernel, workload):
    assert bench.recorded_traffic(kernel, workload) is not None, "counters were taken on other sources: take them again"
