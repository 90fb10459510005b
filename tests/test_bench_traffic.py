"""bench.py's captured DRAM figure of the linear kernel belongs to the sources that are here."""

import bench


def test_captured_traffic_is_of_these_sources():
    """Null in the line means that the kernel or what it is built from changed
    since the capture: capture it again (bench.py --once linear)."""
    assert bench.linear_traffic("flux_mlp_up") == bench.LINEAR_TRAFFIC_CAPTURES["flux_mlp_up"]["bytes"]
    assert bench.linear_traffic("another workload") is None
