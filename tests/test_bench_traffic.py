"""The recorded DRAM traffic of the benchmark's launches is of the sources as they are: the bench
line leaves the figure out otherwise."""
import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_recorded_traffic_is_of_these_sources():
    sys.path.insert(0, ROOT)
    import bench
    with open(os.path.join(ROOT, "profiles", "traffic.json")) as f:
        recorded = json.load(f)
    assert recorded
    for name, t in recorded.items():
        assert t["kernel_rev"] == bench.kernel_revision(t["sources"]), name
