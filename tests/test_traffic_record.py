"""The benchmark's recorded memory traffic belongs to the code that is there (no GPU)."""
import json

import pytest

import bench


def records():
    with open(bench.TRAFFIC_RECORD, encoding="utf-8") as f:
        return json.load(f)


@pytest.mark.parametrize("key", sorted(records()))
def test_recorded_traffic_is_in_use(key):
    """A change to the recorded kernel's own code calls for a new capture, or for the record to go; a helper of other
    kernels belongs into a header that the recorded one does not include."""
    kind, workload, L = key.split("/")
    assert bench.profiled_traffic(kind, workload, int(L[1:])) == records()[key]["dram_bytes_per_launch"]
