"""The committed DRAM counters belong to the kernels as they are."""
import json
import os

import pytest

import bench

with open(os.path.join(bench.ROOT, "profiles", "traffic.json")) as fh:
    ENTRIES = {k: v for k, v in json.load(fh).items() if not k.startswith("_")}


@pytest.mark.parametrize("key", sorted(ENTRIES))
def test_counters_were_taken_on_these_sources(key):
    """A change of a layer kernel's sources makes its counters stale: the capture is to be taken
    again. What other operators need goes into files of their own, which leaves these valid."""
    assert bench.sources_hash(ENTRIES[key]["sources"]) == ENTRIES[key]["sources_sha256_16"]
    kernel, workload = key.split("@")
    assert bench.measured_traffic(kernel, workload, 1)[0] == ENTRIES[key]["dram_bytes_per_launch"]
