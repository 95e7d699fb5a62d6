"""bench.py gives the backward kernel's DRAM traffic from its committed
profile, which is of exactly the sources that the kernel is built from."""
import json
import os

import bench


def test_the_committed_profile_is_of_these_sources():
    path = os.path.join(bench.ROOT, "profiles", "bwd_main_prefill4k_full.traffic.json")
    with open(path) as f:
        profile = json.load(f)
    assert profile["kernel_source_hash"] == bench.kernel_source_hash()
    assert bench.measured_traffic() == profile["dram_bytes_per_launch"] > 0

