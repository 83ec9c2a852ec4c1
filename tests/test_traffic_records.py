"""The recorded DRAM traffic of each benchmark workload belongs to the kernels as they are: a record taken on other sources
is not used, and the benchmark's line then has none."""
import json
import os

import pytest

import bench


@pytest.mark.parametrize("workload", ["decode", "prefill", "attention", "lmhead", "draft"])
def test_the_record_is_of_these_sources(workload):
    now = bench.layer_source_hash(workload)
    with open(os.path.join(bench.ROOT, "profiles", "layer_%s_traffic.json" % workload)) as f:
        record = json.load(f)
    assert record["kernel_source_hash"] == now
    assert bench.ncu_traffic(workload, now) == record["dram_bytes_per_layer"] > 0
