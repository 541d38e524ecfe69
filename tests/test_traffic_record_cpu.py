"""The committed dram records are of the present kernel sources: bench.py gives
`traffic` from them for every workload that they name."""
import json
import os

import pytest

import bench

with open(os.path.join(bench.ROOT, "profiles", "traffic.json")) as f:
    RECORDS = json.load(f)


@pytest.mark.parametrize("kernel,workload", [(k, w) for k, r in RECORDS.items() for w in r["workloads"]])
def test_record_applies_to_the_present_source(kernel, workload):
    got = bench.traffic_record(kernel, workload, RECORDS[kernel]["activations"], 10 ** 8)
    assert got is not None and got >= 10 ** 8
