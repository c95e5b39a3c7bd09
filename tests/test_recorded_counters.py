"""The counters under profiles/ that the benchmark reports are of the kernels as they are compiled now."""
import os

import pytest

import bench

PROFILES = os.path.join(bench.ROOT, "profiles")
RECORDS = [(line.split()[0], name) for name in ("dram_traffic.txt", "inst_per_element.txt")
           for line in open(os.path.join(PROFILES, name)) if line.strip() and not line.startswith("#")]


@pytest.mark.parametrize("kernel, name", RECORDS)
def test_records_are_current(kernel, name):
    assert bench.recorded_value(kernel, os.path.join(PROFILES, name)) is not None
