"""The benchmark's DRAM figures belong to the sources as they stand: each is tied to a hash of the kernel's own sources, and a
figure whose sources have changed drops out of the benchmark's line."""

import pytest

import bench


@pytest.mark.parametrize("key", list(bench.NCU_TRAFFIC))
def test_captured_traffic_is_of_these_sources(key):
    workload, kernel, sources = key.split(":")
    assert bench.src_hash(kernel) == sources
    assert f"one capture of sources {key}" in bench.traffic_source(key, bench.NCU_TRAFFIC.get(key))
