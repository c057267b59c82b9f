"""The counter readings that the benchmark reports stand under the digest of the kernel sources as they are."""
import glob
import os

import pytest

import bench

TABLES = sorted(glob.glob(bench.traffic_table("*")))


def rows(table):
    with open(table) as f:
        cells = [[c.strip() for c in line.strip().strip("|").split("|")] for line in f if line.startswith("|")]
    return [(c[0], c[1]) for c in cells if c[0] in bench.KERNEL_SOURCE]


@pytest.mark.parametrize("table", TABLES, ids=os.path.basename)
def test_traffic_is_that_of_the_current_sources(table):
    workload = os.path.basename(table)[len("hbm_traffic_"):-len(".md")]
    assert rows(table)
    for kernel, digest in rows(table):
        assert digest == bench.source_digest(kernel), kernel
        assert bench.measured_traffic(kernel, workload), kernel


def test_there_are_tables():
    assert len(TABLES) == 4
