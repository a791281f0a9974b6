"""Shared memory that CTAs of a cluster hand to one another in the FP8 product: what the source says. The hardware
issues in order, so no run shows an order that the memory model does not give. No GPU."""
from __future__ import annotations

import os
import re

import pytest

from sandwich_norm_residual_gb300 import build


@pytest.fixture(scope="module")
def source():
    with open(os.path.join(build.CSRC, "matmul_fp8.cuh")) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("bar", ["red_ready", "red_full"])
def test_joins_release_and_acquire_at_the_clusters_scope(source, bar):
    """Both barriers of a join go with memory: red_ready with the places that were read and may be overwritten, red_full
    with the sums. Their arrivals release and their waits acquire for the whole cluster."""
    arrivals = re.findall(rf"(mbar_arrive\w*)\(cluster_addr\({bar}, d\)\)", source)
    waits = re.findall(rf"(mbar_wait\S*)\({bar},", source)
    assert arrivals == ["mbar_arrive_cluster_release"] and waits == ["mbar_wait<2>"]


def test_no_other_arrival_goes_to_another_cta(source):
    assert len(re.findall(r"cluster_addr\(red_", source)) == len(re.findall(r"mbar_arrive_cluster", source)) == 2
