"""The kernels' measured HBM traffic that bench.py reports belongs to the sources of this tree."""
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import bench  # noqa: E402
from post_weight_quantization_gq_amd import synth  # noqa: E402


@pytest.mark.parametrize("stage", sorted(bench._TRAFFIC))
def test_measured_traffic_is_of_these_sources(stage):
    """Every stage's figure is reported: neither its source file nor the headers in its digest have
    changed since its counters were taken (headers of other kernels are not among them)."""
    entry = bench._TRAFFIC[stage]
    assert bench._source_digest(entry[1]) == entry[2]
    assert bench._traffic(stage, synth.WORKLOADS[entry[0]]) == entry[3] + entry[4]
