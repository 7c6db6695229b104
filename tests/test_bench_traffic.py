"""The HBM traffic that bench.py reports for the FC1 kernel was counted on the current sources of its translation unit
(elsewhere the figure is left out of the line, without a word)."""
import json
import os
import re
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import bench  # noqa: E402

CSRC = os.path.join(ROOT, "moe_expert_layer_amd", "csrc")


def test_hash_covers_every_source_of_the_kernel():
    seen, todo = set(), ["grouped_gemm.hip"]
    while todo:
        name = todo.pop()
        seen.add(name)
        todo += set(re.findall(r'#include "([^"]+)"', open(os.path.join(CSRC, name)).read())) - seen
    assert seen == set(bench.FC1_SOURCES)


@pytest.mark.parametrize("workload", bench.GRADED)
def test_traffic_is_of_the_current_sources(workload):
    t = json.load(open(os.path.join(ROOT, "profiles", f"fc1_{workload}_traffic.json")))
    assert t["source_hash"] == bench.source_hash()
    assert t["bytes_per_launch"] > 0
