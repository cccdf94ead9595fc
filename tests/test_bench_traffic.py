"""The benchmark's DRAM bytes per launch come from a capture that holds for the finalize kernels' present sources."""
import os
import re
import shutil
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join("moe_finalize_residual_gb300", "csrc")
KERNELS = ["cluster_decode_T128", "bulk_bandwidth_H7168_T1024"]


@pytest.fixture
def bench():
    sys.path.insert(0, ROOT)
    import bench as b
    return b


@pytest.mark.parametrize("kernel", KERNELS)
def test_the_committed_capture_is_of_the_present_kernels(bench, kernel):
    assert bench.traffic_for(kernel) > 0


def test_only_the_finalize_kernels_sources_make_it_stale(bench, tmp_path, monkeypatch):
    for d in ("profiles", CSRC):
        shutil.copytree(os.path.join(ROOT, d), tmp_path / d)
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    want = bench.traffic_for(KERNELS[0])
    for name in os.listdir(tmp_path / CSRC):
        path = tmp_path / CSRC / name
        text = path.read_text()
        path.write_text(text + "\n")
        assert bench.traffic_for(KERNELS[0]) == (None if name in bench.FINALIZE_SOURCES else want), name
        path.write_text(text)


def test_the_sources_are_all_that_the_finalize_kernels_include(bench):
    """Followed from the four translation units of the finalize."""
    seen, todo = set(), [n for n in bench.FINALIZE_SOURCES if n.endswith(".cu")]
    while todo:
        name = todo.pop()
        seen.add(name)
        text = open(os.path.join(ROOT, CSRC, name)).read()
        todo += [n for n in re.findall(r'#include "(\w+\.\w+)"', text) if os.path.exists(os.path.join(ROOT, CSRC, n)) and n not in seen]
    assert seen == set(bench.FINALIZE_SOURCES)
