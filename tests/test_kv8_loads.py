"""The 8-bit KV cache's kernels are launched with programmatic dependent launch,
so their blocks may be resident while the kernel that writes their tables,
scales, queries or tokens still runs. What they read of those goes through
coherent loads: the non-coherent path is for data that stays constant for a
grid's whole life. (Where it went wrong, it would do so by timing, so the source
is what a test can look at.)"""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_grouped_expert_moe_gb300", "csrc")
SOURCES = sorted(glob.glob(os.path.join(CSRC, "kv8*")))


def _code(path):
    with open(path) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_there_are_sources():
    assert len(SOURCES) >= 5


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_no_load_takes_the_non_coherent_path(path):
    found = re.findall(r"__ldg\b|ldg_nc\w*|ld\.global\.nc[.\w]*|ld\.global\.\w+\.nc[.\w]*", _code(path))
    assert not found, found


@pytest.mark.parametrize("path", [p for p in SOURCES if p.endswith(".cu")], ids=os.path.basename)
def test_what_is_read_before_the_dependency_wait_comes_from_l2(path):
    """Per kernel, up to its griddepcontrol.wait (or the helper that holds it):
    no load but through L2, where everything is that an ended kernel wrote."""
    code = _code(path)
    for kernel in re.split(r"__global__", code)[1:]:
        head = re.split(r"griddepcontrol\.wait|after_predecessors\(\)", kernel)[0]
        assert len(head) < len(kernel), kernel[:120]
        assert not re.findall(r"\bld\(|ld_once_v4\(|\bld\.global", head), head[-400:]
