"""Kernels launched with programmatic dependent launch read what an earlier kernel
may have written (lengths, q, the layer's input) through coherent loads: their
blocks may be resident while that kernel still runs, and the non-coherent path is
for data that stays constant for a grid's whole life."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_grouped_expert_moe_gb300", "csrc")


def _code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_decode_attention():
    code = _code("attention.cu")
    assert not re.findall(r"__ldg\b|ldg_nc\w*|ld\.global\.nc", code)
    for kernel in re.split(r"__global__", code)[1:]:  # before the wait: L2 only
        head = kernel.split("griddepcontrol.wait")[0]
        assert len(head) < len(kernel) and not re.findall(r"\bld\(", head)


def test_fused_decode_layer():
    """After the wait; the weights, constant, are read before it as well."""
    kernel = _code("decode.cu").split("decode_layer_kernel(const DecodeArgs a)")[1]
    _, tail = kernel.split("grid_dep_wait();", 1)
    tail = tail.split("__global__")[0]
    assert not re.findall(r"__ldg\(a\.x\b|ldg_nc_v4\(a\.x\b|__ldg\(a\.r\b", tail)
