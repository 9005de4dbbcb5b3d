"""Kernels placed before the stream's previous kernel is done read its results by coherent loads only.

They start early and wait with griddepcontrol.wait, so what they read may be written while they live. A read-only
load (__ldg, or a const __restrict__ pointer's) is not defined for that, and the compiler may move one ahead of the
wait. And no kernel is launched on the results of one whose set-up or launch failed.
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_layer_dsv3_gb300", "csrc")


def _code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def _files():
    early = {n for n in os.listdir(CSRC) if n.endswith((".cu", ".cuh")) and "griddepcontrol.wait" in _code(n)}
    return sorted(early)


def test_the_files_are_found():
    assert {"k_norm.cu", "k_mla.cu", "k_mla_pair.cu", "mla.cuh"} <= set(_files())


@pytest.mark.parametrize("name", _files())
def test_no_read_only_loads(name):
    code = _code(name)
    assert "__ldg" not in code and "ld.global.nc" not in code
    assert not re.search(r"const [\w:]+\s*\*\s*__restrict__", code)


@pytest.mark.parametrize("name,first,then", [
    ("k_norm.cu", "else bwd<4, false, 2>(", 'launch_kernel_after("norm_dgamma"'),
    ("k_mla.cu", 'launch_kernel_after("mla_decode"', "launch_join<"),
    ("k_mla_pair.cu", 'launch_cluster_after("mla_decode_pair"', "launch_join<")])
def test_no_launch_on_the_results_of_a_failed_one(name, first, then):
    """A workspace that nothing filled is not summed: the call's error is looked at between the two launches."""
    code = _code(name)
    at = code.rindex(first)
    assert re.search(r"if \([^;]*call_error\(\)[^;]*\) return", code[at:code.index(then, at)])
