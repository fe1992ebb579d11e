"""The build refuses kernels that were compiled for another register count than
their register split adds up to (no GPU: made-up compiler output)."""
import os
import re

import pytest

from paged_kv_cache_318_gb300 import _build


def log(*kernels):
    return "\n".join(
        "ptxas info    : Compiling entry function '%s' for 'sm_103a'\n"
        "ptxas info    : Function properties for %s\n"
        "    0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads\n"
        "ptxas info    : Used %d registers, used 1 barriers" % (k, k, n)
        for k, n in kernels)


def tree(t, d, kv):
    return ("_ZN3pkv4tree16tree_attn_kernelI%sLi%dELi%dEEEvNS0_6ParamsE"
            "14CUtensorMap_stS3_S3_" % (t, d, kv))


TYPES = ("6__half", "13__nv_bfloat16")
RIGHT = [(tree(t, d, kv), 128 if d == 256 else 96)
         for t in TYPES for d in (64, 128, 256) for kv in (1, 2)]


def test_the_right_counts_pass():
    assert _build.check_registers(log(*RIGHT)) == len(RIGHT)
    # kernels without a split may have any
    assert _build.check_registers(log(
        (tree("6__half", 128, 0), 168), (tree("13__nv_bfloat16", 256, 0), 90),
        ("_ZN3pkv4tree11fold_kernelI6__halfLi64EEE", 8))) == 0
    assert _build.check_registers("") == 0


@pytest.mark.parametrize("i", range(len(RIGHT)))
@pytest.mark.parametrize("off", [-8, 8])
def test_another_count_is_refused(i, off):
    name, n = RIGHT[i]
    with pytest.raises(RuntimeError, match="needs %d" % n):
        _build.check_registers(log(*RIGHT[:i], (name, n + off),
                                   *RIGHT[i + 1:]))


def test_the_counts_are_those_of_the_source():
    with open(os.path.join(_build.CSRC, "tree_attn.cuh")) as f:
        two, one = re.search(r"LAUNCH_REGS = NX == 2 \? (\d+) : (\d+)",
                             f.read()).groups()
    assert [n for _, n in _build.LAUNCH_REGS] == [int(two), int(one)]
