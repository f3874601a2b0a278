"""Waits on a barrier that threads of another CTA arrive at acquire at the cluster's scope: an acquire
of the CTA's scope does not order what those threads did before. Read from the kernels' source."""
import glob
import os
import re

import pytest

from combine_topk_ids_expert_gb300 import build as B

KERNELS = [p for p in sorted(glob.glob(os.path.join(B.CSRC, "*.cu*")))
           if "mbar_arrive_cluster" in open(p).read() and not p.endswith(("umma.cuh", "fp4_umma.cuh"))]


def remote_barriers(src):
    """Names of the barriers that are arrived at by way of a cluster address."""
    alias = dict(re.findall(r"(\w+) = PAIR \? map_to_rank\((\w+), 0\)", src))
    names = re.findall(r"mbar_arrive_cluster(?:_own)?\((?:map_to_rank\()?(\w+)", src)
    return {alias.get(n, n) for n in names}


def waits(src, name):
    """The template arguments of each wait on barrier `name` ('' without any)."""
    return re.findall(r"wait_or_abort(<\w+>)?\(\s*" + name + r"\b", src)


def test_files_are_found():
    assert {os.path.basename(p) for p in KERNELS} >= {"expert_fp4.cu", "expert_tile.cuh",
                                                      "expert_wgrad.cu", "moe_layer.cu"}


@pytest.mark.parametrize("path", KERNELS, ids=os.path.basename)
def test_waits_for_other_ctas_acquire_at_cluster_scope(path):
    src = open(path).read()
    names = remote_barriers(src)
    assert names
    for name in names:
        found = waits(src, name)
        assert found, name
        for scope in found:
            assert scope in ("<PAIR>", "<true>"), f"{name}: wait_or_abort{scope}"
