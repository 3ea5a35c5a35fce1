"""Distributed shared memory is touched only after a cluster barrier: until then
another CTA of the cluster may not have started. No run shows this reliably, so
it is read off the kernels' sources: in each kernel, in the order of the text,
a wait at the cluster's barrier comes before the first access to another CTA's
shared memory.
"""
import os
import re

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "moe_decode_gemm_gb300", "csrc")
REMOTE = re.compile(r"\b(st_dsmem_\w+|ld_dsmem_\w+|mbar_arrive_remote)\s*\(")
WAIT = re.compile(r"\b(cluster_wait_all|cluster_sync_all)\s*\(")


def _kernels():
    for name in sorted(os.listdir(CSRC)):
        if not name.endswith((".cu", ".cuh")) or name == "dg_common.cuh":
            continue
        with open(os.path.join(CSRC, name)) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for part in re.split(r"__global__", text)[1:]:
            if REMOTE.search(part):
                kernel = re.search(r"(\w+_kernel)\s*\(", part)
                yield "%s:%s" % (name, kernel.group(1) if kernel else "?"), part


KERNELS = list(_kernels())


def test_kernels_are_found():
    assert {"k_kv.cu:kv_change_kernel", "k_kv.cu:kv_rank_kernel"} <= {n for n, _ in KERNELS}


@pytest.mark.parametrize("part", [p for _, p in KERNELS], ids=[n for n, _ in KERNELS])
def test_a_cluster_barrier_comes_first(part):
    wait = WAIT.search(part)
    assert wait and wait.start() < REMOTE.search(part).start()
