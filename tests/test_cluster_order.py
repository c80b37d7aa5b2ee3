"""Every kernel that touches another CTA's shared memory has passed a cluster
barrier before its first such access: only the barrier says that the other
CTAs of the cluster have started.  Read from the sources; needs no GPU."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "mixture_experts_layer_12_gb300", "csrc")

# accesses to (possibly) another CTA's shared memory: the helpers of tc_common.cuh
# and whatever else is given an address mapped into the cluster
REMOTE = re.compile(r"\b(dsmem_st\w*|dsmem_ld\w*|atomicAdd_cluster\w*|mbar_arrive\w*_cluster|tma_load_\w*pair)\s*\(")
BARRIER = re.compile(r"\bcluster_(sync_all|wait)\s*\(")


def kernels(src):
    """(name, body) of every __global__ function, comments taken out."""
    src = re.sub(r"/\*.*?\*/", " ", src, flags=re.S)
    src = re.sub(r"//[^\n]*", " ", src)
    for m in re.finditer(r"__global__", src):
        at = src.index("{", m.end())
        head = src[m.end():at]
        depth, end = 0, at
        while True:
            depth += {"{": 1, "}": -1}.get(src[end], 0)
            end += 1
            if depth == 0:
                break
        name = [w for w in re.findall(r"(\w+)\s*\(", head) if not w.startswith("__")][-1]
        yield name, src[at:end]


def all_kernels():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))):
        with open(path, encoding="utf-8") as f:
            for name, body in kernels(f.read()):
                if REMOTE.search(body):
                    yield pytest.param(body, id=f"{os.path.basename(path)}:{name}")


def test_kernels_with_remote_accesses_are_found():
    names = {p.id for p in all_kernels()}
    assert "decode_route.cu:decode_route_kernel" in names and len(names) >= 3


@pytest.mark.parametrize("body", list(all_kernels()))
def test_a_cluster_barrier_comes_before_the_first_remote_access(body):
    barrier, remote = BARRIER.search(body), REMOTE.search(body)
    assert barrier and barrier.start() < remote.start()
