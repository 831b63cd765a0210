"""Rules of the kernels' synchronisation that no run shows reliably, checked in their source."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "compressed_sparse_attention_step_gb300",
                    "csrc")


def kernels(name):
    """(kernel, body without comments and strings) for every __global__ function of a source."""
    src = open(os.path.join(CSRC, name)).read()
    src = re.sub(r'//[^\n]*|/\*.*?\*/', " ", src, flags=re.S)
    out = []
    for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\([^{;]*?\)\s*)?(\w+)\s*\(", src):
        i = src.index("{", m.end())
        depth = 0
        for j in range(i, len(src)):
            depth += (src[j] == "{") - (src[j] == "}")
            if depth == 0:
                break
        out.append((m.group(1), src[i:j + 1]))
    assert len(out) == src.count("__global__")
    return out


@pytest.mark.parametrize("source,n", [("matvec.cu", 3), ("tree_attn.cu", 1)])
def test_the_block_meets_between_cluster_barriers(source, n):
    """A warp that is still to wait for one cluster barrier may be counted as having arrived at the next: between
    the wait for one and the next arrival every kernel brings its block together."""
    found = kernels(source)
    assert len(found) == n
    token = re.compile(r"\b(cluster_arrive_wait|cluster_arrive|cluster_wait|__syncthreads|__syncthreads_or)\s*\(")
    for name, body in found:
        waited = False  # a wait that no block barrier has followed yet
        for t in token.findall(body):
            if t.startswith("__syncthreads"):
                waited = False
            if t in ("cluster_arrive", "cluster_arrive_wait"):
                assert not waited, f"{name}: a cluster barrier behind another without __syncthreads between them"
            if t in ("cluster_wait", "cluster_arrive_wait"):
                waited = True


SOURCES = sorted(f for f in os.listdir(CSRC) if f.endswith(".cu"))


@pytest.mark.parametrize("source", SOURCES)
def test_every_kernel_waits_before_it_reads(source):
    """A kernel that may start while the one before it in the stream still runs reads and writes global memory
    behind griddepcontrol.wait alone: every kernel has one such wait, unconditional, before its first load, and lets
    the next kernel start behind it."""
    for name, body in kernels(source):
        assert len(re.findall(r"\bpdl_wait\s*\(\s*\)", body)) == 1, f"{name}: one wait"
        wait = re.search(r"[;{}]\s*pdl_wait\s*\(\s*\)\s*;", body)
        assert wait, f"{name}: the wait is conditional"
        head = body[1:wait.start() + 1]
        assert not re.search(r"__ldg|\bld_|\basm\b|atomic|\bif\b|\bfor\b|\bwhile\b", head), f"{name}: work before the wait"
        depth = head.count("{") - head.count("}")
        assert depth == 0, f"{name}: the wait stands in a block of its own"
        trigger = body.find("pdl_trigger")
        assert trigger == -1 or trigger > wait.end() - 1, f"{name}: the next kernel may start before the wait"
