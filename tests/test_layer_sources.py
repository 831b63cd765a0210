"""The rules of test_kernel_sources.py that it holds other sources to, for the kernels with clusters and with mbarriers
around the attention step; and the routing's arithmetic on the host."""
import os
import re

import pytest

from tests.test_kernel_sources import CSRC, kernels


@pytest.mark.parametrize("source,n", [("experts.cu", 5), ("adapters.cu", 1), ("logprobs.cu", 3), ("grouped.cu", 2)])
def test_the_block_meets_between_cluster_barriers(source, n):
    """Between the wait for one cluster barrier and the next arrival every kernel brings its block together."""
    found = kernels(source)
    assert len(found) == n
    token = re.compile(r"\b(cluster_arrive|cluster_wait|__syncthreads)\s*\(")
    for name, body in found:
        waited = False
        for t in token.findall(body):
            if t == "__syncthreads":
                waited = False
            if t == "cluster_arrive":
                assert not waited, f"{name}: a cluster barrier behind another without __syncthreads between them"
            if t == "cluster_wait":
                waited = True


@pytest.mark.parametrize("source", ["adapters.cu", "experts.cu", "grouped.cu", "logprobs.cu"])
def test_no_wait_without_a_limit(source):
    """Every wait on an mbarrier goes through the bounded one."""
    src = open(os.path.join(CSRC, source)).read()
    assert "try_wait" not in src and "test_wait" not in src


def test_a_token_by_multiplication():
    """The token of entry i of a block, i / k, is the high word of i times ceil(2^32 / k) for every size that is served."""
    for k in range(2, 17):
        magic = ((1 << 32) + k - 1) // k
        most = 131072 * k  # tokens of a call times experts
        for i in list(range(3 * k)) + [most - 1, most - k, most // 2, most // 2 + 1]:
            assert (i * magic) >> 32 == i // k
        assert most * (k - 1) < 1 << 32
