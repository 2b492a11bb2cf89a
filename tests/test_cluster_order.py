"""No kernel may touch another CTA's shared memory before its cluster's first barrier: until then the peer may not run yet, or
may still write its first values over what came.  Looked for in the source, where a call's place is its order."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_201_gb300", "csrc")
BARRIER = re.compile(r"cluster_barrier\(\)|sync_all\(|barrier\.cluster\.wait")
REMOTE = re.compile(r"peer_addr\(|mapa\.")


def _kernels():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for body in text.split("__global__")[1:]:
            body = body.split("\ntemplate")[0]
            if REMOTE.search(body):
                yield pytest.param(body, id=re.search(r"\b(paged_attn_\w+|\w+_kernel)\(", body).group(1))


@pytest.mark.parametrize("body", list(_kernels()))
def test_a_barrier_comes_first(body):
    first = BARRIER.search(body)
    assert first and first.start() < REMOTE.search(body).start()


def test_kernels_are_found():
    names = [p.id for p in _kernels()]
    assert {"paged_attn_free_kernel", "paged_attn_compact_kernel", "paged_attn_kv4_kernel"} <= set(names)
