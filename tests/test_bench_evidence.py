"""The committed counter summaries that the bench line quotes belong to the kernel
in the tree: without that, its traffic figure is silently left out."""
import os
import re

import pytest

import bench

CSRC = os.path.join(bench.ROOT, "pagedattention_kv_cache_attention_gb300", "csrc")


def headers(name, seen=()):
    """Local headers that a source includes, and theirs."""
    for h in re.findall(r'#include "(\w+\.\w+)"', open(os.path.join(CSRC, name)).read()):
        if h not in seen:
            seen = headers(h, seen + (h,))
    return seen


def test_the_hash_covers_every_header_of_the_decode_kernel():
    """All but the launch arguments' header, which holds no device code."""
    assert set(bench.DECODE_SOURCES) == {"pa_decode.cu", *headers("pa_decode.cu")} - {"pa_internal.h"}
    text = open(os.path.join(CSRC, "pa_internal.h")).read()
    assert "__device__" not in text and "__global__" not in text


@pytest.mark.parametrize("name,partition", [("llama3_70b_cb", 2048), ("llama3_8b_gqa", 1024),
                                            ("shared_prefix_cow", 1024), ("long_context", 512)])
def test_the_summaries_are_of_the_current_kernel(name, partition):
    traffic = bench.profiled_traffic(name, partition)
    assert traffic is not None and traffic > 100e6
