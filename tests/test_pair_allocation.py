"""A tensor-memory allocation for a pair of CTAs has no limit to its wait and needs both CTAs
running: every kernel that makes one waits for its peer at the cluster barrier before it."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "routing_token_shuffle_gb300", "csrc")
SOURCES = [p for p in sorted(glob.glob(os.path.join(CSRC, "*.cu"))) if "tmem_alloc_pair(" in open(p).read()]


def test_there_are_pairs():
    assert {os.path.basename(p) for p in SOURCES} >= {"expert_i8.cu", "ffn.cu"}


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_the_peer_is_awaited_before_a_pair_allocates(path):
    for body in re.split(r"\n__global__ ", open(path).read())[1:]:
        for at in re.finditer(r"tmem_alloc_pair\(", body):
            assert re.search(r"cluster_(wait|sync)\(", body[:at.start()]), os.path.basename(path)
