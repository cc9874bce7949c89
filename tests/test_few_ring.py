"""The stage ring of the few-token layer, checked on the host.

A stage's barrier tells phases apart by their parity alone, so a wait for a block may only be
made when the block before it on the same stage is known to have landed: a barrier that is two
phases behind looks as if it were done. The fp32 layer's two consumer groups take every other
block of a segment (blocks in ring order, segments of any length, a barrier of both groups
between two segments) and step over the other group's without waiting for them."""
import ctypes
import os
import random
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "routing_token_shuffle_gb300", "csrc")
SOURCE = """
#include "few_ring.cuh"
extern "C" int stages(int f32, int E, int TK, int nd) { return smoe::few_stages(f32 != 0, E, TK, nd); }
extern "C" int group(int i) { return smoe::few_group(i); }
extern "C" int bytes(int f32, int E, int TK, int nd) {
  return (int)smoe::few_misc_bytes(f32 != 0, E, TK) +
         smoe::few_stages(f32 != 0, E, TK, nd) * (smoe::kFewStageA + nd * 128);
}
extern "C" int limit() { return smoe::kFewSmem; }
"""


@pytest.fixture(scope="module")
def ring(tmp_path_factory):
    d = tmp_path_factory.mktemp("ring")
    (d / "ring.cpp").write_text(SOURCE)
    so = str(d / "ring.so")
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-x", "c++", "-I", CSRC,
                    str(d / "ring.cpp"), "-o", so], check=True)
    return ctypes.CDLL(so)


def shapes():
    """(fp32, E, T K, rows of the down product's B tile) over the entry point's range."""
    for T in (1, 7, 8, 9, 13, 16, 17, 24, 32, 33, 48, 64):
        for E in (1, 8, 24, 64, 128, 160, 256, 512):
            for K in (1, 2, 6, 8, 16, 32):
                if K <= E:
                    np = 16 if T <= 16 else 32 if T <= 32 else 64
                    yield 1, E, T * K, np
                    yield 0, E, T * K, 16 if T <= 8 else 2 * np


def test_the_stages_fit(ring):
    for f32, E, TK, nd in shapes():
        assert ring.stages(f32, E, TK, nd) >= 2
        assert ring.bytes(f32, E, TK, nd) <= ring.limit()


def test_no_wait_follows_a_block_that_nobody_waited_for(ring):
    rng = random.Random(1)
    for S in sorted({ring.stages(*s) for s in shapes() if s[0]}):
        for _ in range(20):
            landed = [set(), set()]  # what each group knows to have landed
            block = 0
            for _ in range(12):
                n = rng.randint(1, 4 * S + 1)
                for i in range(n):
                    g = ring.group(i)
                    before = block - S
                    assert before < 0 or before in landed[g], (S, i)
                    landed[g].add(block)
                    block += 1
                landed = [set(range(block)), set(range(block))]  # the segment's closing barrier
