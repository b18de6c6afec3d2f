"""Where the kernels let their dependents launch.

A kernel that allocates tensor memory waits without a limit until its columns are free.  A dependent that is
launched before then may take them and wait in griddep_wait() for that kernel to end: neither goes on.  So every
such kernel triggers its dependents behind its allocation: in the allocating warp, or behind a barrier of the CTA."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "decoder_only_transformer_causal_b200", "csrc")


def _kernels():
    """(file, line, body) of each __global__ function that allocates tensor memory."""
    for name in sorted(os.listdir(CSRC)):
        if not name.endswith((".cu", ".cuh")):
            continue
        text = re.sub(r"//[^\n]*", lambda m: " " * len(m.group()), open(os.path.join(CSRC, name)).read())
        for m in re.finditer(r"__global__", text):
            i = text.index(") {", m.end()) + 2
            depth, j = 0, i
            while True:
                depth += {"{": 1, "}": -1}.get(text[j], 0)
                j += 1
                if depth == 0:
                    break
            if re.search(r"\btmem_alloc(_pair)?\(", text[i:j]):
                yield name, text.count("\n", 0, m.start()) + 1, text[i:j]


KERNELS = list(_kernels())


def test_finds_the_kernels():
    assert {n for n, _, _ in KERNELS} >= {"tree_attention.cu", "head_last.cu", "gemm_tc.cuh", "attention_bwd_tc.cu"}


@pytest.mark.parametrize("name,line,body", KERNELS, ids=[f"{n}:{l}" for n, l, _ in KERNELS])
def test_dependents_are_launched_behind_the_allocation(name, line, body):
    triggers = [m.start() for m in re.finditer(r"\bgriddep_launch_dependents\(\)", body)]
    last = [m.end() for m in re.finditer(r"\btmem_alloc(_pair)?\(", body)][-1]
    for t in triggers:
        assert t > last
        between = body[last:t]
        depths = [between[:k].count("{") - between[:k].count("}") for k in range(len(between) + 1)]
        assert min(depths) >= 0 or re.search(r"\b(__syncthreads|cluster_sync)\(\)", between)
