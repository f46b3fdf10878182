"""The expert sort's hand-over between the blocks of its cluster, checked on the CPU.

Each block pushes its totals into every block's shared memory.  That memory may be touched
only between its owner's start and its end, and read only when all have written.  The steps
of a block (its cluster barriers, its writes to the others, its reads of its own) are taken
from the kernel's source in their order and run under random interleavings in which blocks
start at any time and a barrier opens when all blocks have arrived.
"""
import os
import random
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "hyper_connection_mix_gb300", "csrc", "hcmix_experts.cuh")

STEPS = [("arrive", r"cluster_arrive\(\)"), ("wait", r"cluster_wait\(\)"),
         ("sync", r"cluster\.sync\(\)"), ("write", r"map_shared_rank\(totals"),
         ("read", r"here \+= totals\[")]


def kernel_steps():
    text = re.sub(r"//[^\n]*", "", open(SOURCE).read())
    body = text[text.index("hcmix_expert_sort_kernel(const SortArgs"):text.index("launch_sort(")]
    found = sorted((m.start(), name) for name, pattern in STEPS for m in re.finditer(pattern, body))
    steps = []
    for _, name in found:
        steps += ["arrive", "wait"] if name == "sync" else [name]
    return steps


def run(steps, blocks, seed):
    """None, or what a block did too early or too late in one interleaving."""
    rnd = random.Random(seed)
    at = [-1] * blocks  # steps done; -1: not started
    arrived = [0] * blocks
    wrote = [set() for _ in range(blocks)]
    late = rnd.randrange(blocks)  # a block that starts after most of the others' steps
    for _ in range(100000):
        ready = [b for b in range(blocks) if at[b] < len(steps)]
        if not ready:
            return None
        b = rnd.choice(ready)
        if b == late and at[b] < 0 and rnd.random() < 0.98:
            continue
        if at[b] < 0:
            at[b] = 0
            continue
        step = steps[at[b]]
        if step == "arrive":
            arrived[b] += 1
        elif step == "wait" and min(arrived) < arrived[b]:
            continue
        elif step == "write":
            for to in range(blocks):
                if at[to] < 0:
                    return "write to a block that has not started"
                if at[to] == len(steps):
                    return "write to a block that has ended"
                wrote[to].add(b)
        elif step == "read" and len(wrote[b]) < blocks:
            return "read before all have written"
        at[b] += 1
    return "never ends"


def faults(steps, blocks):
    return {run(steps, blocks, seed) for seed in range(200)} - {None}


@pytest.mark.parametrize("blocks", [4, 16])
def test_the_kernel_touches_started_blocks_only(blocks):
    steps = kernel_steps()
    assert "write" in steps and "read" in steps
    assert not faults(steps, blocks)


def test_the_model_sees_missing_barriers():
    sound = ["arrive", "wait", "write", "arrive", "wait", "read"]
    assert not faults(sound, 4)
    assert "write to a block that has not started" in faults(sound[2:], 4)
    assert "read before all have written" in faults(sound[:3] + sound[5:], 4)
