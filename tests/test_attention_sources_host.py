"""The attention kernels' threads leave together after a bounded wait that gave up.

A wait that runs out ends with a status code instead of a hang only if no thread then waits at a
barrier, or in a vote of its warp, for one that has already left.  That cannot be shown on a
GPU without making a wait run out, so it is read from the sources: between a wait that can clear
`ok` and the next `break` there is a barrier or a vote that tells the others.
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "kda_gated_delta_chunk_gb300", "csrc")


def section(name, first, last):
    text = open(os.path.join(CSRC, name)).read()
    a = text.index(first)
    lines = text[a:text.index(last, a)].splitlines()
    return [re.sub(r"//.*", "", x) for x in lines]


@pytest.mark.parametrize("name,first,last", [
    ("kda_attn_decode_kernel.cu", "= softmax and accumulation", "p.desc[blockIdx.x] = part"),
    ("kda_attn_decode_kernel.cu", "= producer", "= MMA issuer"),      # (one thread issues: no one waits for it)
    ("kda_attn_prefill_kernel.cu", "auto seg_wait", "DEVICE_TIMEOUT, 336"),
])
def test_nobody_leaves_alone(name, first, last):
    told = True           # since the last wait: the others know its outcome
    breaks = 0
    for line in section(name, first, last):
        if re.search(r"\bok\s*=.*mbar_wait|\badd_o\(it", line):
            told = False
        if "__all_sync(" in line or "bar_any(" in line:
            told = True
        if re.search(r"\bbreak;", line):
            breaks += 1
            assert told or re.search(r"if \(left\)", line), line.strip()
    assert breaks > 0


def test_the_decode_kernel_leaves_its_tile_loop_by_the_barriers_answer():
    text = open(os.path.join(CSRC, "kda_attn_decode_kernel.cu")).read()
    assert re.findall(r"\bleft = ([^;]*);", text) == ["false", "bar_any(1, 128, !ok)"]
