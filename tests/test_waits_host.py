"""The bounded waits of the tensor-core kernels, by their source: a wait that
gives up would take seconds on a GPU, so what follows one is shown by reading."""

import os
import re

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "ring_allreduce_gb300", "csrc")


def blocks_of_one_thread(text):
    """The parts of a kernel that one lane alone runs: what `if (... lane == 0 ...)` guards."""
    spans = []
    for m in re.finditer(r"if \([^{;]*lane == 0[^{;]*\) \{", text):
        depth, i = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        spans.append((m.end(), i))
    return spans


@pytest.mark.parametrize("name", ["ra_ffn_mma.cuh", "ra_ffn_few.cuh"])
def test_a_warp_waits_as_one(name):
    """Where all lanes wait, all have the same answer before they load from
    tensor memory or synchronise together; one thread's waits are its own."""
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    alone = blocks_of_one_thread(text)
    calls = [(m.start(), bool(m.group(1))) for m in re.finditer(r"\bwait(\.warp)?\((?=&sh\.|full\b)", text)]
    assert len(calls) >= 3 and any(warp for _, warp in calls)
    for at, warp in calls:
        inside = any(lo <= at < hi for lo, hi in alone)
        line = text[:at].count("\n") + 1
        assert warp != inside, f"{name}: the wait in line {line}"
