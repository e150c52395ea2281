"""What the kernels' sources have to hold and no run shows."""
import glob
import math
import os
import re

import pytest
import torch

from selective_state_space_34_b200 import build


def _statements():
    """(file, text) of every inline assembly statement."""
    for path in sorted(glob.glob(os.path.join(build.CSRC, "*.cu*"))):
        with open(path) as f:
            text = f.read()
        for m in re.finditer(r"\basm\b", text):
            at, depth = text.index("(", m.end()), 0
            for end in range(at, len(text)):  # the matching bracket (those in strings pair up)
                depth += (text[end] == "(") - (text[end] == ")")
                if depth == 0:
                    break
            yield os.path.basename(path), text[m.start():end + 1]


@pytest.mark.parametrize("what", ["cp.async", "mbarrier", "bar.sync"])
def test_copies_and_waits_order_memory(what):
    """A thread that reads its own slots behind a wait has nothing but the wait itself to keep the reads there: an asynchronous copy,
    its commit and its wait tell the compiler that they touch memory, and so do barriers."""
    found = [(f, s) for f, s in _statements() if what in s]
    assert found
    bad = ["%s: %s" % (f, " ".join(s.split())) for f, s in found if '"memory"' not in s]
    assert not bad, "\n".join(bad)


def test_clamped_gates_have_finite_denominators():
    """bf16 gates are clamped to -41.5 - bias rounded to bf16: up to the bias from which the arguments themselves are clamped, the product of two
    denominators 1 + e^-v stays below the largest fp32 value."""
    with open(os.path.join(build.CSRC, "ssm_lru.cu")) as f:
        limit = float(re.search(r"!\(fabsf\(bias\) <= ([0-9.]+)f\)", f.read()).group(1))
    bias = torch.arange(-limit, limit + 0.125, 0.125, dtype=torch.float32)
    low = (-41.5 - bias).to(torch.bfloat16)
    worst = float((low.double() + bias.double()).min())
    assert worst >= -44.0 and 2 * math.log2(1 + math.exp(-worst)) < 127.9
