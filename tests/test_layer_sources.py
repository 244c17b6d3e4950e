"""Rules of the layer operators' kernel sources that no output shows (CPU)."""
import os
import re

import pytest

import fake_quant_numerics_gb300 as fq

CSRC = os.path.join(os.path.dirname(fq.__file__), "csrc")


def kernels(name):
    """(kernel name, parameters, body) of every kernel of a source file."""
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    for m in re.finditer(r"__global__", text):
        head = re.compile(r"\b(k_\w+)\s*\(").search(text, m.end())
        depth, i = 1, head.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(text[i], 0)
            i += 1
        start = text.index("{", i)
        depth, j = 1, start + 1
        while depth:
            depth += {"{": 1, "}": -1}.get(text[j], 0)
            j += 1
        yield head.group(1), text[head.end():i - 1], text[start:j]


@pytest.mark.parametrize("name", ["kernels_w4.cu", "kernels_norm.cu", "kernels_few.cu", "kernels_dense.cu"])
def test_chained_kernels_read_what_others_write_coherently(name):
    """A kernel that waits for the call's previous one may be resident while its input
    is written.  The read-only path (__ldg, or const __restrict__ parameters, which the
    compiler takes for it) asks for data that nobody writes meanwhile and may be moved
    across the wait: only weights and their parameters, which no kernel of the call
    writes, are read through it."""
    found = 0
    for kernel, params, body in kernels(name):
        if "pdl_wait" not in body:
            continue
        found += 1
        assert not re.search(r"const\s+\w+\s*\*\s*__restrict__", params), kernel
        for arg in re.findall(r"__ldg\(((?:[^()]|\([^()]*\))*)\)", body):
            assert re.search(r"\bw\.", arg), (kernel, arg)
    assert found
