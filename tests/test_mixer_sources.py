"""The sources of the mixer kernels, read as text (no GPU): a kernel that may start before the one
ahead of it in the stream has ended waits first (grid_begin), and nothing that it reads may be loaded
ahead of that wait.  A __restrict__ pointer, or a load of the read-only path, lets the compiler do so."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "spatially_sharded_cnn_gb300", "csrc")


def kernels(name):
    """(name, parameters, body) of every __global__ function of a source file."""
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    found = []
    for m in re.finditer(r"__global__", text):
        head = re.compile(r"(\w+_kernel)\s*\(").search(text, m.end())
        at, depth = head.end(), 1
        while depth:
            depth += {"(": 1, ")": -1}.get(text[at], 0)
            at += 1
        params, start = text[head.end():at - 1], text.index("{", at)
        end, depth = start + 1, 1
        while depth:
            depth += {"{": 1, "}": -1}.get(text[end], 0)
            end += 1
        found.append((head.group(1), params, text[start:end]))
    return found


@pytest.mark.parametrize("source", ["groupnorm.cu", "causal_conv.cu", "scan.cu", "scan_fwd.cu", "scan_bwd.cu",
                                    "scan_carry.cu", "reduce.cu"])
def test_reads_stay_behind_the_wait(source):
    waiting = [k for k in kernels(source) if "grid_begin()" in k[2]]
    assert waiting
    for name, params, body in waiting:
        assert body.lstrip("{ \n").startswith("grid_begin();"), f"{name} acts before its wait"
        assert "__restrict__" not in params + body, f"{name} has a __restrict__ pointer"
        assert "__ldg" not in body and "global.nc" not in body, f"{name} reads through the read-only path"


@pytest.mark.parametrize("source", ["rows.cuh", "scan.cuh"])
def test_shared_loads_stay_behind_the_wait(source):
    """The functions that those kernels share: no such load, and no hinted one that the compiler may move."""
    with open(os.path.join(CSRC, source)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    for word in ("__restrict__", "__ldg", "__ldcs", "__ldcg", "__ldca", "global.nc"):
        assert word not in text, word
    for m in re.finditer(r"asm( volatile)?\(\s*\"(ld|cp|prefetch)\b[^\"]*", text):
        assert m.group(1), f"a load that may move: {m.group(0)}"
