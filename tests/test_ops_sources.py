"""Rules that the sources of the pool operators keep, read from the sources: no test on a GPU can show a
load that is right by luck."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OPS = os.path.join(ROOT, "speculative_decode_persistent_gb300", "csrc", "ops")
FILES = sorted(f for f in os.listdir(OPS) if f.endswith((".cu", ".cuh")))


def _code(name):
    """A source without its comments."""
    s = open(os.path.join(OPS, name)).read()
    return re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", s, flags=re.S))


@pytest.mark.parametrize("name", FILES)
def test_no_read_only_loads(name):
    """Kernels that are launched while the one before them still writes take what it wrote with ordinary loads:
    read-only ones hold only for memory that nothing writes while the kernel runs, and no wait orders them."""
    assert not re.search(r"__ldg\b|\.global\.nc|__restrict__|\btex1D|ldu\.", _code(name))


@pytest.mark.parametrize("name", FILES)
def test_kernels_wait_for_the_one_before(name):
    """Every kernel waits for the end of the one before it in the stream, at the top level of its body (so that
    every thread of every block does), and before it lets its own second part start what follows."""
    code = _code(name)
    for m in re.finditer(r"__global__ void[^;{]*?(\w+)\(const [^{]*\{", code):
        depth, i, top = 1, m.end(), ""
        while depth:
            c = code[i]
            depth += (c == "{") - (c == "}")
            top += c if depth == 1 else ""
            i += 1
        assert "wait_for_previous();" in top, m.group(1)
        before = top[:top.index("wait_for_previous();")]
        assert "return" not in before, m.group(1)
    assert ("__global__" in code) <= ("wait_for_previous();" in code)
