"""Kernels that are set up while the one before them runs wait for it before they read (no GPU).

griddepcontrol.wait makes what earlier kernels on the stream wrote visible to the grid that executes it,
and to no other.  So a kernel launched with programmatic serialization has it ahead of its first use
of an argument other than by prefetch; a wait of the kernel before it does not count.
"""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(__file__), "..", "selected_block_attention_gb300", "csrc")


def _body(text, at):
    """The braces' content that begins behind `at`."""
    begin = text.index("{", at)
    depth = 0
    for i in range(begin, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[begin:i]
    raise AssertionError("braces do not match")


def _kernels(text):
    """Kernels of a source file, comments left out: name and body."""
    text = re.sub(r"//[^\n]*", "", text)
    for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\([^()]*(?:\([^()]*\)[^()]*)*\)\s*)?(\w+)\s*\(", text):
        yield m.group(1), _body(text, text.index(")", m.end()))


def unsafe(text):
    """Kernels of the file launched by cudaLaunchKernelEx that read an argument before they wait."""
    found = []
    for name, body in _kernels(text):
        if re.search(rf"{name}(<[^;()]*?>)?\s*<<<", text):
            continue  # an ordinary launch begins when all before it has ended
        wait = re.search(r"griddepcontrol\.wait|paged_wait_before\(\)", body)
        ahead = body[:wait.start()] if wait else body
        if re.search(r"\bp\.\w+\s*(\[|\+|->)|\(.*\bp\s*[,)]|&p\.", ahead):
            found.append(name)
    return found


def test_block_sparse_gradients_wait_for_prep():
    with open(os.path.join(CSRC, "blocksparse_backward.cu")) as f:
        text = f.read()
    names = [name for name, _ in _kernels(text)]
    assert "bsa_bwd_prep_kernel" in names and len(names) >= 3
    assert unsafe(text) == []


@pytest.mark.parametrize("wait_at_the_end", [False, True])
def test_the_reading_sees_a_wait_that_comes_late(wait_at_the_end):
    text = """
    __global__ void __launch_bounds__(128, 1) late_kernel(const Params p) {
      %s
      int item = atomicAdd(&p.next[1], 1);
      float x = p.rows[item];
      %s
    }
    """
    wait = 'asm volatile("griddepcontrol.wait;" ::: "memory");'
    assert unsafe(text % (("", wait) if wait_at_the_end else (wait, ""))) == (["late_kernel"] if wait_at_the_end else [])
