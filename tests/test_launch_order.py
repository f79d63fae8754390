"""Kernels that are launched beside the tail of the one before them wait for it before
they touch memory.  griddepcontrol.wait is what makes an earlier kernel's writes visible,
and those of the kernels before that one, which it waited for itself: a kernel that reads
ahead of its wait is promised neither.  So the wait stands once, in every thread's way,
and no global access comes before it."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "speculative_decoding_draft_dspark_gb300", "csrc")
WAIT = "wait_for_earlier_kernel();"


def kernels(name):
    """(kernel, its body's lines) of a file's kernels."""
    with open(os.path.join(CSRC, name)) as f:
        lines = re.sub(r"//[^\n]*", "", f.read()).split("\n")
    i = 0
    while i < len(lines):
        if lines[i].lstrip().startswith("__global__"):
            head = lines[i]
            while "{" not in lines[i]:
                i += 1
                head += " " + lines[i].strip()
            body = []
            while lines[i + 1] != "}":
                i += 1
                body.append(lines[i])
            yield re.search(r"(\w+)\s*\((?:const|float|int|HeadParams)", head).group(1), body
        i += 1


@pytest.mark.parametrize("name", ["adjust.cu", "attention.cu", "rotary.cu", "norm.cu", "head_loss.cu"])
def test_every_thread_waits_before_it_reads(name):
    found = list(kernels(name))
    with open(os.path.join(CSRC, name)) as f:
        launched = set(re.findall(r"launch_overlapped\((\w+_kernel)\b", f.read()))
    assert launched and launched <= {k for k, _ in found}
    for kernel, body in found:
        at = [i for i, line in enumerate(body) if "wait_for_earlier_kernel" in line]
        # a statement of the kernel's own block: not under a condition, a loop or in a lambda
        assert len(at) == 1 and body[at[0]] == "  " + WAIT, kernel
        before = "\n".join(body[:at[0]])
        assert "return;" not in before, kernel
        # arguments by value (sizes) may be used; the pointers among them may not
        assert not re.search(r"\b[pa]\.\w+\s*(\[|->)|\*\s*[pa]\.\w+\s*\)|__ld|tma_load|cp_async|row_span\(|"
                             r"raise_status\(", before), kernel
