"""Kernels that may start before their predecessor has finished (programmatic dependent
launch): what the predecessor writes is not constant for their lifetime, so it may not be read
through the read-only path.  Read from the sources; no GPU."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "csr_spmm_gb300", "csrc")
INPUTS = {"row_ptr", "col_idx", "values"}       # the caller's arrays: no kernel writes them


def _kernels():
    """(file, name, parameters, body) of every kernel."""
    for name in sorted(os.listdir(CSRC)):
        if not name.endswith((".cu", ".cuh")):
            continue
        with open(os.path.join(CSRC, name)) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for m in re.finditer(r"__global__", text):
            open_at = text.index("{", m.end())
            head = text[m.end():open_at]
            depth, at = 0, open_at
            while True:
                depth += {"{": 1, "}": -1}.get(text[at], 0)
                at += 1
                if depth == 0:
                    break
            kernel = re.search(r"(\w+)\s*\(([^()]*)\)\s*$", head)
            yield name, kernel.group(1), kernel.group(2), text[open_at:at]


def test_what_a_predecessor_writes_is_read_through_ordinary_loads():
    waiting = 0
    for file, name, params, body in _kernels():
        if "wait_for_predecessor()" not in body:
            continue
        waiting += 1
        read_only = set(re.findall(r"const\s+[\w:<>]+\s*\*\s*__restrict__\s+(\w+)", params))
        assert read_only <= INPUTS, f"{file}: {name} declares {read_only - INPUTS} constant"
        assert "__ldg(" not in body, f"{file}: {name} reads through __ldg"
    assert waiting >= 6
