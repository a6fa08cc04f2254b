"""A kernel that may start under the one ahead of it takes tensor memory only once that one has ended:
else each could hold what the other waits for, for ever.  Read from the sources, as nothing may try it."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_deltanet_linear_bwd_gb300", "csrc")


def kernels():
    """(file: name, body) of every __global__ function, comments removed."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        text = re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", open(path).read(), flags=re.S))
        for m in re.finditer(r"__global__[^;{]*?(\w+)\s*\((?:[^(){}]|\([^()]*\))*\)\s*\{", text):
            depth, i = 1, m.end()
            while depth:
                depth += {"{": 1, "}": -1}.get(text[i], 0)
                i += 1
            yield f"{os.path.basename(path)}: {m.group(1)}", text[m.end():i]


TAKERS = [(n, b) for n, b in kernels() if "tmem_alloc" in b]


def test_the_kernels_with_tensor_memory_are_found():
    files = {n.split(":")[0] for n, _ in TAKERS}
    sources = {os.path.basename(p) for p in glob.glob(os.path.join(CSRC, "*.cu")) if "tmem_alloc" in open(p).read()}
    assert files == sources and len(TAKERS) >= 8


@pytest.mark.parametrize("name,body", TAKERS, ids=[n for n, _ in TAKERS])
def test_tensor_memory_is_taken_after_the_wait(name, body):
    wait = re.search(r"pdl_enter\(\)|griddepcontrol\.wait", body)
    assert wait and wait.start() < body.index("tmem_alloc")
    # the wait may be left out only behind a kernel that has none and began when all before it had ended
    lead = body[:wait.start()].rstrip().removesuffix('asm volatile("').rstrip()
    if lead.endswith(")"):
        assert lead.endswith("if (!a.early_w)"), lead[-80:]
