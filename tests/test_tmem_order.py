"""Read from the source: no kernel takes tensor memory before it has waited for the kernel before it on the stream.

pdl_enter lets the next kernel start and waits for the last one.  tcgen05.alloc waits without a limit for columns that
another CTA of the SM holds; a CTA that held its own through that wait could keep them from a CTA of the very kernel it
waits for."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_attention_fp4_quant_b200", "csrc")
SOURCES = sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh")))


def code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def bodies(text, head):
    """The brace-matched bodies of the functions whose declarations match `head`, with their names."""
    for m in re.finditer(head, text):
        start = text.index("{", m.end())
        depth, at = 0, start
        while True:
            depth += {"{": 1, "}": -1}.get(text[at], 0)
            at += 1
            if depth == 0:
                break
        yield m.group(1), text[start:at]


def allocating_functions():
    """tmem_alloc and the device functions that call it."""
    names = {"tmem_alloc"}
    for f in SOURCES:
        for name, body in bodies(code(f), r"__device__ __forceinline__ void (\w+)\([^;{]*\)\s*(?={)"):
            if "tmem_alloc(" in body:
                names.add(name)
    return names


def kernels():
    call = re.compile(r"\b(?:%s)\(" % "|".join(sorted(allocating_functions())))
    for f in SOURCES:
        for name, body in bodies(code(f), r"__global__ void[^;{]*?(\w+_kernel)\([^;{]*\)\s*(?={)"):
            m = call.search(body)
            if m:
                yield f, name, body, m.start()


def test_every_allocation_is_looked_at():
    """Each source that allocates has a kernel in the list, or a function that the kernels of the list call."""
    found = {f for f, _, _, _ in kernels()}
    assert {"index_tc.cu", "index_cluster.cu", "index_mq.cu", "pages_attn.cu"} <= found
    for f in SOURCES:
        if "tmem_alloc(" in code(f) and f.endswith(".cu"):
            assert f in found


@pytest.mark.parametrize("f,name,body,at", [pytest.param(*k, id=f"{k[0]}:{k[1]}") for k in kernels()])
def test_allocation_behind_the_wait(f, name, body, at):
    assert -1 < body.find("pdl_enter();") < at
