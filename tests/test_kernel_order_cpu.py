"""Order of the steps that start a kernel, read from the sources.

A kernel of a programmatic launch chain is scheduled while the previous one
still runs.  Were it to take tensor memory before it has waited for that one, a
CTA of the previous kernel on the same SM could wait for the tensor memory of a
CTA that waits for it: such an order is never run, only read."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "speculative_decode_verify_kv_gb300", "csrc")


def kernels():
    """(file, kernel, body without comments) of every kernel that takes tensor memory."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"__global__[^;{]*?(\w+_kernel)\s*\([^;{]*\)\s*\{", text):
            depth, i = 1, m.end()
            while depth:
                depth += {"{": 1, "}": -1}.get(text[i], 0)
                i += 1
            body = text[m.end():i]
            if "tmem_alloc(" in body:
                yield os.path.basename(path), m.group(1), body


def test_kernels_are_found():
    assert {k for _, k, _ in kernels()} == {"attn_umma_kernel", "attn_pm_kernel", "proxy_umma_kernel", "rows_attn_kernel"}


@pytest.mark.parametrize("kernel", ["attn_umma_kernel", "attn_pm_kernel", "proxy_umma_kernel", "rows_attn_kernel"])
def test_tensor_memory_after_the_wait(kernel):
    body = {k: b for _, k, b in kernels()}[kernel]
    assert 0 <= body.index("pdl_wait(") < body.index("tmem_alloc(")
