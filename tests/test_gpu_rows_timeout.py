"""The bounded waits of prompt and tree attention: with pages withheld from the
page loads (the library's test hook) every wait gives up after its limit, the
call ends with the device error bit, and the next call is right."""
import time

import pytest
import torch

import speculative_decode_verify_kv_gb300 as T
from rows_common import Rows

pytestmark = pytest.mark.gpu

WAIT_US = 20000


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decode_verify_kv_gb300 import _build
    _build.build()
    T.load()
    T.trtv_get_device_error()
    yield
    T.trtv_test_withhold_pages(-1)


@pytest.mark.parametrize("pages", [0, 1, 2, 5])
@pytest.mark.parametrize("kind,hq,hk,d,fp8", [("prompt", 32, 4, 128, False), ("prompt", 8, 2, 64, False),
                                              ("prompt", 32, 4, 128, True), ("tree", 32, 4, 128, False),
                                              ("tree", 32, 4, 128, True), ("tree", 8, 2, 64, False)])
def test_withheld_pages_end_the_call(kind, hq, hk, d, fp8, pages):
    new = [16, 9, 12] if kind == "tree" else [300, 40, 129]
    p = Rows(new, [2000, 3000, 100], hq, hk, d, fp8=fp8, num_ctas=8)
    m = p.tree_masks()
    go = (lambda: p.tree(m)) if kind == "tree" else p.prompt
    want = go()
    torch.cuda.synchronize()
    assert T.trtv_get_device_error() == 0
    T.trtv_test_withhold_pages(pages, WAIT_US)
    try:
        t = time.perf_counter()
        go()
        torch.cuda.synchronize()
        took = time.perf_counter() - t
    finally:
        T.trtv_test_withhold_pages(-1)
    assert T.trtv_get_device_error() & T.DEVERR_TIMEOUT
    assert took < 2, took
    assert torch.equal(go(), want)
    assert T.trtv_get_device_error() == 0
