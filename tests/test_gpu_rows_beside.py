"""Prompt and tree attention before, after and beside other kernels that take
tensor memory: the verify step's, their own and a library's products, on two
streams.  Every result is what the call gives by itself."""
import pytest
import torch

import speculative_decode_verify_kv_gb300 as T
from rows_common import Rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decode_verify_kv_gb300 import _build
    _build.build()
    T.load()
    T.trtv_get_device_error()


def test_beside_other_kernels():
    from speculative_decode_verify_kv_gb300 import workloads as W
    from speculative_decode_verify_kv_gb300.runtime import DeviceVerify
    small = Rows([200, 30], [0, 900], 8, 2, 64, seed=1)
    tree = Rows([16, 8], [2000, 100], 32, 4, 128, seed=2)
    codes = Rows([16, 8], [2000, 100], 32, 4, 128, seed=2, fp8=True)
    m = tree.tree_masks()
    step = DeviceVerify(W.make_problem(kv_lens=[700, 300, 2000], qo_len=4, num_q_heads=16, num_kv_heads=2, head_dim=128, seed=3,
                                       topk=2, out_dtype="f32"))
    x = torch.randn(1024, 1024, device="cuda").bfloat16()
    calls = dict(small=small.prompt, tree=lambda: tree.tree(m), codes=lambda: codes.tree(m), dense=lambda: step.dense().clone(),
                 product=lambda: x @ x)
    want = {k: f() for k, f in calls.items()}
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    orders = (["product", "small", "tree", "product", "codes", "small"],
              ["dense", "tree", "product", "small", "product", "dense", "codes"])
    for _ in range(5):
        got = []
        for s, order in zip(streams, orders):
            with torch.cuda.stream(s):
                got += [(k, calls[k]()) for k in order]
        torch.cuda.synchronize()
        for k, out in got:
            assert torch.equal(out, want[k]), k
    assert T.trtv_get_device_error() == 0
