"""Packed-row calls at the limits that the header gives: the largest batch, the
most heads, the last cache positions that a page table can hold."""
import math

import pytest
import torch

import speculative_decode_verify_kv_gb300 as T
from rows_common import Rows, norm_rope, rope_table
from test_gpu_rows_attn import check
from test_gpu_rows_stage import check_stage, commit, commit_ref, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decode_verify_kv_gb300 import _build
    _build.build()
    T.load()
    T.trtv_get_device_error()


@pytest.mark.parametrize("fp8,qo_len", [(False, 3), (False, 4096), (True, 3), (True, 4096)])
def test_largest_batch(fp8, qo_len):
    new = [(i * 7) % 4 for i in range(2048)]
    p = Rows(new, [(i * 37) % 100 for i in range(2048)], 2, 1, 128, fp8=fp8, qo_len=qo_len, pad=5)
    check(p, p.prompt())
    if qo_len <= 128:
        m = p.tree_masks()
        check(p, p.tree(m), m)
    check_stage(p, 128, False)


@pytest.mark.parametrize("hq,hk,d,fp8", [(65536, 512, 64, False), (1024, 512, 128, True)])
def test_most_heads(hq, hk, d, fp8):
    p = Rows([3, 2], [130, 5], hq, hk, d, fp8=fp8)
    check(p, p.prompt())
    m = p.tree_masks("random")
    check(p, p.tree(m), m)
    raw = torch.uint8 if fp8 else torch.int16
    want, lens = commit_ref(p, [[0, 2], [1]], p.pool.view(raw))
    got = commit(p, [[0, 2], [1]])
    assert got.tolist() == lens and torch.equal(p.pool.view(raw), want)
    check_stage(p, 64, False)


@pytest.mark.parametrize("fp8", [False, True])
def test_last_positions_of_the_largest_table(fp8):
    """2^23 pages, 2^30 positions: every page but the last is the same slot, so the reference needs two.  The sums over the
    7 million positions of a CTA are binary32: 27600 pages of eight steps on each softmax group, each cut off by up to a
    unit in the last place (2^-23) of a sum that grows evenly, 2^-24 of it on average over the way: 221000 * 2^-24."""
    p = Rows([3], [125], 4, 1, 128, fp8=fp8)
    if fp8:
        p.pool[(p.pool & 127) == 127] = 0
    else:
        p.pool[p.pool.isnan()] = 0
    p.mp = p.geom.max_pages_per_req = 1 << 23
    slot, last = int(p.table[0, 0]), (int(p.table[0, 0]) + 1) % p.slots
    p.table = torch.full((1, p.mp), slot, dtype=torch.int32, device=p.dev)
    p.table[0, -1] = last
    p.kv, p.ctx = [1 << 30], [(1 << 30) - 3]
    p.kv_lens.fill_(1 << 30)
    q, k, v, w = inputs(p)
    tab, pos = rope_table(16, 128).to(p.dev), torch.tensor([3, 4, 15], dtype=torch.int32, device=p.dev)
    p.q = torch.empty_like(p.q)
    T.trtv_norm_rope_stage(p.geom, q, k, v, *w, 1e-6, tab, 128, False, pos, p.indptr, p.q, p.pool, p.table, p.kv_lens)
    vals = p.values()
    ref = norm_rope(k, w[1], 1e-6, tab[pos.long()], 128, False) / p.k_scale
    got = vals[last * 2, 3, :, 29:32].transpose(0, 1)
    assert ((got - ref).abs() <= ref.abs() * (2.0 ** -4 if fp8 else 2.0 ** -8) * 1.001 + ref.abs().amax() * 2.0 ** -15 + 2.0 ** -10).all()
    out = p.prompt(T.TRTV_F32)
    torch.cuda.synchronize()
    assert T.trtv_get_device_error() == 0
    K, V = (torch.cat([vals[s * 2 + kv, :, 0].reshape(128, 128) for s in (slot, last)]) * scale
            for kv, scale in ((0, p.k_scale), (1, p.v_scale)))
    x = torch.einsum("thd,pd->thp", p.q.double(), K) * p.geom.sm_scale
    x[..., :128] += math.log(p.mp - 1)   # the same page that often
    for t in range(3):
        x[t, :, 128 + 126 + t:] = -math.inf
    wgt = torch.softmax(x, -1)
    off = (out.double() - wgt @ V).abs() / (wgt @ V.abs())
    assert off.max().item() <= (2.0 ** -11 if fp8 else 2.0 ** -8) + 2.0 ** -11 + 221000 * 2.0 ** -24, off.max().item()
    path, plen = (torch.tensor(a, dtype=torch.int32, device=p.dev) for a in ([[0, 2]], [2]))
    want = p.pool.clone()
    want[last * 2:last * 2 + 2, 3, :, 30] = want[last * 2:last * 2 + 2, 3, :, 31]
    T.trtv_tree_commit(p.geom, p.pool, p.table, p.kv_lens, p.indptr, path, plen, p.kv_lens)
    assert p.kv_lens.tolist() == [(1 << 30) - 1] and T.trtv_get_device_error() == 0
    assert torch.equal(p.pool.view(torch.uint8), want.view(torch.uint8))
