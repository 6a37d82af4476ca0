"""Packed-row calls on qo_indptr tables with wrong entries: the requests whose
own entries do not fit are left out and flagged, every other one is served as
if the table were right."""
import pytest
import torch

import speculative_decode_verify_kv_gb300 as T
from rows_common import Rows, rope_table
from test_gpu_rows_attn import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decode_verify_kv_gb300 import _build
    _build.build()
    T.load()
    T.trtv_get_device_error()


# tokens of the requests, and {entry: wrong value}; the entries of a request that stays keep their values
TABLES = [([4, 2, 2], {2: -9}), ([4, 2, 2], {2: 0}), ([4, 2, 2], {1: -1}), ([4, 2, 2], {1: 7}), ([4, 2, 2], {3: -3}), ([4, 2, 2], {3: 9}), ([4, 2, 2], {0: 1}),
          ([4, 2, 2], {2: 1 << 30}), ([4, 4], {2: -3}), ([4, 4], {2: 9}), ([4, 4], {1: 9}), ([2] * 64, {40: -9}), ([2] * 64, {40: 3}),
          ([2] * 64, {40: 1000}), ([2] * 64, {1: -1, 33: -5, 34: -6}), ([1, 3] * 20, {20: -1}),
          ([0, 3, 0, 2] * 300, {500: -(1 << 31), 900: 2})]
IDS = [f"{len(new)}-{'-'.join(map(str, bad))}-{list(bad.values())[0]}" for new, bad in TABLES]


def spoil(p, bad):
    """Requests that stay, after the table's entries are overwritten."""
    t = p.indptr.tolist()
    for i, v in bad.items():
        t[i] = v
    keep = []
    for b in range(p.B):
        lo, hi = t[b], t[b + 1]
        keep.append(0 <= lo <= hi <= p.rows and hi - lo <= p.qo_len and (b > 0 or lo == 0))
        assert not keep[-1] or p.new[b] == hi - lo
    assert not all(keep)
    p.indptr.copy_(torch.tensor(t, dtype=torch.int32))
    return keep


def rows_of(p, keep):
    return torch.tensor([keep[b] for b in range(p.B) for _ in range(p.new[b])] + [False] * (p.rows - p.toks), device=p.dev)


@pytest.mark.parametrize("new,bad", TABLES, ids=IDS)
def test_stage(new, bad):
    p = Rows(new, [(13 * b) % 90 for b in range(len(new))], 4, 2, 64, seed=len(new))
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(p.rows, h, 64, generator=g).to(torch.bfloat16).to(p.dev) for h in (4, 2, 2))
    tab = rope_table(max(p.kv) + 1, 64).to(p.dev)
    before = p.pool.clone()

    def stage():
        out, pool = torch.full_like(q, 3.0), before.clone()
        T.trtv_norm_rope_stage(p.geom, q, k, v, None, None, 0.0, tab, 64, False, None, p.indptr, out, pool, p.table, p.kv_lens)
        return out, pool.view(torch.int16), T.trtv_get_device_error()

    q_ok, pool_ok, err = stage()
    assert err == 0
    keep = spoil(p, bad)
    q_bad, pool_bad, err = stage()
    assert err == T.DEVERR_INDPTR
    live = rows_of(p, keep)
    assert torch.equal(q_bad[live], q_ok[live])
    assert (q_bad[~live] == 3).all()
    want = before.view(torch.int16).clone()
    for b in range(p.B):
        for pos in range(p.ctx[b], p.kv[b]) if keep[b] else ():
            at = int(p.table[b, pos // 128]) * p.stride
            want[at:at + 2, pos % 128 // 32, :, pos % 32] = pool_ok[at:at + 2, pos % 128 // 32, :, pos % 32]
    assert torch.equal(pool_bad, want)


@pytest.mark.parametrize("call", ["prompt", "tree"])
@pytest.mark.parametrize("new,bad", TABLES, ids=IDS)
def test_attention(new, bad, call):
    p = Rows(new, [(37 * b) % 300 for b in range(len(new))], 8, 2, 128, seed=len(new))
    mask = p.tree_masks() if call == "tree" else None
    keep = spoil(p, bad)
    out = p.prompt() if mask is None else p.tree(mask)
    live = rows_of(p, keep)
    check(p, out, mask, err=T.DEVERR_INDPTR, rows=live)
    assert (out[~live] == 7).all()


@pytest.mark.parametrize("new,bad", TABLES, ids=IDS)
def test_commit(new, bad):
    """The commit reads no rows, so it has no num_tokens: an entry that only passes it is no fault here."""
    p = Rows(new, [(13 * b) % 90 for b in range(len(new))], 4, 2, 64, seed=len(new))
    t = p.indptr.tolist()
    for i, v in bad.items():
        t[i] = v
    p.indptr.copy_(torch.tensor(t, dtype=torch.int32))
    keep = [0 <= lo <= hi and hi - lo <= p.qo_len and (b > 0 or lo == 0) for b, (lo, hi) in enumerate(zip(t, t[1:]))]
    # one node of every tree is kept
    node = [max(0, n - 1) for n in new]
    path = torch.tensor([[x] for x in node], dtype=torch.int32, device=p.dev)
    plen = torch.tensor([min(1, n) for n in new], dtype=torch.int32, device=p.dev)
    want, lens = p.pool.view(torch.int16).clone(), list(p.kv)
    for b in range(p.B):
        n = t[b + 1] - t[b]
        if not keep[b] or not n:
            continue
        ctx = p.kv[b] - n
        (s, sg, sr), (d, dg, dr) = ((int(p.table[b, c // 128]) * p.stride, c % 128 // 32, c % 32) for c in (ctx + node[b], ctx))
        want[d:d + 2, dg, :, dr] = want[s:s + 2, sg, :, sr]
        lens[b] = ctx + 1
    got = torch.full((p.B,), -7, dtype=torch.int32, device=p.dev)
    T.trtv_tree_commit(p.geom, p.pool, p.table, p.kv_lens, p.indptr, path, plen, got)
    assert T.trtv_get_device_error() == (0 if all(keep) else T.DEVERR_INDPTR)
    assert got.tolist() == lens
    assert torch.equal(p.pool.view(torch.int16), want)
