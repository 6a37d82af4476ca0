"""Host-side checks of the packed-row calls, without a GPU: every refusal
happens before any CUDA call."""
import ctypes

import pytest

import speculative_decode_verify_kv_gb300 as T
from speculative_decode_verify_kv_gb300 import _build

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 4


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return T.load()


def geom(**over):
    g = dict(batch=2, qo_len=40, num_q_heads=8, num_kv_heads=2, head_dim=128, max_pages_per_req=3, num_slots=8,
             slot_stride=2, kv_dtype=0, sm_scale=0.125, k_scale=1.0, v_scale=1.0, num_ctas=4)
    g.update(over)
    return T.Geom(**g)


def calls(lib, g, rows=80, indptr=16):
    """Statuses of the four calls with otherwise valid arguments (never launched: the geometry is bad)."""
    n = T.NormRope(q=16, k=16, v=16, q_stride=4096, k_stride=4096, v_stride=4096, rope_table=16, table_len=9, rot_dim=64)
    r = ctypes.byref(g)
    return {lib.trtv_norm_rope_stage(r, ctypes.byref(n), indptr, rows, 16, 16, 16, 16, None),
            lib.trtv_prompt_attn(r, 16, 16, 16, 16, indptr, rows, 16, 0, 256, 1 << 40, None),
            lib.trtv_verify_tree(r, 16, 16, 16, 16, indptr, rows, 16, 16, 0, 256, 1 << 40, None),
            lib.trtv_tree_commit(r, 16, 16, 16, indptr, 16, 16, 4, 16, None)}


@pytest.mark.parametrize("over,status", [
    (dict(batch=0), INVALID), (dict(qo_len=0), INVALID), (dict(num_q_heads=6, num_kv_heads=4), INVALID),
    (dict(num_kv_heads=0), INVALID), (dict(slot_stride=1), INVALID), (dict(max_pages_per_req=0), INVALID),
    (dict(num_slots=0), INVALID), (dict(kv_dtype=2), INVALID), (dict(sm_scale=0.0), INVALID),
    (dict(sm_scale=float("nan")), INVALID), (dict(k_scale=0.0), INVALID), (dict(v_scale=float("inf")), INVALID),
    (dict(num_ctas=-1), INVALID), (dict(num_ctas=1025), INVALID), (dict(head_dim=96), UNSUPPORTED),
    (dict(kv_dtype=1, head_dim=64), UNSUPPORTED), (dict(batch=2049), UNSUPPORTED),
    (dict(num_q_heads=129, num_kv_heads=1), UNSUPPORTED), (dict(num_slots=1 << 20, slot_stride=8), UNSUPPORTED),
    (dict(max_pages_per_req=(1 << 23) + 1), UNSUPPORTED), (dict(num_q_heads=65664, num_kv_heads=513), UNSUPPORTED),
    (dict(sm_scale=1e-20), INVALID), (dict(sm_scale=1e-12, k_scale=1e-12), INVALID), (dict(sm_scale=1e30, k_scale=1e30), INVALID),
])
def test_geometry(lib, over, status):
    g = geom(**over)
    assert calls(lib, g) == {status}
    assert lib.trtv_workspace_bytes_rows(ctypes.byref(g)) == 0


@pytest.mark.parametrize("over", [dict(), dict(head_dim=64), dict(kv_dtype=1)])
@pytest.mark.parametrize("qo_len", [1, 4096])
def test_largest_batch(lib, over, qo_len):
    """Every batch up to the documented limit has a workspace (its shared memory fits)."""
    assert lib.trtv_workspace_bytes_rows(ctypes.byref(geom(batch=2048, qo_len=qo_len, **over))) > 0


def test_null_geometry(lib):
    assert lib.trtv_workspace_bytes_rows(None) == 0
    assert lib.trtv_prompt_attn(None, 16, 16, 16, 16, 16, 8, 16, 0, 256, 1 << 40, None) == INVALID
    assert lib.trtv_verify_tree(None, 16, 16, 16, 16, 16, 8, 16, 16, 0, 256, 1 << 40, None) == INVALID
    assert lib.trtv_tree_commit(None, 16, 16, 16, 16, 16, 16, 4, 16, None) == INVALID
    assert lib.trtv_norm_rope_stage(None, ctypes.byref(T.NormRope()), 16, 8, 16, 16, 16, 16, None) == INVALID


def test_attention_arguments(lib):
    r = ctypes.byref(geom())
    need = lib.trtv_workspace_bytes_rows(r)
    assert need > 0
    good = [r, 16, 16, 16, 16, 16, 80, 16, 0, 256, need, None]
    for i, bad, st in ((1, 0, INVALID), (2, 0, INVALID), (3, 0, INVALID), (4, 0, INVALID), (7, 0, INVALID),
                       (1, 24, INVALID), (2, 24, INVALID), (7, 8, INVALID), (3, 18, INVALID), (4, 18, INVALID),
                       (5, 18, INVALID), (6, -1, INVALID), (8, 1, INVALID), (8, 3, INVALID), (9, 0, WORKSPACE),
                       (9, 128, WORKSPACE), (10, need - 1, WORKSPACE)):
        a = list(good)
        a[i] = bad
        assert lib.trtv_prompt_attn(*a) == st, (i, bad)
        assert lib.trtv_verify_tree(*a[:7], 16, *a[7:]) == st, (i, bad)
    assert lib.trtv_verify_tree(*good[:7], 0, *good[7:]) == INVALID
    assert lib.trtv_verify_tree(*good[:7], 18, *good[7:]) == INVALID
    big = ctypes.byref(geom(qo_len=129))
    assert lib.trtv_verify_tree(big, *good[1:7], 16, *good[7:]) == UNSUPPORTED
    # equal rows per request need batch * qo_len of them; no rows: nothing to do
    assert lib.trtv_prompt_attn(r, 16, 16, 16, 16, None, 79, 16, 0, 256, need, None) == INVALID
    assert lib.trtv_prompt_attn(r, None, None, None, None, 16, 0, None, 0, None, 0, None) == 0
    assert lib.trtv_verify_tree(r, None, None, None, None, 16, 0, 16, None, 0, None, 0, None) == 0


def test_stage_arguments(lib):
    r = ctypes.byref(geom())

    def call(rows=80, q_out=16, pool=16, table=16, lens=16, indptr=16, **over):
        f = dict(q=32, k=16, v=16, q_stride=1536, k_stride=1536, v_stride=1536, q_weight=16, k_weight=16, rope_table=16,
                 positions=16, table_len=9, rot_dim=64, interleaved=0, eps=1e-6)
        f.update(over)
        n = T.NormRope(**f)
        return lib.trtv_norm_rope_stage(r, ctypes.byref(n), indptr, rows, q_out, pool, table, lens, None)

    for over in (dict(q=0), dict(k=0), dict(v=0), dict(q=24), dict(k=8), dict(v=8), dict(q_stride=1016), dict(k_stride=248),
                 dict(v_stride=0), dict(q_stride=1540), dict(k_stride=260), dict(v_stride=-256), dict(q_weight=8),
                 dict(k_weight=8), dict(rope_table=0), dict(rope_table=8), dict(table_len=0), dict(rot_dim=-8),
                 dict(rot_dim=136), dict(rot_dim=12), dict(interleaved=2), dict(eps=-1.0), dict(eps=float("nan")),
                 dict(eps=float("inf")), dict(positions=18), dict(q_out=0), dict(q_out=24), dict(pool=0), dict(pool=8),
                 dict(table=0), dict(table=18), dict(lens=0), dict(lens=18), dict(indptr=18), dict(rows=-1),
                 dict(indptr=None, rows=79), dict(q=16)):  # the last: q_out is q, whose rows lie apart
        assert call(**over) == INVALID, over
    assert lib.trtv_norm_rope_stage(r, None, 16, 8, 16, 16, 16, 16, None) == INVALID
    assert call(rows=0, q=0, q_out=0) == 0
    big = geom(num_q_heads=64, num_kv_heads=64)
    n = T.NormRope(q=16, k=16, v=16, q_stride=8192, k_stride=8192, v_stride=8192)
    assert lib.trtv_norm_rope_stage(ctypes.byref(big), ctypes.byref(n), 16, 2 ** 31 - 1, 32, 16, 16, 16, None) == UNSUPPORTED


def test_commit_arguments(lib):
    good = [ctypes.byref(geom()), 16, 16, 16, 16, 16, 16, 4, 16, None]
    for i, bad in ((1, 0), (1, 8), (2, 0), (2, 18), (3, 0), (3, 18), (4, 18), (5, 0), (5, 18), (6, 0), (6, 18), (7, 0), (7, -1),
                   (8, 0), (8, 18)):
        a = list(good)
        a[i] = bad
        assert lib.trtv_tree_commit(*a) == INVALID, (i, bad)
    a = list(good)
    a[0] = ctypes.byref(geom(qo_len=129))
    assert lib.trtv_tree_commit(*a) == UNSUPPORTED


def test_no_rows_no_buffers(lib):
    """A step without new tokens: empty tensors have no address."""
    r = ctypes.byref(geom())
    assert lib.trtv_verify_tree(r, None, None, None, None, 16, 0, None, None, 0, None, 0, None) == 0
    assert lib.trtv_prompt_attn(r, None, None, None, None, 16, 0, None, 0, None, 0, None) == 0
    assert lib.trtv_verify_tree(r, 16, 16, 16, 16, 16, -1, None, 16, 0, 256, 1 << 40, None) == INVALID


@pytest.mark.parametrize("v_scale", [0.0, -0.0])
def test_stage_divides_by_no_zero(lib, v_scale):
    """Staging into an E4M3 cache divides the values by v_scale."""
    n = T.NormRope(q=32, k=16, v=16, q_stride=4096, k_stride=4096, v_stride=4096)
    r = ctypes.byref(geom(kv_dtype=1, v_scale=v_scale))
    assert lib.trtv_norm_rope_stage(r, ctypes.byref(n), 16, 80, 16, 16, 16, 16, None) == INVALID
