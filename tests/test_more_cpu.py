"""Host-side checks of the E2M1 caches and of the page calls, without a GPU: every refusal happens before any CUDA call."""
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
    g = dict(batch=2, qo_len=4, num_q_heads=8, num_kv_heads=2, head_dim=128, max_pages_per_req=3, num_slots=8,
             slot_stride=2, kv_dtype=T.TRTV_FP4_E2M1, sm_scale=0.125, k_scale=1.0, v_scale=1.0, num_ctas=4)
    g.update(over)
    return T.Geom(**g)


def test_calls_without_a_4_bit_form(lib):
    r = ctypes.byref(geom())
    assert lib.trtv_verify_dense_noalloc(r, 16, 16, 16, 16, 16, 0, None) == UNSUPPORTED
    assert lib.trtv_msa_proxy_score(r, 16, 16, 16, 16, 16, None) == UNSUPPORTED
    assert lib.trtv_msa_sparse_attn(r, 16, 16, 16, 16, 16, 2, 16, 0, 256, 1 << 30, None) == UNSUPPORTED
    assert lib.trtv_msa_select(r, 16, 16, 16, 16, 2, 16, 16, 256, 1 << 30, None) == UNSUPPORTED
    assert lib.trtv_msa_verify(r, 16, 16, 16, 16, 2, 16, 16, 16, 0, 256, 1 << 30, None) == UNSUPPORTED
    assert lib.trtv_stage_kv(r, 16, 16, 16, 16, 16, None) == UNSUPPORTED
    assert lib.trtv_verify_dense_flat(r, 16, 16, 16, 16, 16, 0, 256, 1 << 30, None) == UNSUPPORTED
    assert lib.trtv_draft_attn_p32(r, 16, 16, 16, 16, 16, 16, 0, 256, 1 << 30, None) == UNSUPPORTED
    assert lib.trtv_workspace_bytes(r, 2) == 0 and lib.trtv_workspace_bytes_flat(r) == 0


@pytest.mark.parametrize("over,status", [
    (dict(batch=0), INVALID), (dict(qo_len=0), INVALID), (dict(qo_len=33), UNSUPPORTED), (dict(batch=2049), UNSUPPORTED),
    (dict(head_dim=96), UNSUPPORTED), (dict(slot_stride=1), INVALID), (dict(k_scale=0.0), INVALID),
    (dict(num_q_heads=129, num_kv_heads=1), UNSUPPORTED), (dict(num_slots=1 << 20, slot_stride=8), UNSUPPORTED),
    (dict(v_scale=float("nan")), INVALID), (dict(num_ctas=1025), INVALID)])
def test_ladder_geometry(lib, over, status):
    r = ctypes.byref(geom(**over))
    assert lib.trtv_verify_dense(r, 16, 16, 16, 16, 16, 0, 256, 1 << 40, None) == status
    assert lib.trtv_workspace_bytes(r, 0) == 0


@pytest.mark.parametrize("d", [64, 128])
def test_ladder_arguments(lib, d):
    r = ctypes.byref(geom(head_dim=d))
    need = lib.trtv_workspace_bytes(r, 0)
    assert need == lib.trtv_workspace_bytes_rows(r) > 0
    good = [r, 16, 16, 16, 16, 16, 0, 256, need, None]
    for i, bad, st in ((1, 0, INVALID), (2, 0, INVALID), (3, 0, INVALID), (4, 0, INVALID), (5, 0, INVALID), (1, 24, INVALID),
                       (2, 24, INVALID), (5, 8, INVALID), (6, 1, INVALID), (6, 3, INVALID), (7, 128, WORKSPACE),
                       (7, 0, WORKSPACE), (8, need - 1, WORKSPACE)):
        a = list(good)
        a[i] = bad
        assert lib.trtv_verify_dense(*a) == st, (i, bad)
    for batch in (1, 2048):
        for qo in (1, 32):
            assert lib.trtv_workspace_bytes(ctypes.byref(geom(head_dim=d, batch=batch, qo_len=qo)), 0) > 0


def test_stage_divides_by_no_zero(lib):
    n = T.NormRope(q=32, k=16, v=16, q_stride=4096, k_stride=4096, v_stride=4096)
    for v in (0.0, -0.0):
        r = ctypes.byref(geom(v_scale=v))
        assert lib.trtv_norm_rope_stage(r, ctypes.byref(n), 16, 80, 16, 16, 16, 16, None) == INVALID


@pytest.mark.parametrize("kv", [0, 1, 3])
def test_read_arguments(lib, kv):
    good = [ctypes.byref(geom(kv_dtype=kv)), 16, 16, 16, 16, 8, 16, 16, None]
    for i, bad in ((1, 0), (1, 8), (2, 0), (2, 18), (3, 0), (3, 18), (4, 18), (5, -1), (6, 24), (7, 24)):
        a = list(good)
        a[i] = bad
        assert lib.trtv_read_kv(*a) == INVALID, (i, bad)
    a = list(good)
    a[6] = a[7] = 0
    assert lib.trtv_read_kv(*a) == INVALID
    a = list(good)
    a[4], a[5] = None, 7          # equal rows per request need batch * qo_len of them
    assert lib.trtv_read_kv(*a) == INVALID
    a[4], a[5] = 16, 0            # no rows: nothing to do
    assert lib.trtv_read_kv(*a) == 0
    assert lib.trtv_read_kv(None, *good[1:]) == INVALID
    a = list(good)
    a[0] = ctypes.byref(geom(kv_dtype=2))
    assert lib.trtv_read_kv(*a) == INVALID


@pytest.mark.parametrize("kv", [0, 1, 3])
def test_fork_arguments(lib, kv):
    r = ctypes.byref(geom(kv_dtype=kv))
    need = lib.trtv_workspace_bytes_pages(r, 3)
    assert need > 0
    #       geom pool buf ref table lens pages parent tokens n new_ref new_table new_lens new_pages ws bytes stream
    good = [r, 16, 2, 32, 48, 64, 80, 96, 112, 3, 128, 144, 160, 176, 256, need, None]
    for i, bad, st in ((1, 0, INVALID), (1, 8, INVALID), (2, 0, INVALID), (2, 3, INVALID), (3, 0, INVALID), (3, 34, INVALID),
                       (4, 0, INVALID), (4, 50, INVALID), (5, 0, INVALID), (5, 66, INVALID), (6, 82, INVALID), (7, 0, INVALID),
                       (7, 98, INVALID), (8, 114, INVALID), (9, 0, INVALID), (9, -1, INVALID), (9, 2049, UNSUPPORTED),
                       (10, 0, INVALID), (10, 130, INVALID), (11, 0, INVALID), (11, 146, INVALID), (11, 48, INVALID),
                       (12, 0, INVALID), (12, 162, INVALID), (12, 64, INVALID), (13, 178, INVALID), (13, 80, INVALID),
                       (14, 0, WORKSPACE), (14, 128, WORKSPACE), (15, need - 1, WORKSPACE)):
        a = list(good)
        a[i] = bad
        assert lib.trtv_pages_fork(*a) == st, (i, bad)
    assert lib.trtv_pages_fork(None, *good[1:]) == INVALID


def test_compact_arguments(lib):
    r = ctypes.byref(geom())
    need = lib.trtv_workspace_bytes_pages(r, 0)
    #       geom pool buf ref table pages map used new_ref new_table ws bytes stream
    good = [r, 16, 2, 32, 48, 64, 80, 96, 112, 128, 256, need, None]
    for i, bad, st in ((1, 0, INVALID), (1, 8, INVALID), (2, 0, INVALID), (2, 3, INVALID), (3, 0, INVALID), (3, 34, INVALID),
                       (4, 0, INVALID), (4, 50, INVALID), (5, 0, INVALID), (5, 66, INVALID), (6, 0, INVALID), (6, 82, INVALID),
                       (7, 0, INVALID), (7, 98, INVALID), (8, 0, INVALID), (8, 114, INVALID), (9, 0, INVALID), (9, 130, INVALID),
                       (10, 0, WORKSPACE), (10, 128, WORKSPACE), (11, need - 1, WORKSPACE)):
        a = list(good)
        a[i] = bad
        assert lib.trtv_pages_compact(*a) == st, (i, bad)
    assert lib.trtv_pages_compact(None, *good[1:]) == INVALID


def test_page_workspaces(lib):
    assert lib.trtv_workspace_bytes_pages(None, 1) == 0
    r = ctypes.byref(geom())
    assert lib.trtv_workspace_bytes_pages(r, -1) == 0 and lib.trtv_workspace_bytes_pages(r, 2049) == 0
    assert lib.trtv_workspace_bytes_pages(ctypes.byref(geom(batch=2049)), 1) == 0
    big = geom(num_slots=(1 << 23) - 1, num_kv_heads=1, num_q_heads=4)
    # two words a slot (lists in whole chunks of 1024), and what the requests need
    assert 2 * 4 * big.num_slots < lib.trtv_workspace_bytes_pages(ctypes.byref(big), 2048) < 2 * 4 * big.num_slots + (1 << 17)
