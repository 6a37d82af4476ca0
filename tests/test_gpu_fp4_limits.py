"""E2M1 caches at the edges: bounded waits, the largest batches, pools past 32 bits, shifted addresses, calls without
tokens, rows of infinities and NaN, other kernels on the same SMs."""
import time

import pytest
import torch

import speculative_decode_verify_kv_gb300 as T
from fp4_common import Fp4Rows, check
from pages_common import ints
from rows_common import pack

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


@pytest.mark.parametrize("pages", [0, 1, 2, 9])
@pytest.mark.parametrize("kind,hq,hk,d,n", [("ladder", 32, 4, 128, 1), ("ladder", 32, 4, 128, 2), ("ladder", 32, 4, 128, 4),
                                            ("ladder", 8, 2, 64, 1), ("ladder", 32, 4, 128, 16), ("prompt", 32, 4, 128, 300),
                                            ("prompt", 8, 2, 64, 300), ("tree", 32, 4, 128, 16), ("tree", 8, 2, 64, 8)])
def test_withheld_pages_end_the_call(kind, hq, hk, d, n, pages):
    p = Fp4Rows([n] * 3, [2000, 3000, 100], hq, hk, d, uniform=True, num_ctas=4)
    m = p.tree_masks()
    go = {"ladder": p.dense, "prompt": p.prompt, "tree": lambda: p.tree(m)}[kind]
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


@pytest.mark.parametrize("batch", [1500, 2048])
@pytest.mark.parametrize("n,hq,d", [(1, 8, 128), (2, 8, 128), (4, 8, 128), (1, 8, 64), (4, 8, 64)])
def test_largest_batches(batch, n, hq, d):
    """A long scan leaves less shared memory for pages."""
    p = Fp4Rows([n] * batch, [(i * 37) % 170 if i % 97 else 1200 for i in range(batch)], hq, 1, d, uniform=True, seed=batch + n)
    v = p.values()
    p.values = lambda pool=None: v
    check(p, p.dense())


@pytest.mark.parametrize("kind,d", [("prompt", 128), ("prompt", 64), ("tree", 128), ("tree", 64)])
def test_largest_batches_of_tiles(kind, d):
    """The same beside 256-row items (some requests have many tokens) and 128-row items."""
    most = 300 if kind == "prompt" else 20
    new = [most if i % 211 == 0 else i % 3 for i in range(2048)]
    p = Fp4Rows(new, [(i * 37) % 170 if i % 97 else 1200 for i in range(2048)], 4, 1, d, pad=1, seed=d)
    v = p.values()
    p.values = lambda pool=None: v
    if kind == "prompt":
        check(p, p.prompt())
    else:
        m = p.tree_masks()
        check(p, p.tree(m), m)


@pytest.mark.parametrize("hq,n", [(32, 1), (32, 4), (32, 20)])
def test_slots_past_four_gigabytes(hq, n):
    """The same pages at the start of a small pool and at the end of one of 5.9 GB."""
    hk, d, far = 8, 128, 40000
    outs = []
    g = torch.Generator(device="cuda").manual_seed(n)
    new = [n, n]
    kv = [150 + n, 300 + n]
    x = torch.randn(sum(kv), (hq + 2 * hk) * d, generator=g, device="cuda").to(torch.bfloat16)
    q, k, v = x[:, :hq * d].view(-1, hq, d), x[:, hq * d:(hq + hk) * d].view(-1, hk, d), x[:, (hq + hk) * d:].view(-1, hk, d)
    mask = torch.tril(torch.ones(n, n, dtype=torch.bool, device="cuda")).repeat(2, 1)
    mask[:, 0] = True
    for slots in (8, far):
        pool = torch.empty(slots * 2, 4, hk, 18 * d, dtype=torch.uint8, device="cuda")
        pool[-16:] = 255
        geom = T.Geom(batch=2, qo_len=max(kv), num_q_heads=hq, num_kv_heads=hk, head_dim=d, max_pages_per_req=3, num_slots=slots,
                      slot_stride=2, kv_dtype=T.TRTV_FP4_E2M1, sm_scale=0.1, k_scale=0.01, v_scale=0.01, num_ctas=0)
        table = ints([[7, 2, 0], [1, 6, 4]]) + (slots - 8)
        lens, indptr = ints(kv), ints([0, kv[0], sum(kv)])
        q_out = torch.empty_like(q)
        T.trtv_norm_rope_stage(geom, q, k, v, None, None, 1e-6, None, 0, False, None, indptr, q_out, pool, table, lens)
        back = [torch.empty(sum(kv), hk, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        T.trtv_read_kv(geom, pool, table, lens, indptr, *back)
        rows = torch.cat([q_out[kv[0] - n:kv[0]], q_out[-n:]])
        geom.qo_len = n
        nb = T.trtv_workspace_bytes(geom)
        ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
        out = [torch.empty_like(rows) for _ in range(3)]
        T.trtv_verify_dense(geom, rows, pool, table, lens, out[0], T.TRTV_BF16, ws, nb)
        T.trtv_prompt_attn(geom, rows, pool, table, lens, None, out[1], T.TRTV_BF16, ws, nb)
        T.trtv_verify_tree(geom, rows, pool, table, lens, None, pack(mask, n), out[2], T.TRTV_BF16, ws, nb)
        path = ints([[0, n - 1] if n > 1 else [0, -1]] * 2)
        T.trtv_tree_commit(geom, pool, table, lens, None, path, ints([2 if n > 1 else 1] * 2), lens)
        torch.cuda.synchronize()
        assert T.trtv_get_device_error() == 0
        outs.append((pool[-16:].clone(), q_out, *back, *out, lens))
        if slots == far:   # a copy on write into the first slot, and every page moved to the front
            want = pool[-16:].clone()
            ref = torch.zeros(slots, dtype=torch.int32, device="cuda")
            ref[table.view(-1).long()] = 1
            nb = T.trtv_workspace_bytes_pages(geom, 3)
            ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
            # (request 1's last page is begun)
            held = ints([(int(y) + 127) // 128 for y in lens])
            t2 = torch.empty(3, 3, dtype=torch.int32, device="cuda")
            l2, n2 = ints([0] * 3), ints([0] * 3)
            T.trtv_pages_fork(geom, pool, 2, ref, table, lens, held, ints([0, 1, 1]), ints([0, 0, 1]), ref, t2, l2, n2, ws, nb)
            torch.cuda.synchronize()
            assert T.trtv_get_device_error() == 0
            assert t2[2, 2] == 0 and (t2[0] == table[0])[:2].all() and (t2[1] == table[1]).all()
            part = int(lens[1]) % 128
            a = pool[:2].view(2, 4, hk, -1)[..., :16 * d].unflatten(-1, (32, -1)).transpose(2, 3).flatten(1, 2)[:, :part]
            b = want[8:10].view(2, 4, hk, -1)[..., :16 * d].unflatten(-1, (32, -1)).transpose(2, 3).flatten(1, 2)[:, :part]
            assert torch.equal(a, b)
            slot_map, used = torch.empty_like(ref), ints([0])
            g3 = T.Geom.from_buffer_copy(geom)
            g3.batch = 3
            T.trtv_pages_compact(g3, pool, 2, ref, t2, n2, slot_map, used, ref, t2, ws, nb)
            torch.cuda.synchronize()
            assert T.trtv_get_device_error() == 0
            assert int(used) == int((ref > 0).sum()) == 7
            for old, new_at in ((7, t2[0, 0]), (2, t2[0, 1]), (1, t2[1, 0]), (6, t2[1, 1]), (4, t2[1, 2])):
                at = int(new_at)
                assert at < 7 and torch.equal(pool[2 * at:2 * at + 2], want[2 * old:2 * old + 2])
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def shifted(x, by):
    """The same values `by` bytes into an allocation."""
    raw = torch.empty(x.numel() * x.element_size() + by, dtype=torch.uint8, device=x.device)
    y = raw[by:].view(x.dtype).view(x.shape)
    y.copy_(x)
    return y


@pytest.mark.parametrize("n,hq,hk,d", [(1, 32, 4, 128), (4, 32, 4, 128), (16, 32, 4, 128), (200, 8, 2, 64)])
def test_least_alignment(n, hq, hk, d):
    p = Fp4Rows([n] * 3, [333, 90, 1000], hq, hk, d, uniform=True)
    m = p.tree_masks()
    a = p.dense() if n <= 32 else p.prompt()
    b = p.tree(m) if n <= 128 else None
    read = p.read()
    p.pool, p.q = shifted(p.pool, 16), shifted(p.q, 16)
    p.table, p.kv_lens = shifted(p.table, 4), shifted(p.kv_lens, 4)
    assert p.pool.data_ptr() % 32 == 16 and p.q.data_ptr() % 32 == 16
    assert torch.equal(a, p.dense() if n <= 32 else p.prompt())
    assert b is None or torch.equal(b, p.tree(m))
    assert all(torch.equal(x, y) for x, y in zip(read, p.read()))
    assert T.trtv_get_device_error() == 0


def test_calls_without_tokens():
    p = Fp4Rows([0, 0], [100, 0], 8, 2, 128)
    before = p.pool.clone()
    none = lambda h: torch.empty(0, h, 128, dtype=torch.bfloat16, device="cuda")   # noqa: E731
    q_out, out, k, v = none(8), none(8), none(2), none(2)
    T.trtv_norm_rope_stage(p.geom, none(8), none(2), none(2), None, None, 1e-6, None, 0, False, None, p.indptr, q_out, p.pool, p.table,
                           p.kv_lens)
    T.trtv_read_kv(p.geom, p.pool, p.table, p.kv_lens, p.indptr, k, v)
    ws, nb = p.workspace()
    T.trtv_prompt_attn(p.geom, none(8), p.pool, p.table, p.kv_lens, p.indptr, out, T.TRTV_BF16, ws, nb)
    torch.cuda.synchronize()
    assert T.trtv_get_device_error() == 0 and torch.equal(p.pool, before)


@pytest.mark.parametrize("n,hq,hk,d", [(1, 32, 4, 128), (2, 32, 4, 128), (4, 32, 4, 128), (16, 32, 4, 128), (4, 8, 2, 64)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_row_of_nan_or_infinity_is_its_own(n, hq, hk, d, bad):
    """Other rows of the same products keep every bit."""
    p = Fp4Rows([n] * 3, [700, 90, 1000], hq, hk, d, uniform=True)
    clean = p.dense()
    row = (p.rows - 1, 3)
    p.q[row][5] = bad
    out = p.dense()
    torch.cuda.synchronize()
    assert T.trtv_get_device_error() == 0
    assert torch.isnan(out[row]).all()
    out[row] = clean[row]
    assert torch.equal(out, clean)


@pytest.mark.parametrize("n,hq,hk,d", [(1, 32, 4, 128), (4, 32, 4, 128), (16, 32, 4, 128), (1, 8, 2, 64), (4, 8, 2, 64)])
def test_tiny_and_large_queries(n, hq, hk, d):
    """Rows of 2^-30: scores of nearly zero.  Rows of 2^30, whose logits' rounding is above their differences, are
    reported; other rows keep every bit."""
    p = Fp4Rows([n] * 3, [700, 90, 1000], hq, hk, d, uniform=True)
    clean = p.dense(T.TRTV_F32)
    p.q[:, 0::3] *= 2.0 ** -30
    out = p.dense(T.TRTV_F32)
    check(p, out)
    p.q[:, 0::3] *= 2.0 ** 60
    out = p.dense(T.TRTV_F32)
    torch.cuda.synchronize()
    assert T.trtv_get_device_error() == T.DEVERR_LOGITS
    for h in range(hq):
        assert h % 3 == 0 or torch.equal(out[:, h], clean[:, h])


def test_beside_other_kernels():
    from rows_common import Rows
    few = Fp4Rows([1] * 6, [3000, 5, 700, 128, 1000, 64], 32, 4, 128, uniform=True, seed=1)
    some = Fp4Rows([4] * 4, [3000, 5, 700, 128], 32, 4, 128, uniform=True, seed=2)
    tree = Fp4Rows([16, 8], [2000, 100], 32, 4, 128, seed=3)
    prompt = Fp4Rows([300, 30], [0, 900], 8, 2, 64, seed=4)
    full = Rows([200, 30], [0, 900], 8, 2, 64, seed=1)
    m = tree.tree_masks()
    x = torch.randn(1024, 1024, device="cuda").bfloat16()
    calls = dict(few=few.dense, some=some.dense, tree=lambda: tree.tree(m), prompt=prompt.prompt, full=full.prompt, product=lambda: x @ x)
    want = {k: f() for k, f in calls.items()}
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    orders = (["product", "few", "tree", "product", "prompt", "some"],
              ["full", "prompt", "product", "few", "product", "tree", "some"])
    for _ in range(5):
        got = []
        for s, order in zip(streams, orders):
            with torch.cuda.stream(s):
                got += [(k, calls[k]()) for k in order]
        torch.cuda.synchronize()
        for k, out in got:
            assert torch.equal(out, want[k]), k
    assert T.trtv_get_device_error() == 0
