"""Forking and compacting pages against the same steps done one page after the other on the host (everything is
compared bit for bit, the whole pool included)."""
import random

import pytest
import torch

import speculative_decode_verify_kv_gb300 as T
from pages_common import Pages, check_compact, check_fork, compact, fork, ints, pages_for, walk_fork

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decode_verify_kv_gb300 import _build
    _build.build()
    T.load()
    T.trtv_get_device_error()


KINDS = [("bf16", 2, 128, 2, 2), ("bf16", 1, 64, 3, 2), ("fp8", 3, 128, 8, 8), ("fp4", 2, 128, 2, 2), ("fp4", 3, 64, 5, 4),
         ("fp4", 1, 64, 2, 1)]


@pytest.mark.parametrize("kv,hk,d,stride,buffers", KINDS)
@pytest.mark.parametrize("in_place", [False, True])
def test_fork_kinds(kv, hk, d, stride, buffers, in_place):
    p = Pages(60, 9, hk, d, kv, stride, buffers, seed=d)
    for length in (0, 1, 127, 128, 129, 300, 512, 1000):
        p.add(length, spare=length % 2)
    check_fork(p, [7, 7, 5, 4, 4, 4, 2, 0, -1, 6, 3, 1], [1, 0, 64, 128, 3, 0, 1, 5, 200, 0, 0, 127], in_place=in_place, junk=-3)


@pytest.mark.parametrize("length", [0, 1, 31, 32, 33, 95, 96, 127, 128, 129, 255, 256])
def test_fork_lengths(length):
    p = Pages(40, 5, 2, 64, "fp4", 2, 2, seed=length)
    p.add(length)
    p.add(300)
    check_fork(p, [0, 0, 0, 1], [0, 1, 130, 0])


def test_only_reordered_and_ended():
    p = Pages(40, 4)
    for length in (100, 200, 300, 5):
        p.add(length, spare=1)
    check_fork(p, [3, 1], None, num=True, new_num=False)      # 0 and 2 end, spare pages are given back
    check_fork(p, [1, 0], None, num=False)                     # held: the pages of the lengths
    check_fork(p, [-1], [0])                                   # all end
    assert p.ref == [0] * 40


def test_shared_pages_and_other_holders():
    p = Pages(60, 8, seed=2)
    a = p.add(500)
    for _ in range(3):
        p.add(640, share=a)
    p.ref[p.rows[0][3]] += 1       # somebody else holds the page that request 0 would write to
    p.ref[p.rows[2][0]] += 2
    p.ref[7 if p.ref[7] == 0 else p.ref.index(0)] = 5           # a slot that only others hold
    check_fork(p, [0, 0, 2, 3, 3], [1, 1, 1, 1, 1])
    check_fork(p, [4, 0, 1, 1], [1, 100, 1, 1])


@pytest.mark.parametrize("slots", [1023, 1024, 1025, 2048, 5000])
def test_slots_over_several_chunks(slots):
    p = Pages(slots, 40, 1, 64, "fp4", 2, 2, seed=slots)
    while sum(x == 0 for x in p.ref) > slots // 3:
        p.add(p.r.randint(0, 39 * 128))
    n = len(p.rows)
    parent = [p.r.randrange(-1, n) for _ in range(n)]
    check_fork(p, parent, [p.r.randint(0, 60) if q < 0 or p.lens[q] < 39 * 128 else 0 for q in parent])
    check_compact(p)
    check_fork(p, list(range(n)), [1] * n)


def test_slots_over_more_chunks_than_threads():
    """300 chunks of slots, a third of them held by others."""
    p = Pages(300 * 1024 + 5, 5, 1, 64, "fp4", 2, 2, seed=3)
    for i in random.Random(3).sample(range(p.slots), p.slots // 3):
        p.ref[i] = 1
    for length in (130, 500, 1, 640):
        p.add(length)
    check_fork(p, [1, 1, 0, 3, 3, 3, 2, -1], [1, 128, 0, 0, 0, 0, 400, 513], in_place=True)
    check_compact(p)


def test_the_last_free_slot():
    p = Pages(12, 4, 1, 64, seed=1)
    p.add(300)
    p.add(128)
    p.add(500)                    # 8 slots
    check_fork(p, [0, 0, 1, 2, 2], [100, 1, 128, 0, 1])   # four fresh ones
    assert 0 not in p.ref


@pytest.mark.parametrize("seed", range(4))
def test_many_steps(seed):
    """Requests fork, end, start and grow for many steps, and the pool is compacted in between."""
    r = random.Random(seed)
    p = Pages(700, 10, 1, 64, r.choice(["bf16", "fp4"]), 2, 2, seed=seed)
    for _ in range(12):
        p.add(r.randint(0, 900), spare=r.randint(0, 1))
    for step in range(25):
        n = r.randint(1, 40)
        parent = [r.choice([-1] + list(range(len(p.rows)))) for _ in range(n)]
        grow = [r.choice([0, 1, 1, 17, 200]) for _ in parent]
        grow = [min(g, 1280 - (p.lens[q] if q >= 0 else 0)) for q, g in zip(parent, grow)]
        if walk_fork(p.ref, p.rows, p.lens, p.num, parent, grow) is None:
            parent, grow = parent[:2], grow[:2]
        check_fork(p, parent, grow, in_place=step % 2 == 0)
        # a rolled back draft: the length shrinks, the pages are still held
        for b in range(len(p.lens)):
            if r.random() < 0.3:
                p.lens[b] = r.randint(0, p.lens[b])
        if step % 5 == 4:
            check_compact(p, in_place=step % 2 == 0)


@pytest.mark.parametrize("batch", [1, 2048])
def test_largest_batches(batch):
    p = Pages(9000, 2, 1, 64, "fp4", 2, 2, seed=batch)
    for b in range(batch):
        p.add(b % 200 + 1, scattered=False)
    check_fork(p, [(i * 7) % batch for i in range(2048)], [i % 3 for i in range(2048)])
    check_compact(p)


def untouched(p, parent, grow, err, **kw):
    before = p.bytes.clone()
    ref, table, lens, pages = fork(p, parent, grow, **kw)
    torch.cuda.synchronize()
    assert T.trtv_get_device_error() == err
    assert ref.tolist() == p.ref
    assert (table == -7).all() and (lens == -7).all() and (pages == -7).all()
    assert torch.equal(p.bytes, before)


@pytest.mark.parametrize("in_place", [False, True])
def test_fork_errors_change_nothing(in_place):
    def make():
        p = Pages(14, 4, seed=3)
        for length in (300, 128, 500):
            p.add(length)
        return p

    kw = dict(in_place=in_place)
    p = make()
    untouched(p, [0, 1, 2, 0, 0, 0, 0, 0, 0], [1] * 9, T.DEVERR_SLOTS, **kw)
    untouched(p, [-1, -1], [512, 400], T.DEVERR_SLOTS, **kw)
    untouched(p, [0, 3], [0, 0], T.DEVERR_PARENT, **kw)
    untouched(p, [0, -2], [0, 0], T.DEVERR_PARENT, **kw)
    untouched(p, [0], [-1], T.DEVERR_KV_LEN, **kw)
    untouched(p, [2], [13], T.DEVERR_KV_LEN, **kw)
    untouched(p, [0], [2 ** 31 - 1], T.DEVERR_KV_LEN, **kw)
    for field, b, x in (("lens", 1, -1), ("lens", 1, 513), ("num", 0, 2), ("num", 0, 5), ("num", 0, -1)):
        p = make()
        getattr(p, field)[b] = x
        untouched(p, [2], [0], T.DEVERR_KV_LEN, **kw)     # of a request that is nobody's parent, too
    for x in (-1, 14, 2 ** 30):
        p = make()
        p.rows[0][1] = x
        untouched(p, [2], [0], T.DEVERR_PAGE_ID, **kw)
    p = make()
    p.ref[p.rows[0][1]] = 0
    untouched(p, [2], [0], T.DEVERR_REFS, **kw)
    p = make()
    p.ref[p.ref.index(0)] = -1
    untouched(p, [2], [0], T.DEVERR_REFS, **kw)


@pytest.mark.parametrize("kv,hk,d,stride,buffers", KINDS)
@pytest.mark.parametrize("in_place", [False, True])
def test_compact_kinds(kv, hk, d, stride, buffers, in_place):
    p = Pages(90, 9, hk, d, kv, stride, buffers, seed=d + 1)
    for length in (0, 1, 300, 1000, 512, 128):
        p.add(length, spare=length % 2)
    p.add(700, share=3)
    p.ref[p.ref.index(0)] = 3       # held by others
    check_compact(p, in_place=in_place)
    check_compact(p, in_place=in_place)   # nothing moves any more


def test_compact_full_and_empty_pools():
    p = Pages(16, 4, 1, 64)
    p.add(0)
    check_compact_empty(p)
    for _ in range(4):
        p.add(512)
    assert 0 not in p.ref
    check_compact(p)


def check_compact_empty(p):
    ref, table, slot_map, used = compact(p)
    torch.cuda.synchronize()
    assert T.trtv_get_device_error() == 0
    assert used.tolist() == [0] and slot_map.tolist() == [-1] * p.slots and ref.tolist() == [0] * p.slots
    assert (table == 0).all()


def test_compact_errors_change_nothing():
    for what, err in (("num", T.DEVERR_KV_LEN), ("id", T.DEVERR_PAGE_ID), ("free", T.DEVERR_REFS), ("negative", T.DEVERR_REFS)):
        p = Pages(40, 4, 1, 64, seed=5)
        for length in (300, 128, 500):
            p.add(length)
        if what == "num":
            p.num[1] = 5
        elif what == "id":
            p.rows[2][1] = 40
        elif what == "free":
            p.ref[p.rows[2][1]] = 0
        else:
            p.ref[p.ref.index(0)] = -2
        before = p.bytes.clone()
        ref, table, slot_map, used = compact(p)
        torch.cuda.synchronize()
        assert T.trtv_get_device_error() == err
        assert ref.tolist() == p.ref
        assert (table == -7).all() and (slot_map == -7).all() and (used == -7).all()
        assert torch.equal(p.bytes, before)


def test_captured_and_replayed():
    """A graph of fork and compact on a device state that changes between replays."""
    p = Pages(50, 5, 2, 64, "fp4", 2, 2, seed=11)
    for length in (100, 300, 17, 500):
        p.add(length)
    geom = p.geom(4)
    n1, n2 = T.trtv_workspace_bytes_pages(geom, 4), T.trtv_workspace_bytes_pages(geom, 0)
    ws = torch.full((n1 + n2,), 255, dtype=torch.uint8, device="cuda")
    assert n1 % 256 == 0
    ref, table, lens, num = ints(p.ref), p.table(), ints(p.lens), ints(p.num)
    parent, grow = ints([0, 0, 1, 3]), ints([1, 1, 1, 1])
    t2, l2, n2p = torch.zeros_like(table), torch.zeros_like(lens), torch.zeros_like(num)
    slot_map, used = torch.zeros_like(ref), ints([0])

    def step():
        T.trtv_pages_fork(geom, p.pool(), 2, ref, table, lens, num, parent, grow, ref, t2, l2, n2p, ws, n1)
        T.trtv_pages_compact(geom, p.pool(), 2, ref, t2, n2p, slot_map, used, ref, table, ws[n1:], n2)
        lens.copy_(l2)
        num.copy_(n2p)

    saved = [x.clone() for x in (p.bytes, ref, table, lens, num)]
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for x, y in zip((p.bytes, ref, table, lens, num), saved):
        x.copy_(y)
    for who in ([0, 0, 1, 3], [3, 2, 1, 0], [1, 1, 1, 1], [0, 1, 2, -1]):
        parent.copy_(ints(who))
        want_ref, rows, want_lens, copies = walk_fork(p.ref, p.rows, p.lens, p.num, who, [1] * 4)
        keep = p.copied(copies)
        graph.replay()
        torch.cuda.synchronize()
        assert T.trtv_get_device_error() == 0
        from pages_common import walk_compact
        to, total = walk_compact(want_ref)
        x = keep.view(p.slots, p.stride, -1)
        src = [i for i, t in enumerate(to) if t >= 0 and t != i]
        if src:
            x[torch.tensor([to[i] for i in src]).cuda(), :2] = x[torch.tensor(src).cuda(), :2]
        p.ref = [0] * p.slots
        for i, t in enumerate(to):
            if t >= 0:
                p.ref[t] = want_ref[i]
        p.rows = [[to[s] for s in r] for r in rows]
        p.lens, p.num = want_lens, [len(r) for r in rows]
        assert ref.tolist() == p.ref and lens.tolist() == p.lens and used.tolist() == [total]
        assert table.tolist() == [r + [0] * (p.mp - len(r)) for r in p.rows]
        assert torch.equal(p.bytes, keep)


def test_on_another_stream():
    p = Pages(60, 9, seed=4)
    for length in (100, 900, 300):
        p.add(length)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        check_fork(p, [1, 1, 0, 2], [1, 2, 3, 4])
        check_compact(p)


def test_attention_of_forked_requests():
    """Over an E2M1 cache: samples forked from one prompt attend what the prompt's request would, then grow apart, and
    moving their pages changes no bit."""
    from fp4_common import Fp4Rows, check
    q = Fp4Rows([1, 1], [300, 150], 8, 2, 128, uniform=True, seed=6, extra_pages=1)
    slots, mp = 40, q.mp
    pool = torch.full((slots * 2, 4, 2, 18 * 128), 255, dtype=torch.uint8, device="cuda")
    pool[:q.pool.shape[0]] = q.pool
    ref = torch.zeros(slots, dtype=torch.int32, device="cuda")
    num = ints([pages_for(x) for x in q.kv])
    for b in range(2):
        ref[q.table[b, :int(num[b])].long()] += 1
    geom = T.Geom(batch=2, qo_len=1, num_q_heads=8, num_kv_heads=2, head_dim=128, max_pages_per_req=mp, num_slots=slots,
                  slot_stride=2, kv_dtype=T.TRTV_FP4_E2M1, sm_scale=q.geom.sm_scale, k_scale=q.k_scale, v_scale=q.v_scale,
                  num_ctas=0)
    parent = ints([0, 1, 0, 0, 1])
    nb = T.trtv_workspace_bytes_pages(geom, 5)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    table, lens, pages = torch.empty(5, mp, dtype=torch.int32, device="cuda"), ints([0] * 5), ints([0] * 5)
    T.trtv_pages_fork(geom, pool, 2, ref, q.table, q.kv_lens, num, parent, ints([1] * 5), ref, table, lens, pages, ws, nb)
    torch.cuda.synchronize()
    assert T.trtv_get_device_error() == 0
    assert lens.tolist() == [302, 152, 302, 302, 152]
    # every sample stages its own next token, then attends
    p = Fp4Rows([1] * 5, [301, 151, 301, 301, 151], 8, 2, 128, uniform=True, seed=7)
    p.table, p.mp, p.slots, p.pool, p.kv_lens = table, mp, slots, pool, lens
    g5 = T.Geom.from_buffer_copy(geom)
    g5.batch = 5
    p.geom = g5
    kv = torch.randn(5, 2, 128, device="cuda").to(torch.bfloat16)
    q_out = torch.empty_like(p.q)
    T.trtv_norm_rope_stage(g5, p.q, kv, kv + 1, None, None, 1e-6, None, 0, False, None, None, q_out, pool, table, lens)
    out = p.dense()
    check(p, out)
    slot_map, used = torch.empty_like(ref), ints([0])
    nb = T.trtv_workspace_bytes_pages(g5, 0)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    T.trtv_pages_compact(g5, pool, 2, ref, table, pages, slot_map, used, ref, table, ws, nb)
    again = p.dense()
    torch.cuda.synchronize()
    assert T.trtv_get_device_error() == 0
    assert torch.equal(out, again)
    assert int(used) == int((ref > 0).sum()) == int(table.unique().numel())
