"""Norm + rotation + staging, and tree commits, against 64-bit references.

Tolerances: a value is rounded once, by half a step (bf16: 2^-8 of its size;
E4M3: 2^-4, or 2^-10 absolute below the normals), after a chain of binary32
operations whose relative errors (sum of squares over 128 terms, rsqrt,
products, a rotation's difference of two products, the table's own rounding
being an input) stay under 2^-17 of the largest magnitude involved: the
rotation's two terms, at most sqrt(2) times the pair's length.
"""
import pytest
import torch

import speculative_decode_verify_kv_gb300 as T
from rows_common import Rows, norm_rope, rope_table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decode_verify_kv_gb300 import _build
    _build.build()
    T.load()
    T.trtv_get_device_error()


def inputs(p, packed=True, seed=5):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(p.rows, (p.hq + 2 * p.hk) * p.d, generator=g).to(torch.bfloat16).to(p.dev)
    a, b = p.hq * p.d, (p.hq + p.hk) * p.d
    q, k, v = (x.view(p.rows, -1, p.d) for x in (qkv[:, :a], qkv[:, a:b], qkv[:, b:]))
    if not packed:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    w = [(1 + 0.3 * torch.randn(p.d, generator=g)).to(torch.bfloat16).to(p.dev) for _ in range(2)]
    return q, k, v, w


def place(p):
    """(request, cache position) of every token row."""
    req, pos = [], []
    for b in range(p.B):
        req += [b] * p.new[b]
        pos += [p.ctx[b] + t for t in range(p.new[b])]
    return torch.tensor(req, device=p.dev), torch.tensor(pos, device=p.dev)


def check_stage(p, rot, interleaved, norm=True, positions=None, packed=True, eps=1e-6, in_place=False):
    q, k, v, w = inputs(p, packed)
    qw, kw = w if norm else (None, None)
    table = rope_table(max(p.kv + [1]) + 7, rot).to(p.dev) if rot else None
    req, cell = place(p)
    pos = cell if positions is None else positions.to(p.dev)
    before = p.pool.clone()
    q_ref = norm_rope(q[:p.toks], qw, eps, None if not rot else table[pos[:p.toks].long()], rot, interleaved)
    k_ref = norm_rope(k[:p.toks], kw, eps, None if not rot else table[pos[:p.toks].long()], rot, interleaved)
    q_out = q if in_place else torch.full((p.rows, p.hq, p.d), 3.0, dtype=torch.bfloat16, device=p.dev)
    tail = q_out[p.toks:].clone()
    T.trtv_norm_rope_stage(p.geom, q, k, v, qw, kw, eps, table, rot, interleaved,
                           None if positions is None else pos.int(), p.indptr, q_out, p.pool, p.table, p.kv_lens)
    torch.cuda.synchronize()
    assert T.trtv_get_device_error() == 0

    def near(got, ref, half, floor=0.0):
        size = ref.abs()
        slack = ref.abs().amax(-1, keepdim=True) * 2.0 ** -15 if ref.numel() else 0
        assert ((got.double() - ref).abs() <= size * half * (1 + 2.0 ** -10) + slack + floor).all()

    near(q_out[:p.toks], q_ref, 2.0 ** -9 * 2)
    assert torch.equal(q_out[p.toks:], tail)
    buf = p.table.long()[req, cell // 128] * p.stride
    grp, row = cell % 128 // 32, cell % 32
    vals = p.values()
    if p.fp8:
        near(vals[buf, grp, :, row], (k_ref / p.k_scale).clamp(-448, 448), 2.0 ** -4, 2.0 ** -10)
        want = (v[:p.toks].float() / p.v_scale).clamp(-448, 448).to(torch.float8_e4m3fn).double()
        assert torch.equal(vals[buf + 1, grp, :, row], want)
    else:
        near(vals[buf, grp, :, row], k_ref, 2.0 ** -9 * 2)
        assert torch.equal(p.pool[buf + 1, grp, :, row], v[:p.toks])
    # nothing else of the pool is written
    p.pool[buf, grp, :, row] = before[buf, grp, :, row]
    p.pool[buf + 1, grp, :, row] = before[buf + 1, grp, :, row]
    raw = torch.uint8 if p.fp8 else torch.int16
    assert torch.equal(p.pool.view(raw), before.view(raw))


@pytest.mark.parametrize("hq,hk,d,fp8", [(32, 4, 128, False), (64, 4, 128, False), (32, 4, 128, True), (8, 2, 64, False),
                                         (1, 1, 128, False), (1, 1, 64, False), (6, 3, 128, True), (5, 5, 64, False)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_stage_heads_and_types(hq, hk, d, fp8, interleaved):
    p = Rows([5, 1, 130, 17], [0, 127, 250, 3], hq, hk, d, fp8=fp8, stride=3, pad=3, seed=hq)
    check_stage(p, d, interleaved)


@pytest.mark.parametrize("rot", [0, 8, 24, 64, 96, 128])
@pytest.mark.parametrize("interleaved", [False, True])
def test_stage_partial_rotation(rot, interleaved):
    p = Rows([3, 40], [60, 5], 8, 2, 128, seed=rot)
    check_stage(p, rot, interleaved)


@pytest.mark.parametrize("norm", [False, True])
def test_stage_without_norm_and_from_contiguous(norm):
    check_stage(Rows([9, 2], [0, 500], 12, 2, 128, seed=1), 64, False, norm=norm, packed=False)


def test_stage_in_place_queries():
    check_stage(Rows([9, 2, 33], [0, 500, 1], 12, 2, 128, seed=1, pad=2), 128, False, packed=False, in_place=True)


def test_stage_uniform_rows_and_empty_requests():
    check_stage(Rows([4] * 5, [0, 1, 124, 128, 700], 8, 2, 128, uniform=True, pad=6), 128, False)
    check_stage(Rows([0, 4, 0, 0, 7, 0], [10, 1, 0, 5, 128, 3], 8, 2, 128, pad=1), 128, False)


@pytest.mark.parametrize("batch", [1, 31, 33, 1100])
def test_stage_many_requests(batch):
    """The 32-ary request search over one, two and three rounds, empty requests among them."""
    new = [(i * 7) % 4 for i in range(batch)]
    new[0] = 2
    check_stage(Rows(new, [(i * 13) % 90 for i in range(batch)], 2, 1, 64), 64, False)


def test_stage_positions():
    p = Rows([6, 3], [40, 10], 8, 2, 128, pad=2)
    pos = torch.tensor([40, 41, 41, 42, 42, 42, 10, 11, 11, -5, 1 << 30])  # padded rows' positions are not looked at
    check_stage(p, 128, False, positions=pos)


def test_stage_far_positions_and_extremes():
    """Rows of zeros, of one large value and of the type's largest values."""
    p = Rows([8], [100], 4, 1, 128)
    q, k, v, w = inputs(p, packed=False)
    q[0], k[0] = 0, 0
    q[1], k[1] = 0, 0
    q[1, :, 5], k[1, :, 9] = 1e18, -1e18   # the squares' mean stays in range
    table = rope_table(200000, 128, 1e6).to(p.dev)
    pos = torch.tensor([199999, 131071, 65537, 0, 1, 2, 3, 4], dtype=torch.int32, device=p.dev)
    q_out = torch.empty_like(q)
    T.trtv_norm_rope_stage(p.geom, q, k, v, w[0], w[1], 1e-6, table, 128, False, pos, p.indptr, q_out, p.pool, p.table,
                           p.kv_lens)
    ref = norm_rope(q, w[0], 1e-6, table[pos.long()], 128, False)
    assert torch.isfinite(q_out.float()).all() and (q_out[0] == 0).all()
    assert ((q_out.double() - ref).abs() <= ref.abs() * 2.0 ** -8 + ref.abs().amax(-1, keepdim=True) * 2.0 ** -15).all()


def test_stage_device_errors():
    """Bad lengths, pages, positions and qo_indptr set their bits; the tokens concerned are not staged."""
    def call(p, positions=None, indptr=None, table_len=None):
        q, k, v, w = inputs(p)
        tab = rope_table(table_len or max(p.kv) + 1, 128).to(p.dev)
        out = torch.full((p.rows, p.hq, p.d), 3.0, dtype=torch.bfloat16, device=p.dev)
        before = p.pool.clone()
        T.trtv_norm_rope_stage(p.geom, q, k, v, *w, 1e-6, tab, 128, False, positions,
                               p.indptr if indptr is None else indptr, out, p.pool, p.table, p.kv_lens)
        err = T.trtv_get_device_error()
        changed = (p.pool.view(torch.int16) != before.view(torch.int16)).any(-1).any(2).sum().item()  # K and V cells
        return out, err, changed

    p = Rows([4, 4], [10, 20], 4, 2, 128)
    p.kv_lens[0] = 3   # fewer than its new tokens
    out, err, changed = call(p)
    assert err == T.DEVERR_KV_LEN and (out[:4] == 0).all() and (out[4:] != 0).any() and changed == 8
    p = Rows([4, 4], [10, 20], 4, 2, 128)
    p.kv_lens[1] = 129 * p.mp
    out, err, changed = call(p)
    assert err == T.DEVERR_KV_LEN and (out[4:] == 0).all() and changed == 8
    for bad in (-1, 1 << 20):
        p = Rows([4, 4], [10, 20], 4, 2, 128)
        p.table[1, 0] = bad
        out, err, changed = call(p)
        assert err == T.DEVERR_PAGE_ID and changed == 8 and (out[4:] != 0).any()
    p = Rows([4, 4], [10, 20], 4, 2, 128)
    pos = torch.tensor([0, -1, 2, 3, 24, 1, 1, 1], dtype=torch.int32, device=p.dev)
    out, err, changed = call(p, positions=pos, table_len=24)
    assert err == T.DEVERR_POSITION and changed == 12 and (out[1] == 0).all() and (out[4] == 0).all()
    for bad, kept in (([0, 5, 4], 0), ([1, 4, 8], 8), ([0, 4, 9], 8), ([0, 4, -3], 8), ([0, 4, 1 << 30], 8)):
        p = Rows([4, 4], [10, 20], 4, 2, 128)
        out, err, changed = call(p, indptr=torch.tensor(bad, dtype=torch.int32, device=p.dev))
        assert changed <= 16
        if bad != [0, 4, -3]:
            assert err == T.DEVERR_INDPTR


# ---------------------------------------------------------------------------
# commits

def commit_ref(p, paths, pool):
    pool = pool.clone()
    lens = list(p.kv)
    for b, path in enumerate(paths):
        if path is None or p.new[b] == 0:
            continue
        def cell(i):
            pos = p.ctx[b] + i
            return int(p.table[b, pos // 128]) * p.stride, pos % 128 // 32, pos % 32
        src = [[pool[cell(t)[0] + kv, cell(t)[1], :, cell(t)[2]].clone() for kv in (0, 1)] for t in path]
        for i, rows in enumerate(src):
            for kv in (0, 1):
                pool[cell(i)[0] + kv, cell(i)[1], :, cell(i)[2]] = rows[kv]
        lens[b] = p.ctx[b] + len(path)
    return pool, lens


def commit(p, paths, width=None, in_place=False, stream=None):
    width = width or max(1, max(len(x) for x in paths))
    path = torch.tensor([list(x) + [99999] * (width - len(x)) for x in paths], dtype=torch.int32, device=p.dev)
    plen = torch.tensor([len(x) for x in paths], dtype=torch.int32, device=p.dev)
    new = p.kv_lens if in_place else torch.full((p.B,), -7, dtype=torch.int32, device=p.dev)
    T.trtv_tree_commit(p.geom, p.pool, p.table, p.kv_lens, p.indptr, path, plen, new, stream)
    return new


@pytest.mark.parametrize("fp8,d,hq,hk,stride", [(False, 128, 32, 4, 2), (True, 128, 32, 4, 8), (False, 64, 8, 2, 3),
                                                (False, 128, 1, 1, 2), (False, 128, 64, 40, 2)][:4])
@pytest.mark.parametrize("in_place", [False, True])
def test_commit(fp8, d, hq, hk, stride, in_place):
    new = [16, 64, 1, 33, 128, 7, 0, 20]
    p = Rows(new, [0, 120, 500, 127, 255, 3, 9, 380], hq, hk, d, fp8=fp8, stride=stride, seed=3)
    g = torch.Generator().manual_seed(1)
    paths = []
    for i, n in enumerate(new):
        keep = torch.rand(n, generator=g) < (0.4 if i % 2 else 0.8)
        paths.append([t for t in range(n) if keep[t]])
    paths[2], paths[5] = [0], []                        # one node; nothing accepted
    paths[4] = list(range(128))                         # all of it: nothing moves
    raw = torch.uint8 if fp8 else torch.int16
    want, lens = commit_ref(p, paths, p.pool.view(raw))
    got = commit(p, paths, width=128, in_place=in_place)
    assert T.trtv_get_device_error() == 0
    assert got.tolist() == lens
    assert torch.equal(p.pool.view(raw), want)


def test_commit_uniform_and_long_moves():
    p = Rows([64] * 3, [64, 100, 1000], 4, 2, 128, uniform=True)
    paths = [list(range(1, 64)), list(range(0, 64, 2)), [63]]
    want, lens = commit_ref(p, paths, p.pool.view(torch.int16))
    got = commit(p, paths)
    assert got.tolist() == lens and torch.equal(p.pool.view(torch.int16), want)


def test_commit_device_errors():
    def both(change, bit):
        p = Rows([8, 8], [125, 20], 4, 2, 128)
        paths = [[0, 3, 5], [1, 2, 7]]
        change(p, paths)
        ok = [None, paths[1]]
        want, lens = commit_ref(p, ok, p.pool.view(torch.int16))
        lens[0] = int(p.kv_lens[0])
        got = commit(p, paths)
        assert T.trtv_get_device_error() == bit
        assert got.tolist() == lens
        assert torch.equal(p.pool.view(torch.int16), want)

    def path(x):
        def f(p, paths):
            paths[0] = x
        return f
    for bad in ([3, 3], [4, 2], [-1, 2], [0, 8], [0, 1 << 30], list(range(9))):
        both(path(bad), T.DEVERR_PATH)

    def table(j, v):
        def f(p, paths):
            p.table[0, j] = v
        return f
    both(table(0, -1), T.DEVERR_PAGE_ID)
    both(table(1, 1 << 20), T.DEVERR_PAGE_ID)

    def length(v):
        def f(p, paths):
            p.kv_lens[0] = v
        return f
    both(length(7), T.DEVERR_KV_LEN)
    both(length(1 << 20), T.DEVERR_KV_LEN)


def test_stage_and_commit_past_32_bit_offsets():
    """A pool of more than 2^31 elements, its last slots used."""
    p = Rows([6, 3], [125, 40], 4, 2, 128)
    slots = 1 << 14
    pool = torch.zeros(slots * 5, 4, 2, 32, 128, dtype=torch.bfloat16, device=p.dev)
    assert pool.numel() > 1 << 31
    for b in range(2):
        for j in range((p.kv[b] + 127) // 128):
            p.table[b, j] = slots - 1 - 3 * (2 * b + j)
    p.pool, p.stride, p.slots = pool, 5, slots
    p.geom.num_slots, p.geom.slot_stride = slots, 5
    q, k, v, w = inputs(p)
    out = torch.empty(p.rows, p.hq, p.d, dtype=torch.bfloat16, device=p.dev)
    T.trtv_norm_rope_stage(p.geom, q, k, v, None, None, 0.0, None, 0, False, None, p.indptr, out, p.pool, p.table, p.kv_lens)
    req, cell = place(p)
    buf = p.table.long()[req, cell // 128] * 5
    got = pool[buf, cell % 128 // 32, :, cell % 32]
    assert torch.equal(out, q) and torch.equal(got, k)
    assert torch.equal(pool[buf + 1, cell % 128 // 32, :, cell % 32], v)
    new = commit(p, [[0, 3, 5], [2]])
    assert new.tolist() == [128, 41] and T.trtv_get_device_error() == 0
    for b, path in ((0, [0, 3, 5]), (1, [2])):
        for i, t in enumerate(path):
            pos = p.ctx[b] + i
            at = int(p.table[b, pos // 128]) * 5
            row = p.start(b) + t
            assert torch.equal(pool[at, pos % 128 // 32, :, pos % 32], k[row])
            assert torch.equal(pool[at + 1, pos % 128 // 32, :, pos % 32], v[row])
    assert (pool != 0).any(-1).sum().item() <= 2 * 2 * 9


def test_calls_in_a_graph_and_on_another_stream():
    """Staging and commit captured once and replayed with lengths changed on the device."""
    p = Rows([4, 9], [10, 300], 8, 2, 128, extra_pages=2)
    q, k, v, w = inputs(p)
    tab = rope_table(1024, 128).to(p.dev)
    out = torch.zeros(p.rows, p.hq, p.d, dtype=torch.bfloat16, device=p.dev)
    path = torch.tensor([[0, 2, 3], [1, 4, 8]], dtype=torch.int32, device=p.dev)
    plen = torch.tensor([3, 2], dtype=torch.int32, device=p.dev)

    def step(pool, o, lens, stream=None):
        T.trtv_norm_rope_stage(p.geom, q, k, v, *w, 1e-6, tab, 128, False, None, p.indptr, o, pool, p.table, lens, stream)
        T.trtv_tree_commit(p.geom, pool, p.table, lens, p.indptr, path, plen, lens, stream)

    step(p.pool.clone(), out, p.kv_lens.clone())
    s = torch.cuda.Stream()
    lens, pool = p.kv_lens.clone(), p.pool.clone()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step(pool, out, lens)
    for first in (p.kv, [13, 200], [77, 129]):
        start = torch.tensor(first, dtype=torch.int32, device=p.dev)
        lens.copy_(start)
        pool.copy_(p.pool)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        pool2, out2, lens2 = p.pool.clone(), torch.zeros_like(out), start.clone()
        torch.cuda.synchronize()
        step(pool2, out2, lens2, s)
        s.synchronize()
        assert torch.equal(out, out2) and torch.equal(lens, lens2) and torch.equal(pool.view(torch.int16), pool2.view(torch.int16))
        assert lens.tolist() == [first[0] - 4 + 3, first[1] - 9 + 2]
