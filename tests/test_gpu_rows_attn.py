"""Prompt and tree attention over the paged cache against a 64-bit reference.

Tolerance of an output element o = sum_p w_p v_p: the weights enter the second
product rounded to 16 bits (relative error at most 2^-8 each, so at most
2^-8 sum w |v| together; their sum is kept in 32 bits), the scores are 32-bit
sums of 128 products (relative weight error below 128 * 2^-23 * sum |q k| /
sqrt(D), under 2^-11 for these inputs), the output is rounded once (bf16:
2^-8 |o|), and split pieces are joined in 32 bits.
"""
import math

import pytest
import torch

import speculative_decode_verify_kv_gb300 as T
from rows_common import Rows, pack

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decode_verify_kv_gb300 import _build
    _build.build()
    T.load()
    T.trtv_get_device_error()


def check(p, out, mask=None, err=0, rows=None):
    torch.cuda.synchronize()
    assert T.trtv_get_device_error() == err
    ref, mag = p.attention(mask)
    rows = slice(0, p.toks) if rows is None else rows
    got = out.double()
    tol = (2.0 ** -8 + 2.0 ** -11) * mag + (2.0 ** -8 * ref.abs() if out.dtype == torch.bfloat16 else 0) + 1e-6
    off = (got - ref).abs()[rows]
    assert torch.isfinite(got[rows]).all()
    worst = (off / tol[rows]).max().item() if off.numel() else 0
    assert worst <= 1, f"{worst} of the tolerance, {off.max().item()} off"
    assert (out[p.toks:] == 7).all()  # rows behind the last request's are left as they were


HEADS = [(32, 4, 128), (8, 8, 128), (64, 4, 128), (12, 2, 128), (7, 1, 128), (48, 1, 128), (96, 1, 128), (128, 1, 128),
         (8, 2, 64), (5, 1, 64), (16, 16, 64), (64, 1, 64)]


@pytest.mark.parametrize("hq,hk,d", HEADS)
def test_prompt_heads(hq, hk, d):
    p = Rows([130, 1, 300, 17, 128], [0, 0, 77, 1000, 128], hq, hk, d, pad=3, seed=hq + d)
    check(p, p.prompt())


@pytest.mark.parametrize("hq,hk", [(32, 4), (8, 8), (7, 1), (128, 2)])
def test_prompt_fp8(hq, hk):
    p = Rows([130, 1, 300, 17, 128], [0, 0, 77, 1000, 128], hq, hk, 128, fp8=True, stride=8, pad=3, seed=hq)
    check(p, p.prompt())


@pytest.mark.parametrize("n,c", [(1, 0), (2, 0), (127, 0), (128, 0), (129, 0), (1, 127), (1, 128), (255, 1), (31, 97), (33, 95),
                                 (1000, 0), (777, 3333)])
@pytest.mark.parametrize("fp8", [False, True])
def test_prompt_lengths(n, c, fp8):
    p = Rows([n], [c], 16, 2, 128, fp8=fp8, seed=n)
    check(p, p.prompt())


def test_prompt_f32_output():
    p = Rows([200, 3], [0, 250], 8, 2, 128)
    check(p, p.prompt(T.TRTV_F32))
    p = Rows([200, 3], [0, 250], 8, 2, 64)
    check(p, p.prompt(T.TRTV_F32))


@pytest.mark.parametrize("num_ctas", [1, 2, 3, 17, 152, 1024])
@pytest.mark.parametrize("hq,hk,d,fp8", [(32, 4, 128, False), (8, 2, 64, False), (32, 4, 128, True)])
def test_prompt_split(num_ctas, hq, hk, d, fp8):
    """The same work over one CTA, over many, over more CTAs than there are pages of it."""
    p = Rows([150, 1, 600, 0, 40], [0, 900, 77, 5, 3], hq, hk, d, fp8=fp8, seed=9, num_ctas=num_ctas, pad=1)
    check(p, p.prompt())


def test_prompt_uniform_and_empty_requests():
    p = Rows([40] * 6, [0, 1, 88, 128, 700, 90], 8, 2, 128, uniform=True, pad=6)
    check(p, p.prompt())
    p = Rows([0, 40, 0, 0, 7, 0], [10, 1, 0, 5, 128, 3], 8, 2, 128, pad=1)
    check(p, p.prompt())
    p = Rows([0, 0], [10, 0], 8, 2, 128, pad=4)
    check(p, p.prompt())


def test_prompt_many_requests():
    new = [(i * 7) % 5 for i in range(1500)]
    p = Rows(new, [(i * 37) % 200 for i in range(1500)], 4, 2, 64)
    check(p, p.prompt())


def test_prompt_qo_len_above_what_is_used():
    """The capacity (a graph's worst case) may be larger than any request."""
    p = Rows([5, 9, 64], [100, 0, 300], 32, 4, 128, qo_len=4096, extra_pages=9)
    check(p, p.prompt())
    p = Rows([5, 9, 1], [100, 0, 300], 32, 4, 128, qo_len=128, extra_pages=9)
    m = p.tree_masks()
    check(p, p.tree(m), m)


def test_prompt_agrees_with_the_ladder():
    p = Rows([4] * 3, [1000, 60, 333], 32, 4, 128, uniform=True)
    out = p.prompt(T.TRTV_F32)
    ws_bytes = T.trtv_workspace_bytes(p.geom)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=p.dev)
    ref = torch.empty_like(out)
    T.trtv_verify_dense(p.geom, p.q, p.pool, p.table, p.kv_lens, ref, T.TRTV_F32, ws, ws_bytes)
    assert (out - ref).abs().max().item() < 2e-2
    check(p, out)


def test_prompt_extreme_scores():
    """Logits far apart and far from zero: the running maximum moves by more than the exponent's range, down as
    well as up, and one position takes all the weight."""
    for sign in (1, -1):
        p = Rows([300], [500], 8, 2, 128, seed=4)
        ramp = torch.linspace(-1, 1, p.mp * 128, device=p.dev) * sign
        for j in range(p.mp):
            s = int(p.table[0, j]) * p.stride
            cells = ramp[j * 128:(j + 1) * 128].view(4, 1, 32, 1)
            p.pool[s] = (p.pool[s].float() + 30 * cells).to(torch.bfloat16)
        p.q[:] = (p.q.float() * 3).to(torch.bfloat16)
        out = p.prompt()
        torch.cuda.synchronize()
        ref, mag = p.attention()
        # scores reach +-1000s, whose binary32 sums are off by up to 128 * 2^-24 of sum |q k| scale
        x = (p.q[:p.toks].double().abs().sum(-1).max() * 34 * p.geom.sm_scale).item()
        tol = (2.0 ** -8 + 128 * 2.0 ** -24 * x * 2) * mag + 2.0 ** -8 * ref.abs() + 1e-6
        assert ((out.double() - ref).abs() <= tol).all()


def test_prompt_infinite_and_nan_keys_past_the_bound():
    """Keys of later tokens may hold anything without touching earlier rows' weights."""
    p = Rows([64], [0], 8, 2, 128)
    clean = p.prompt().clone()
    s = int(p.table[0, 0]) * p.stride
    p.pool[s, 1, :, 8:] = math.nan       # keys of tokens 40 ..
    p.pool[s, 1, :, 20] = math.inf
    out = p.prompt()
    torch.cuda.synchronize()
    assert torch.equal(out[:40], clean[:40])
    T.trtv_get_device_error()


# ---------------------------------------------------------------------------
# trees

@pytest.mark.parametrize("kind", ["tree", "chain", "random", "none", "junk"])
@pytest.mark.parametrize("hq,hk,d,fp8", [(32, 4, 128, False), (8, 2, 64, False), (32, 4, 128, True), (12, 2, 128, False),
                                         (128, 1, 128, False)])
def test_tree_masks(kind, hq, hk, d, fp8):
    """Trees that start inside, at the end and at the start of a page, with and without context; rows that see
    nothing are zero."""
    p = Rows([16, 7, 1, 13, 16, 9], [0, 120, 127, 128, 1000, 500], hq, hk, d, fp8=fp8, pad=2, seed=hq + d)
    m = p.tree_masks(kind)
    out = p.tree(m)
    used = m & (torch.arange(p.qo_len, device=p.dev)[None] < torch.tensor(
        [n for n in p.new for _ in range(n)] + [0] * 2, device=p.dev)[:, None])
    check(p, out, used)
    if kind == "none":
        assert (out[:16] == 0).all()


@pytest.mark.parametrize("n,c", [(1, 0), (1, 5), (31, 0), (32, 97), (33, 96), (64, 64), (65, 1000), (96, 40), (127, 1), (128, 0),
                                 (128, 129), (128, 5000)])
@pytest.mark.parametrize("hq,hk,fp8", [(8, 8, False), (32, 4, False), (32, 4, True)])
def test_tree_sizes(n, c, hq, hk, fp8):
    p = Rows([n], [c], hq, hk, 128, fp8=fp8, seed=n + c)
    for kind in ("tree", "random"):
        m = p.tree_masks(kind)
        check(p, p.tree(m), m)


def test_tree_chain_is_the_prompt():
    p = Rows([24, 60, 3], [100, 1000, 0], 32, 4, 128)
    m = p.tree_masks("chain")
    assert (p.tree(m, T.TRTV_F32) - p.prompt(T.TRTV_F32)).abs().max().item() < 2e-2


@pytest.mark.parametrize("num_ctas", [1, 3, 152, 1024])
def test_tree_split(num_ctas):
    p = Rows([16, 0, 30, 2], [900, 3, 4000, 5], 32, 4, 128, num_ctas=num_ctas)
    m = p.tree_masks()
    check(p, p.tree(m), m)
    p = Rows([4, 0, 3, 2], [900, 3, 4000, 5], 32, 4, 128, num_ctas=num_ctas)
    m = p.tree_masks()
    check(p, p.tree(m), m)


@pytest.mark.parametrize("num_ctas", [0, 1, 2, 3, 7, 152, 1024])
@pytest.mark.parametrize("hq,hk,d,fp8", [(32, 4, 128, False), (16, 2, 64, False), (32, 4, 128, True)])
def test_trees_of_several_items(num_ctas, hq, hk, d, fp8):
    """More than 256 rows a KV head: the items of a head side by side on the CTAs (trees of equal size), or one
    after the other (one large tree among small ones); empty and invalid requests among them."""
    for new, ctx in (([64, 60, 64], [900, 2000, 3]), ([128], [700]), ([100, 0, 3, 2, 1, 5], [40, 9, 1500, 1000, 800, 0])):
        p = Rows(new, ctx, hq, hk, d, fp8=fp8, num_ctas=num_ctas, pad=3, seed=len(new))
        m = p.tree_masks("random")
        check(p, p.tree(m), m)
    p = Rows([64, 60, 64], [900, 2000, 3], hq, hk, d, fp8=fp8, num_ctas=num_ctas)
    p.kv_lens[1] = 5
    m = p.tree_masks()
    out = p.tree(m, T.TRTV_F32)
    torch.cuda.synchronize()
    assert T.trtv_get_device_error() == T.DEVERR_KV_LEN and (out[64:124] == 0).all()
    check(p, out, m, rows=slice(0, 64))
    check(p, out, m, rows=slice(124, 188))


def test_pages_past_32_bit_offsets():
    """Slots whose pages lie beyond 2^32 bytes and 2^31 elements of the pool."""
    p = Rows([40, 16], [200, 1000], 8, 2, 128)
    slots = 1 << 14                                     # 2 x 64 KB each: 2 GiB ...
    p.geom.num_slots, p.geom.slot_stride = slots, 5     # ... times 2.5
    pool = torch.zeros(slots * 5, 4, 2, 32, 128, dtype=torch.bfloat16, device=p.dev)
    assert pool.numel() > 1 << 31
    table = p.table.clone()
    for b in range(2):
        for j in range((p.kv[b] + 127) // 128):
            s, far = int(table[b, j]), slots - 1 - 7 * (16 * b + j)
            pool[far * 5], pool[far * 5 + 1] = p.pool[s * 2], p.pool[s * 2 + 1]
            p.table[b, j] = far
    p.pool, p.stride, p.slots = pool, 5, slots
    check(p, p.prompt())
    p.geom.qo_len = p.qo_len = 40
    m = p.tree_masks()
    check(p, p.tree(m), m)


# ---------------------------------------------------------------------------
# device errors, streams, graphs

@pytest.mark.parametrize("call", ["prompt", "tree"])
def test_device_errors(call):
    def run(p, indptr=None):
        if indptr is not None:
            p.indptr = torch.tensor(indptr, dtype=torch.int32, device=p.dev)
        out = p.prompt() if call == "prompt" else p.tree(p.tree_masks("chain"))
        torch.cuda.synchronize()
        return out, T.trtv_get_device_error()

    for L in (9, 0, -5, 1 << 20, -(1 << 31)):
        p = Rows([40, 10, 20], [100, 200, 300], 8, 2, 128)
        p.kv_lens[1] = L
        out, err = run(p)
        assert err == T.DEVERR_KV_LEN and (out[40:50] == 0).all()
        check(p, out, p.tree_masks("chain") if call == "tree" else None, rows=slice(0, 40))
    for bad in (-1, 1 << 20):
        p = Rows([40, 10, 20], [100, 200, 300], 8, 2, 128)
        p.good_table = p.table.clone()
        p.table[1, 0] = bad
        p.pool[p.pool.isnan()] = 0
        out, err = run(p)
        assert err == T.DEVERR_PAGE_ID and torch.isfinite(out.float()).all()
        check(p, out, p.tree_masks("chain") if call == "tree" else None, rows=slice(0, 40))
    for bad in ([0, 40, 39, 70], [2, 40, 50, 70], [0, 40, 50, 71], [0, 40, 1 << 30, 70], [0, 40, -9, 70]):
        p = Rows([40, 10, 20], [100, 200, 300], 8, 2, 128)
        out, err = run(p, bad)
        assert err & T.DEVERR_INDPTR
        assert torch.isfinite(out.float()).all()


@pytest.mark.parametrize("call", ["prompt", "tree"])
def test_graph_replay_with_changed_lengths(call):
    """Captured once; replayed with other lengths, other row counts and another mask on the device."""
    p = Rows([12, 30, 5], [300, 700, 20], 32, 4, 128, qo_len=32, pad=9, extra_pages=4)
    p.pool[p.pool.isnan()] = 0
    m = p.tree_masks("tree")
    words, out = pack(m, p.qo_len), torch.zeros(p.rows, p.hq, p.d, dtype=torch.bfloat16, device=p.dev)
    ws, nb = p.workspace()

    def go(o, stream=None):
        a = (p.geom, p.q, p.pool, p.table, p.kv_lens, p.indptr)
        if call == "prompt":
            T.trtv_prompt_attn(*a, o, T.TRTV_BF16, ws, nb, stream)
        else:
            T.trtv_verify_tree(*a, words, o, T.TRTV_BF16, ws, nb, stream)

    go(out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        go(out)
    for new, kv in (([12, 30, 5], p.kv), ([32, 0, 20], [400, 0, 25]), ([1, 2, 3], [1, 729, 3]), ([0, 0, 0], [5, 5, 5])):
        p.new, p.kv, p.toks = list(new), list(kv), sum(new)
        p.ctx = [k - n for n, k in zip(new, kv)]
        p.indptr.copy_(torch.tensor([0, new[0], new[0] + new[1], p.toks]))
        p.kv_lens.copy_(torch.tensor(kv))
        m = p.tree_masks("tree")
        words.copy_(pack(m, p.qo_len))
        out.fill_(7)
        torch.cuda.synchronize()
        graph.replay()
        check(p, out, m if call == "tree" else None)


def test_two_streams_with_their_own_workspaces():
    a = Rows([200, 30], [0, 900], 32, 4, 128, seed=1)
    b = Rows([16, 8], [2000, 100], 32, 4, 128, seed=2)
    m = b.tree_masks()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(sa):
        outs_a = [a.prompt() for _ in range(5)]
    with torch.cuda.stream(sb):
        outs_b = [b.tree(m) for _ in range(5)]
    torch.cuda.synchronize()
    for o in outs_a:
        check(a, o)
        assert torch.equal(o, outs_a[0])
    for o in outs_b:
        check(b, o, m)
        assert torch.equal(o, outs_b[0])


def test_a_turn():
    """Prompt, then two tree turns: stage, attend, commit, as a server runs them, against 64 bits throughout."""
    from rows_common import norm_rope, rope_table
    hq, hk, d = 16, 2, 128
    g = torch.Generator().manual_seed(0)
    p = Rows([150, 40], [0, 0], hq, hk, d, extra_pages=1)
    used = set()
    for b in range(2):  # room for the turns: one more page each
        used |= set(p.table[b, :(p.kv[b] + 127) // 128].tolist())
    free = [s for s in range(p.slots) if s not in used]
    for b in range(2):
        p.table[b, (p.kv[b] + 127) // 128] = free[b]
    p.pool.fill_(math.nan)
    tab = rope_table(1024, d).to(p.dev)
    w = [(1 + 0.3 * torch.randn(d, generator=g)).to(torch.bfloat16).to(p.dev) for _ in range(2)]
    K = [torch.zeros(0, hk, d, dtype=torch.float64, device=p.dev) for _ in range(2)]
    V = [torch.zeros(0, hk, d, dtype=torch.float64, device=p.dev) for _ in range(2)]

    def turn(new, masks, paths):
        rows = sum(new)
        qkv = torch.randn(rows, (hq + 2 * hk) * d, generator=g).to(torch.bfloat16).to(p.dev)
        q, k, v = (x.view(rows, -1, d) for x in qkv.split([hq * d, hk * d, hk * d], 1))
        ctx = [x.shape[0] for x in K]
        pos = []
        for b in range(2):
            for t in range(new[b]):
                pos.append(ctx[b] + (t if masks is None else int(masks[b][t].sum()) - 1))
        pos = torch.tensor(pos, dtype=torch.int32, device=p.dev)
        p.geom.qo_len = p.qo_len = max(new)
        p.new, p.ctx, p.rows, p.toks = list(new), ctx, rows, rows
        p.kv = [c + n for c, n in zip(ctx, new)]
        p.indptr = torch.tensor([0, new[0], rows], dtype=torch.int32, device=p.dev)
        p.kv_lens = torch.tensor(p.kv, dtype=torch.int32, device=p.dev)
        p.q = torch.empty(rows, hq, d, dtype=torch.bfloat16, device=p.dev)
        T.trtv_norm_rope_stage(p.geom, q, k, v, *w, 1e-6, tab, d, False, pos, p.indptr, p.q, p.pool, p.table, p.kv_lens)
        mask = None
        if masks is not None:
            mask = torch.zeros(rows, p.qo_len, dtype=torch.bool, device=p.dev)
            for b in range(2):
                mask[p.start(b):p.start(b) + new[b], :new[b]] = masks[b].to(p.dev)
        out = p.prompt() if masks is None else p.tree(mask)
        # what was staged is the rounded reference (to a step), and the attention is that of the staged rows
        kr = norm_rope(k, w[1], 1e-6, tab[pos.long()], d, False)
        for b in range(2):
            r = slice(p.start(b), p.start(b) + new[b])
            ck, cv = p.cache(b, 0), p.cache(b, 1)
            assert torch.equal(ck[:ctx[b]], K[b]) and torch.equal(cv[:ctx[b]], V[b])
            assert ((ck[ctx[b]:] - kr[r]).abs() <= kr[r].abs() * 2.0 ** -7 + 1e-4).all()
            assert torch.equal(cv[ctx[b]:], v[r].double())
            K[b], V[b] = ck, cv
        check(p, out, mask)
        if paths is not None:
            width = max(len(x) for x in paths)
            path = torch.tensor([x + [0] * (width - len(x)) for x in paths], dtype=torch.int32, device=p.dev)
            plen = torch.tensor([len(x) for x in paths], dtype=torch.int32, device=p.dev)
            T.trtv_tree_commit(p.geom, p.pool, p.table, p.kv_lens, p.indptr, path, plen, p.kv_lens)
            for b in range(2):
                keep = list(range(ctx[b])) + [ctx[b] + t for t in paths[b]]
                K[b], V[b] = K[b][keep], V[b][keep]
            assert p.kv_lens.tolist() == [x.shape[0] for x in K]

    turn([150, 40], None, None)
    for paths in ([[0, 2, 5, 6], [0]], [[0, 1, 3], [1, 2, 4, 8]]):
        masks = []
        for n in (12, 9):
            m = torch.zeros(n, n, dtype=torch.bool)
            for t in range(n):
                if t:
                    m[t] = m[int(torch.randint(0, t, (1,), generator=g))]
                m[t, t] = True
            masks.append(m)
        turn([12, 9], masks, paths)


def test_binding_refusals():
    """Tensors of another type, shape, device or layout are refused before anything runs."""
    p = Rows([8, 4], [100, 20], 8, 2, 128)
    ws, nb = p.workspace()
    out = torch.zeros(p.rows, p.hq, p.d, dtype=torch.bfloat16, device=p.dev)
    mask = pack(p.tree_masks(), p.qo_len)
    good = dict(q=p.q, kv_pool=p.pool, page_table=p.table, kv_lens=p.kv_lens, qo_indptr=p.indptr, tree_mask=mask, out=out,
                out_dtype=T.TRTV_BF16, workspace=ws, ws_bytes=nb)

    def prompt(**over):
        a = dict(good, **over)
        a.pop("tree_mask")
        T.trtv_prompt_attn(p.geom, **a)

    def tree(**over):
        T.trtv_verify_tree(p.geom, **dict(good, **over))

    bad = dict(q=[p.q.float(), p.q[:, :4], p.q.cpu(), p.q.transpose(0, 1)], kv_pool=[p.pool[:-2], p.pool.float(), p.pool.cpu()],
               page_table=[p.table.long(), p.table[:1], p.table.cpu()], kv_lens=[p.kv_lens.long(), p.kv_lens[:1]],
               qo_indptr=[p.indptr[:-1], p.indptr.long()], out=[out[:-1], out.float(), out.cpu()],
               workspace=[ws[:-1], ws.cpu()])
    for name, values in bad.items():
        for v in values:
            for call in (prompt, tree):
                with pytest.raises(ValueError, match=name):
                    call(**{name: v})
    for v in (mask.long(), mask[:-1], mask.cpu()):
        with pytest.raises(ValueError, match="tree_mask"):
            tree(tree_mask=v)
    with pytest.raises(T.TrtvError):
        prompt(ws_bytes=nb - 256)
    path, plen, new = (torch.zeros(*s, dtype=torch.int32, device=p.dev) for s in ((2, 3), (2,), (2,)))
    for a in ((path.long(), plen, new), (path[:1], plen, new), (path, plen[:1], new), (path, plen, new.cpu())):
        with pytest.raises(ValueError):
            T.trtv_tree_commit(p.geom, p.pool, p.table, p.kv_lens, p.indptr, *a)
    k = torch.zeros(p.rows, 2, 128, dtype=torch.bfloat16, device=p.dev)
    for a in ((p.q[:, :, :64], k, k), (p.q, k[:-1], k), (p.q, k, k.float()), (p.q, k.transpose(1, 2).contiguous().transpose(1, 2), k)):
        with pytest.raises(ValueError):
            T.trtv_norm_rope_stage(p.geom, *a, None, None, 0.0, None, 0, False, None, p.indptr, out, p.pool, p.table, p.kv_lens)
    # nothing to do: no rows
    empty = torch.zeros(3, dtype=torch.int32, device=p.dev)
    none = torch.zeros(0, p.hq, p.d, dtype=torch.bfloat16, device=p.dev)
    prompt(q=none, out=none, qo_indptr=empty)
    T.trtv_norm_rope_stage(p.geom, none, k[:0], k[:0], None, None, 0.0, None, 0, False, None, empty, none, p.pool, p.table,
                           p.kv_lens)
    torch.cuda.synchronize()
    assert T.trtv_get_device_error() == 0


@pytest.mark.parametrize("hq,hk,d,fp8", [(32, 4, 128, False), (32, 4, 128, True), (8, 2, 64, False), (2, 2, 128, False),
                                         (2, 2, 128, True)])
@pytest.mark.parametrize("call", ["prompt", "tree"])
def test_other_rows_of_a_tile_may_hold_anything(call, hq, hk, d, fp8):
    """Tiles reach past a request's rows into the next request's, and past the last request's: NaN there stays there."""
    p = Rows([37, 5, 3, 90], [100, 0, 300, 10], hq, hk, d, fp8=fp8, pad=40, seed=3)
    m = p.tree_masks()
    clean = p.prompt() if call == "prompt" else p.tree(m)
    p.q[37:42] = math.nan
    p.q[135:] = math.inf
    out = p.prompt() if call == "prompt" else p.tree(m)
    torch.cuda.synchronize()
    assert T.trtv_get_device_error() == 0
    assert torch.equal(out[:37], clean[:37]) and torch.equal(out[42:], clean[42:])
    assert not torch.isfinite(out[37:42]).any()


@pytest.mark.parametrize("fp8", [False, True])
def test_rows_of_zeros_and_tiny_scales(fp8):
    """Queries of zeros or far below one weigh every position they see alike, with a softmax scale that leaves the
    logits at zero as well."""
    for scale in (None, 1e-9, 1e-15):
        p = Rows([150, 3], [70, 0], 8, 2, 128, fp8=fp8, seed=6)
        if scale is not None:
            p.geom.sm_scale = scale
        p.q[0:50] = 0
        p.q[50:60] *= 2.0 ** -60
        p.q[60:62] *= 2.0 ** -110
        p.q[150:] = 0
        check(p, p.prompt())
        p = Rows([50, 3], [70, 0], 8, 2, 128, fp8=fp8, seed=7)
        if scale is not None:
            p.geom.sm_scale = scale
        p.q[0:30] = 0
        m = p.tree_masks("random")
        check(p, p.tree(m), m)


def test_a_step_without_tokens():
    p = Rows([3], [4], 8, 2, 128)
    empty = torch.zeros(2, dtype=torch.int32, device=p.dev)
    q = torch.empty(0, 8, 128, dtype=torch.bfloat16, device=p.dev)
    ws, nb = p.workspace()
    mask = torch.empty(0, 1, dtype=torch.int32, device=p.dev)
    T.trtv_prompt_attn(p.geom, q, p.pool, p.table, p.kv_lens, empty, torch.empty_like(q), T.TRTV_BF16, ws, nb)
    T.trtv_verify_tree(p.geom, q, p.pool, p.table, p.kv_lens, empty, mask, torch.empty_like(q), T.TRTV_BF16, ws, nb)
    torch.cuda.synchronize()
    assert T.trtv_get_device_error() == 0


@pytest.mark.parametrize("out_dtype", [T.TRTV_BF16, T.TRTV_F32])
@pytest.mark.parametrize("hq,hk,d,fp8", [(32, 4, 128, False), (8, 2, 64, False), (32, 4, 128, True)])
def test_buffers_at_the_smallest_alignment(out_dtype, hq, hk, d, fp8):
    """q, out and the pool 16 bytes past a 32-byte boundary, in prompts and trees of one tile and of two."""
    def off(x):
        n = 16 // x.element_size()
        y = torch.empty(x.numel() + n, dtype=x.dtype, device=x.device)
        y[n:] = x.flatten()
        return y[n:].view(x.shape)

    for new in ([130, 3, 40], [7, 9, 2]):
        p = Rows(new, [70, 500, 0], hq, hk, d, fp8=fp8, pad=2, seed=12)
        p.q, p.pool = off(p.q), off(p.pool)
        assert p.q.data_ptr() % 32 == 16
        ws, nb = p.workspace()
        out = off(torch.full((p.rows, hq, d), 7.0, device=p.dev,
                             dtype=torch.float32 if out_dtype == T.TRTV_F32 else torch.bfloat16))
        T.trtv_prompt_attn(p.geom, p.q, p.pool, p.table, p.kv_lens, p.indptr, out, out_dtype, ws, nb)
        check(p, out)
        if p.qo_len <= 128:
            m = p.tree_masks()
            out.fill_(7.0)
            T.trtv_verify_tree(p.geom, p.q, p.pool, p.table, p.kv_lens, p.indptr, pack(m, p.qo_len), out, out_dtype, ws, nb)
            check(p, out, m)


def test_one_request_over_many_ctas():
    """Small work is cut alike for every KV head, whatever the heads and CTAs."""
    for hq, hk, num_ctas in ((6, 3, 0), (14, 7, 0), (10, 5, 16), (12, 12, 7), (32, 4, 151)):
        p = Rows([5], [1900], hq, hk, 128, seed=hq, num_ctas=num_ctas)
        m = p.tree_masks()
        check(p, p.tree(m), m)
        p = Rows([60, 2], [900, 300], hq, hk, 64, seed=hq, num_ctas=num_ctas)
        check(p, p.prompt())
