"""Staging into E2M1 caches, reading rows back (every cache type) and commits of accepted paths in E2M1 caches."""
import pytest
import torch

import speculative_decode_verify_kv_gb300 as T
from fp4_common import Fp4Rows, check, level_values, quantise, split
from rows_common import PAGE, SUB, Rows, norm_rope, rope_table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decode_verify_kv_gb300 import _build
    _build.build()
    T.load()
    T.trtv_get_device_error()


def cells(p):
    """(buffer, group, row) of every token, its position, and its packed row."""
    out, pos, rows = [], [], []
    for b in range(p.B):
        for t in range(p.new[b]):
            c = p.ctx[b] + t
            out.append((int(p.table[b, c // PAGE]) * p.stride, c % PAGE // SUB, c % SUB))
            pos.append(c)
            rows.append(p.start(b) + t)
    i = torch.tensor(out, device=p.dev).T
    return i, torch.tensor(pos, device=p.dev), torch.tensor(rows, device=p.dev)


def stage(p, rot, interleaved, weights=True, seed=0, positions=None, one_projection=True):
    g = torch.Generator().manual_seed(seed)
    hq, hk, d = p.hq, p.hk, p.d
    x = torch.randn(p.rows, (hq + 2 * hk) * d, generator=g).to(torch.bfloat16).to(p.dev)
    q, k, v = x[:, :hq * d].view(-1, hq, d), x[:, hq * d:(hq + hk) * d].view(-1, hk, d), x[:, (hq + hk) * d:].view(-1, hk, d)
    w = [(1 + 0.3 * torch.randn(d, generator=g)).to(torch.bfloat16).to(p.dev) if weights else None for _ in range(2)]
    rope = rope_table(max(p.kv) + 1, rot).to(p.dev) if rot else None
    q_out = torch.full((p.rows, hq, d), 7.0, dtype=torch.bfloat16, device=p.dev)
    T.trtv_norm_rope_stage(p.geom, q, k, v, w[0], w[1], 1e-6, rope, rot, interleaved, positions, p.indptr, q_out, p.pool, p.table,
                           p.kv_lens)
    return q, k, v, w, rope, q_out


@pytest.mark.parametrize("rot,interleaved", [(0, False), (8, False), (24, False), (64, False), (40, True), (64, True)])
@pytest.mark.parametrize("hq,hk,d,stride", [(32, 4, 128, 2), (5, 1, 64, 3), (6, 3, 128, 8)])
def test_stage(rot, interleaved, hq, hk, d, stride):
    p = Fp4Rows([4, 1, 130, 0, 33], [0, 127, 60, 3, 1000], hq, hk, d, stride=stride, pad=2, seed=rot + d)
    before = p.pool.clone()
    q, k, v, w, rope, q_out = stage(p, rot, interleaved)
    torch.cuda.synchronize()
    assert T.trtv_get_device_error() == 0
    at, pos, rows = cells(p)
    angle = rope[pos] if rot else None
    ref_q = norm_rope(q[rows], w[0], 1e-6, angle, rot, interleaved)
    ref_k = norm_rope(k[rows], w[1], 1e-6, angle, rot, interleaved)
    # bf16 once; the norm's 32-bit sums and products, and the rotation of a pair, are off by under 2^-18 of the pair's size
    assert ((q_out[rows].double() - ref_q).abs() <= 2.0 ** -8 * ref_q.abs() + 2.0 ** -16).all()
    assert (q_out[p.toks:] == 7).all()
    codes, scales = split(p.pool, d)
    # values are quantised as they are: bit for bit
    vc, vs = quantise(v[rows].float(), p.v_scale)
    assert torch.equal(scales[at[0] + 1, at[1], :, at[2]], vs)
    assert torch.equal(codes[at[0] + 1, at[1], :, at[2]], vc)
    # keys: 32-bit values off by under 2^-18 of the row's largest; the scale may be the next one, the code the nearest
    # but for that much
    t = (ref_k / p.k_scale).unflatten(-1, (-1, 16))
    err = 2.0 ** -18 * ref_k.abs().amax(-1)[..., None, None] / p.k_scale
    s = scales[at[0], at[1], :, at[2]].contiguous().view(torch.float8_e4m3fn).double()[..., None]
    ideal = (t.abs().amax(-1, keepdim=True) / 6).clamp(max=448)   # scales saturate
    assert ((s - ideal).abs() <= 2.0 ** -4 * ideal + err + 2.0 ** -10).all()   # E4M3: half a step, 2^-10 below its normal range
    byte = codes[at[0], at[1], :, at[2]]
    nib = torch.stack([byte & 15, byte >> 4], -1).flatten(-2).unflatten(-1, (-1, 16)).long()
    levels = level_values(p.dev)
    off = (levels[nib] * s - t).abs()
    best = (levels * s[..., None] - t[..., None]).abs().amin(-1)
    assert (off <= best + 2 * err).all()
    # nothing else of the pool was written
    after, kept = p.pool.clone(), before.clone()
    for kv in (0, 1):
        for buf in (after, kept):
            c, f = split(buf, d)
            c[at[0] + kv, at[1], :, at[2]] = 0
            f[at[0] + kv, at[1], :, at[2]] = 0
    assert torch.equal(after, kept)


@pytest.mark.parametrize("d", [64, 128])
def test_stage_special_values(d):
    """Zeros, one value far above its block, infinities, NaN, the largest and the smallest, ties, a negative value scale."""
    p = Fp4Rows([9], [60], 2, 1, d, k_scale=1.0, v_scale=-1.0)
    v = torch.zeros(9, 1, d, dtype=torch.bfloat16, device="cuda")
    v[1, 0, 3], v[1, 0, 20] = 5000, -1e30
    v[2, 0, 5], v[2, 0, 17] = float("inf"), -float("inf")
    v[3, 0, 7] = float("nan")
    v[4] = 3e38
    v[5] = 2.0 ** -133
    v[6, 0, ::16], v[6, 0, 1::16], v[6, 0, 2::16], v[6, 0, 3::16], v[6, 0, 4::16] = 6, 0.25, 0.75, -2.5, -5   # scale 1: ties
    v[6, 0, 5::16], v[6, 0, 6::16], v[6, 0, 7::16] = 1.25, 1.75, 3.5
    v[7] = 2.0 ** -8     # scale under half of E4M3's smallest: zeros
    v[8] = 3 * 2.0 ** -9
    k = v.clone()
    q = torch.zeros(9, 2, d, dtype=torch.bfloat16, device="cuda")
    q_out = torch.empty_like(q)
    T.trtv_norm_rope_stage(p.geom, q, k, v, None, None, 1e-6, None, 0, False, None, p.indptr, q_out, p.pool, p.table, p.kv_lens)
    torch.cuda.synchronize()
    assert T.trtv_get_device_error() == 0
    at, _, rows = cells(p)
    codes, scales = split(p.pool, d)
    for kv, x, scale in ((0, k, 1.0), (1, v, -1.0)):
        c, f = quantise(x[rows].float(), scale)
        got_c, got_f = codes[at[0] + kv, at[1], :, at[2]], scales[at[0] + kv, at[1], :, at[2]]
        is_nan = (f & 0x7F) == 0x7F
        assert torch.equal(is_nan, (got_f & 0x7F) == 0x7F)
        assert torch.equal(f[~is_nan], got_f[~is_nan])
        keep = ~is_nan.repeat_interleave(8, -1)
        assert torch.equal(c[keep] & 0x77, got_c[keep] & 0x77)   # (a zero may have either sign)
    kk, vv = p.read()
    torch.cuda.synchronize()
    assert torch.isnan(vv[3, 0, :16]).all() and not torch.isnan(vv[3, 0, 16:]).any()
    assert vv[2, 0, 5] == 2688 and vv[2, 0, 17] == -2688 and kk[4].eq(2688).all() and kk[7].eq(0).all()


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp4", "fp4 d64"])
@pytest.mark.parametrize("uniform", [True, False])
def test_read(kind, uniform):
    d = 64 if kind == "fp4 d64" else 128
    new, ctx = ([7] * 4, [0, 121, 500, 25]) if uniform else ([4, 1, 130, 0, 33], [0, 127, 60, 3, 1000])
    p = (Fp4Rows if kind.startswith("fp4") else Rows)(new, ctx, 12, 3, d, uniform=uniform, pad=2, stride=3,
                                                      **({"fp8": True} if kind == "fp8" else {}))
    k, v = (torch.full((p.rows, p.hk, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    T.trtv_read_kv(p.geom, p.pool, p.table, p.kv_lens, p.indptr, k, v)
    torch.cuda.synchronize()
    assert T.trtv_get_device_error() == 0
    at, _, rows = cells(p)
    x = p.values()
    for kv, out in ((0, k), (1, v)):
        ref = x[at[0] + kv, at[1], :, at[2]].float() * torch.tensor([p.geom.k_scale, p.geom.v_scale][kv], device="cuda")
        assert torch.equal(out[rows], ref.to(torch.bfloat16))
        assert (out[p.toks:] == 7).all()
    only = torch.full_like(v, 7.0)
    T.trtv_read_kv(p.geom, p.pool, p.table, p.kv_lens, p.indptr, None, only)
    assert torch.equal(only, v)


def test_read_bad_lengths_and_pages():
    p = Fp4Rows([2, 2, 2], [10, 130, 5], 8, 2, 128)
    p.kv_lens[0] = 1
    p.table[1, 1] = -3
    k, v = p.read()
    torch.cuda.synchronize()
    assert T.trtv_get_device_error() == T.DEVERR_KV_LEN | T.DEVERR_PAGE_ID
    assert (k[:4] == 0).all() and (v[:4] == 0).all() and (k[4:] != 7).all()


@pytest.mark.parametrize("hk,d,stride", [(4, 128, 2), (1, 64, 3), (3, 128, 8), (8, 64, 2)])
def test_commit(hk, d, stride):
    new, ctx = [16, 1, 40, 0, 9], [120, 127, 1000, 5, 30]
    p = Fp4Rows(new, ctx, 2 * hk, hk, d, stride=stride, qo_len=40)
    paths = [[0, 2, 5, 9, 15], [0], [1, 3, 20, 31, 32, 39], [], [0, 1, 2]]
    path = torch.tensor([x + [-1] * (6 - len(x)) for x in paths], dtype=torch.int32, device="cuda")
    want = p.pool.clone()
    wc, wf = split(want, d)
    oc, of = split(p.pool.clone(), d)
    for b, x in enumerate(paths):
        for i, j in enumerate(x):
            src, dst = ctx[b] + j, ctx[b] + i
            s, e = int(p.table[b, src // 128]) * stride, int(p.table[b, dst // 128]) * stride
            for kv in (0, 1):
                wc[e + kv, dst % 128 // 32, :, dst % 32] = oc[s + kv, src % 128 // 32, :, src % 32]
                wf[e + kv, dst % 128 // 32, :, dst % 32] = of[s + kv, src % 128 // 32, :, src % 32]
    T.trtv_tree_commit(p.geom, p.pool, p.table, p.kv_lens, p.indptr, path,
                       torch.tensor([len(x) for x in paths], dtype=torch.int32, device="cuda"), p.kv_lens)
    torch.cuda.synchronize()
    assert T.trtv_get_device_error() == 0
    assert torch.equal(p.pool, want)
    assert p.kv_lens.tolist() == [c + len(x) if n else c + n for c, x, n in zip(ctx, paths, new)]


def test_a_requests_life():
    """A prompt is staged and attended, then a tree, its path is committed, then a single token: all over one pool."""
    hq, hk, d = 16, 2, 128
    p = Fp4Rows([200, 77], [0, 0], hq, hk, d, seed=8, extra_pages=1)
    for step, (new, kind) in enumerate((([200, 77], "prompt"), ([12, 5], "tree"), ([1, 1], "token"))):
        p.new, p.qo_len = new, max(new)
        p.kv = [c + n for c, n in zip(p.ctx, new)]
        p.toks = p.rows = sum(new)
        p.geom.qo_len = max(new)
        p.kv_lens.copy_(torch.tensor(p.kv, dtype=torch.int32))
        p.indptr = torch.tensor([0, new[0], sum(new)], dtype=torch.int32, device="cuda")
        p.q = stage(p, 64, False, seed=step)[-1].contiguous()
        if kind == "prompt":
            check(p, p.prompt())
        elif kind == "tree":
            m = p.tree_masks()
            check(p, p.tree(m), m)
            path = torch.tensor([[0, 3, 7], [0, 1, -1]], dtype=torch.int32, device="cuda")
            T.trtv_tree_commit(p.geom, p.pool, p.table, p.kv_lens, p.indptr, path,
                               torch.tensor([3, 2], dtype=torch.int32, device="cuda"), p.kv_lens)
            p.kv = [203, 79]
            assert p.kv_lens.tolist() == p.kv
        else:
            p.indptr = None
            check(p, p.dense())
        p.ctx = list(p.kv)
