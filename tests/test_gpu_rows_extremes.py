"""Staging of zeros, of one value that outweighs its row and of the type's
largest values, and commits of caches with many heads.

Tolerances as in test_gpu_rows_stage.py: half a step of the stored type (bf16
2^-8, E4M3 2^-4 or 2^-10 below its normals) after binary32 arithmetic whose
error is under 2^-15 of the row's largest value."""
import math

import pytest
import torch

import speculative_decode_verify_kv_gb300 as T
from rows_common import Rows, norm_rope, rope_table
from test_gpu_rows_stage import commit, commit_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decode_verify_kv_gb300 import _build
    _build.build()
    T.load()
    T.trtv_get_device_error()


BIG = torch.finfo(torch.bfloat16).max


def staged(p, kv, pool=None):
    """The cache's rows of the new tokens, as values (E4M3 codes unscaled)."""
    x = []
    for b in range(p.B):
        for pos in range(p.ctx[b], p.kv[b]):
            x.append(p.values(pool)[int(p.table[b, pos // 128]) * p.stride + kv, pos % 128 // 32, :, pos % 32])
    return torch.stack(x)


def near(got, ref, half, floor=0.0):
    slack = ref.abs().amax(-1, keepdim=True) * 2.0 ** -15
    off = (got.double() - ref).abs()
    assert (off <= ref.abs() * half * (1 + 2.0 ** -10) + slack + floor).all(), off.max().item()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
def test_normed_rows_of_zeros_and_of_one_value(fp8, interleaved):
    """Queries, keys and values far apart in size; positions far out in the table."""
    p = Rows([9], [100], 4, 2, 128, fp8=fp8)
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(9, h, 128, generator=g).to(torch.bfloat16).to(p.dev) for h in (4, 2, 2))
    w = [(1 + 0.3 * torch.randn(128, generator=g)).to(torch.bfloat16).to(p.dev) for _ in range(2)]
    for x in (q, k, v):
        x[0] = 0
        x[1] = 0
        x[1, :, 5] = 1e18
        x[2] = 0
        x[2, :, 9] = -1e18
        x[3] *= 1e-18
        x[4] = 1e18
        x[5, :, 0] = 1e4
    v[6], v[7], v[8, :, ::2], v[8, :, 1::2] = BIG, -BIG, 2.0 ** -133, 0
    table = rope_table(200000, 128, 1e6).to(p.dev)
    pos = torch.tensor([199999, 131071, 65537, 0, 1, 2, 3, 199998, 5], dtype=torch.int32, device=p.dev)
    out = torch.full_like(q, 3.0)
    T.trtv_norm_rope_stage(p.geom, q, k, v, *w, 1e-6, table, 128, interleaved, pos, p.indptr, out, p.pool, p.table, p.kv_lens)
    assert T.trtv_get_device_error() == 0
    near(out, norm_rope(q, w[0], 1e-6, table[pos.long()], 128, interleaved), 2.0 ** -8)
    ref = norm_rope(k, w[1], 1e-6, table[pos.long()], 128, interleaved)
    if fp8:
        near(staged(p, 0), (ref / p.k_scale).clamp(-448, 448), 2.0 ** -4, 2.0 ** -10)
        assert staged(p, 0).abs().max() == 448   # rows of one value outgrow the scale: saturated
        assert torch.equal(staged(p, 1), (v.float() / p.v_scale).clamp(-448, 448).to(torch.float8_e4m3fn).double())
    else:
        near(staged(p, 0), ref, 2.0 ** -8)
        assert torch.equal(staged(p, 1), v.double())
    assert (out[0] == 0).all() and (staged(p, 0)[0] == 0).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_largest_values_without_norm(fp8):
    """Neither normed nor rotated: bf16 caches take the bits, E4M3 caches the saturated quotient; infinities saturate too,
    NaN stays."""
    p = Rows([3], [130], 4, 2, 128, fp8=fp8)
    g = torch.Generator().manual_seed(4)
    q, k, v = (torch.randn(3, h, 128, generator=g).to(torch.bfloat16).to(p.dev) for h in (4, 2, 2))
    for x in (q, k, v):
        x[0, :, ::2], x[0, :, 1::2] = BIG, -BIG
        x[1, :, 3], x[1, :, 4], x[1, :, 5] = math.inf, -math.inf, math.nan
        x[2, :, :64] = 2.0 ** -133
    out = torch.full_like(q, 3.0)
    T.trtv_norm_rope_stage(p.geom, q, k, v, None, None, 0.0, None, 0, False, None, p.indptr, out, p.pool, p.table, p.kv_lens)
    assert T.trtv_get_device_error() == 0
    assert torch.equal(out.view(torch.int16)[~q.isnan()], q.view(torch.int16)[~q.isnan()]) and (out.isnan() == q.isnan()).all()
    for kv, x, scale in ((0, k, p.k_scale), (1, v, p.v_scale)):
        want = (x.float() / scale).clamp(-448, 448).to(torch.float8_e4m3fn).double() if fp8 else x.double()
        assert torch.equal(staged(p, kv).nan_to_num(nan=7e30), want.nan_to_num(nan=7e30))


def test_value_scales():
    """A negative v_scale turns the codes' sign and the output's back; bf16 caches do not use it."""
    p = Rows([5, 3], [90, 0], 4, 2, 128, fp8=True)
    g = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn(8, h, 128, generator=g).to(torch.bfloat16).to(p.dev) for h in (4, 2, 2))
    p.geom.v_scale = p.v_scale = -p.v_scale
    T.trtv_norm_rope_stage(p.geom, q, k, v, None, None, 0.0, None, 0, False, None, p.indptr, p.q, p.pool, p.table, p.kv_lens)
    assert torch.equal(staged(p, 1), (v.float() / p.v_scale).clamp(-448, 448).to(torch.float8_e4m3fn).double())
    out = p.prompt(T.TRTV_F32)
    torch.cuda.synchronize()
    ref, mag = p.attention()
    assert ((out.double() - ref).abs() <= (2.0 ** -11 + 2.0 ** -10) * mag + 1e-6).all()
    p = Rows([5, 3], [90, 0], 4, 2, 128)
    p.geom.v_scale = 0.0
    T.trtv_norm_rope_stage(p.geom, q, k, v, None, None, 0.0, None, 0, False, None, p.indptr, p.q, p.pool, p.table, p.kv_lens)
    assert torch.equal(staged(p, 1), v.double())
    assert T.trtv_get_device_error() == 0


@pytest.mark.parametrize("fp8,d,hk", [(False, 128, 8), (False, 128, 9), (False, 128, 40), (False, 128, 32), (True, 128, 40), (True, 128, 33),
                                      (False, 64, 17), (False, 64, 1)])
def test_commit_of_many_heads(fp8, d, hk):
    """More 16-byte columns than the block has threads: some, all or no threads take another column."""
    new = [16, 40, 1, 33]
    p = Rows(new, [0, 120, 500, 127], hk, hk, d, fp8=fp8, stride=3, seed=hk)
    g = torch.Generator().manual_seed(hk)
    paths = [[t for t in range(n) if torch.rand(1, generator=g).item() < 0.5] for n in new]
    raw = torch.uint8 if fp8 else torch.int16
    want, lens = commit_ref(p, paths, p.pool.view(raw))
    got = commit(p, paths)
    assert T.trtv_get_device_error() == 0
    assert got.tolist() == lens and torch.equal(p.pool.view(raw), want)
