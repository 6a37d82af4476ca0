"""How exactly prompt and tree attention weigh positions that count for little.

E4M3 caches take the weights into the second product as f16 (2^-11 of a weight;
below 2^-21 of the row's reference maximum 2^-32 of that), bf16 caches as bf16
(2^-8 of a weight).  Besides that, with N positions: the product is summed in
N / 16 steps that may each cut off a unit in the last place of its result
(2^-23), the weights in binary32 (N / 128 roundings of 2^-24 and some within a
page), and a logit of L bits (log2) is off by some 2^-24 L.  Outputs are f32.
"""
import math

import pytest
import torch

import speculative_decode_verify_kv_gb300 as T
from rows_common import Rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decode_verify_kv_gb300 import _build
    _build.build()
    T.load()
    T.trtv_get_device_error()


def line(n, fp8, unit, codes, values, hq=1, qo_len=1, num_ctas=1):
    """One request of n positions whose last token asks: position i has a logit (log2) of codes(i) * unit and the
    value values(i) in all dims (times the caches' scales); both are numbers that E4M3 holds exactly."""
    p = Rows([1], [127], hq, 1, 128, fp8=fp8, seed=1, qo_len=qo_len, num_ctas=num_ctas)
    p.mp = (n + 127) // 128
    p.slots, p.ctx, p.kv = p.mp + 1, [n - 1], [n]
    p.table = torch.randperm(p.slots, device=p.dev)[:p.mp].int().view(1, p.mp)
    p.kv_lens = torch.tensor([n], dtype=torch.int32, device=p.dev)
    p.geom.max_pages_per_req, p.geom.num_slots = p.mp, p.slots
    p.geom.sm_scale = unit * math.log(2) / p.k_scale
    p.q.zero_()
    p.q[:, :, 0] = 1
    pos = torch.arange(p.mp * 128, device=p.dev)
    pool = torch.zeros(p.slots * p.stride, 4, 1, 32, 128, device=p.dev)
    at = p.table[0].long() * p.stride
    pool[at, ..., 0] = codes(pos).float().view(p.mp, 4, 1, 32)
    pool[at + 1] = values(pos).float().view(p.mp, 4, 1, 32, 1)
    p.pool = pool.to(torch.float8_e4m3fn) if fp8 else pool.to(torch.bfloat16)
    assert torch.equal(p.pool.float(), pool)
    p.pool = p.pool.view(torch.uint8) if fp8 else p.pool
    return p


def tail_tolerance(n, fp8, bits, mag):
    """See the head of this file; `bits`: the logits' span."""
    return ((2.0 ** -11 + n * 2.0 ** -32 if fp8 else 2.0 ** -8) + n / 16 * 2.0 ** -23 + n / 128 * 2.0 ** -24 + 64 * 2.0 ** -24 +
            2 * bits * 2.0 ** -24) * mag + 1e-7


@pytest.mark.parametrize("call,hq,qo_len", [("prompt", 1, 1), ("prompt", 1, 200), ("prompt", 8, 1), ("tree", 1, 1), ("tree", 2, 128)])
@pytest.mark.parametrize("at", [0, 1, 70000, 131071])
@pytest.mark.parametrize("fp8,drop", [(True, 25.0), (True, 26.0), (True, 20.0), (True, 30.0), (False, 26.0)])
def test_one_position_and_many_far_below(call, hq, qo_len, at, fp8, drop):
    """One CTA reads the whole row: one dominant position among 131072, each 2^-drop of it, with other values."""
    n = 1 << 17
    p = line(n, fp8, drop / 256, lambda i: torch.where(i == at, 0.0, -256.0), lambda i: torch.where(i == at, 1.0, 4.0), hq=hq,
             qo_len=qo_len)
    if call == "tree":
        m = torch.ones(1, p.qo_len, dtype=torch.bool, device=p.dev)
        out = p.tree(m, T.TRTV_F32)
    else:
        m, out = None, p.prompt(T.TRTV_F32)
    torch.cuda.synchronize()
    assert T.trtv_get_device_error() == 0
    ref, mag = p.attention(m)
    assert ((out.double() - ref).abs() <= tail_tolerance(n, fp8, drop, mag)).all(), (out[0, 0, 0].item(), ref[0, 0, 0].item())


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("qo_len", [1, 200])
@pytest.mark.parametrize("step", [0.5, 1.0, 2.0, 3.5, 4.0, 4.5, 7.5, 8.0])
def test_rising_rows(fp8, qo_len, step):
    """Every page's logits lie `step` above the last page's, so the reference maximum lags behind or moves each time;
    the largest weight a row may reach above it is within f16."""
    n = 33 * 128
    p = line(n, fp8, step, lambda i: i // 128 - 16, lambda i: 1.0 + i // 128 % 3, qo_len=qo_len)
    out = p.prompt(T.TRTV_F32)
    torch.cuda.synchronize()
    assert T.trtv_get_device_error() == 0
    ref, mag = p.attention()
    assert ((out.double() - ref).abs() <= tail_tolerance(n, fp8, 16 * step, mag)).all(), (out[0, 0, 0].item(), ref[0, 0, 0].item())


def test_logits_beyond_their_own_precision_stay_finite():
    """Logits of 2^24 and more differ from each other by whole bits of rounding: the weights are then somewhere within
    f16, not infinite, and the row is an average of values of 1 and 2 (each within 2^-11)."""
    for qo_len in (1, 200):
        p = line(4096, True, 0.25, lambda i: i // 128 - 16, lambda i: 1.0 + i % 2, qo_len=qo_len)
        for scale in (2.0 ** 20, 2.0 ** 22, 2.0 ** 24):
            g = p.geom.sm_scale
            p.geom.sm_scale = g * scale
            out = p.prompt(T.TRTV_F32)
            torch.cuda.synchronize()
            p.geom.sm_scale = g
            assert torch.isfinite(out).all() and (out >= 0).all() and (out <= 2 * (1 + 2.0 ** -10) * p.v_scale).all()


@pytest.mark.parametrize("hq,hk", [(32, 4), (8, 8), (64, 1), (6, 2)])
@pytest.mark.parametrize("new,ctx", [([1, 3, 5], [700, 0, 2000]), ([200, 1, 130], [90, 1000, 0])])
def test_e4m3_weights_have_eleven_bits(hq, hk, new, ctx):
    """2^-11 for the weights, and the binary32 sums of the logits' 128 products (keys reach 4 here)."""
    p = Rows(new, ctx, hq, hk, 128, fp8=True, seed=hq)
    out = p.prompt(T.TRTV_F32)
    torch.cuda.synchronize()
    ref, mag = p.attention()
    x = max((p.q[p.start(b):p.start(b) + new[b]].double().abs().sum(-1).amax() * p.geom.sm_scale) for b in range(3)).item()
    assert 128 * 2.0 ** -23 * x * 4 < 2.0 ** -9
    assert ((out.double() - ref).abs() <= (2.0 ** -11 + 128 * 2.0 ** -23 * x * 4) * mag + 1e-6).all()
    if max(new) <= 128:
        m = p.tree_masks("random")
        out = p.tree(m, T.TRTV_F32)
        torch.cuda.synchronize()
        ref, mag = p.attention(m)
        assert ((out.double() - ref).abs() <= (2.0 ** -11 + 128 * 2.0 ** -23 * x * 4) * mag + 1e-6).all()
    assert T.trtv_get_device_error() == 0
