"""Attention over E2M1 caches against a 64-bit reference: the ladder (single tokens and a few), prompts, trees."""
import pytest
import torch

import speculative_decode_verify_kv_gb300 as T
from fp4_common import Fp4Rows, check, split

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decode_verify_kv_gb300 import _build
    _build.build()
    T.load()
    T.trtv_get_device_error()


HEADS = [(32, 4, 128), (8, 8, 128), (64, 4, 128), (12, 2, 128), (7, 1, 128), (48, 1, 128), (128, 1, 128), (8, 2, 64), (5, 1, 64),
         (16, 16, 64), (64, 1, 64), (20, 4, 64)]


@pytest.mark.parametrize("hq,hk,d", HEADS)
@pytest.mark.parametrize("n", [1, 2, 3, 4, 8])
def test_ladder_heads(hq, hk, d, n):
    p = Fp4Rows([n] * 5, [0, 31, 127, 300, 1000], hq, hk, d, uniform=True, seed=hq + d + n)
    check(p, p.dense())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("c", [0, 1, 15, 16, 30, 31, 32, 63, 95, 96, 126, 127, 128, 129, 255, 256, 1023, 5000])
def test_single_token_lengths(c, d):
    p = Fp4Rows([1], [c], 16, 2, d, uniform=True, seed=c, stride=3)
    check(p, p.dense())


@pytest.mark.parametrize("n,hq,hk", [(16, 8, 8), (32, 4, 4), (17, 2, 1), (32, 32, 8), (9, 8, 2), (31, 2, 2)])
def test_ladder_many_tokens(n, hq, hk):
    p = Fp4Rows([n] * 3, [0, 100, 777], hq, hk, 128, uniform=True, seed=n)
    check(p, p.dense())


@pytest.mark.parametrize("num_ctas", [1, 2, 3, 17, 152, 1024])
@pytest.mark.parametrize("hq,hk,d,n", [(32, 4, 128, 1), (8, 2, 64, 1), (32, 4, 128, 4), (64, 4, 128, 8)])
def test_ladder_split(num_ctas, hq, hk, d, n):
    """The same work over one CTA, over many, over more CTAs than there are pages of it."""
    p = Fp4Rows([n] * 6, [0, 900, 77, 2500, 3, 128], hq, hk, d, uniform=True, seed=9, num_ctas=num_ctas)
    check(p, p.dense())
    check(p, p.dense(T.TRTV_F32))


@pytest.mark.parametrize("hq,hk,d", HEADS)
def test_prompt_heads(hq, hk, d):
    p = Fp4Rows([130, 1, 300, 17, 128], [0, 0, 77, 1000, 128], hq, hk, d, pad=3, seed=hq + d)
    check(p, p.prompt())


@pytest.mark.parametrize("n,c", [(1, 0), (2, 0), (127, 0), (128, 0), (129, 0), (1, 127), (1, 128), (255, 1), (31, 97), (33, 95),
                                 (1000, 0), (777, 3333)])
@pytest.mark.parametrize("d", [64, 128])
def test_prompt_lengths(n, c, d):
    p = Fp4Rows([n], [c], 16, 2, d, seed=n)
    check(p, p.prompt())


@pytest.mark.parametrize("num_ctas", [1, 2, 3, 17, 152, 1024])
@pytest.mark.parametrize("hq,hk,d", [(32, 4, 128), (8, 2, 64)])
def test_prompt_split(num_ctas, hq, hk, d):
    p = Fp4Rows([150, 1, 600, 0, 40], [0, 900, 77, 5, 3], hq, hk, d, seed=9, num_ctas=num_ctas, pad=1)
    check(p, p.prompt())
    check(p, p.prompt(T.TRTV_F32))


def test_ragged_small_requests():
    """Few tokens a request, different numbers, some without any."""
    p = Fp4Rows([1, 0, 3, 2, 0, 4], [10, 5, 0, 127, 0, 700], 32, 4, 128, pad=2, stride=8)
    check(p, p.prompt())
    p = Fp4Rows([0, 0], [10, 0], 8, 2, 128, pad=4)
    check(p, p.prompt())
    new = [(i * 7) % 5 for i in range(1500)]
    p = Fp4Rows(new, [(i * 37) % 200 for i in range(1500)], 4, 2, 64)
    check(p, p.prompt())


@pytest.mark.parametrize("kind", ["tree", "chain", "random", "none", "junk"])
@pytest.mark.parametrize("hq,hk,d,hi", [(32, 4, 128, 16), (64, 4, 128, 40), (8, 8, 128, 128), (8, 2, 64, 7), (16, 4, 128, 4),
                                        (2, 2, 64, 31)])
def test_trees(kind, hq, hk, d, hi):
    new = [hi, 1, max(1, hi // 2), 0, hi]
    p = Fp4Rows(new, [0, 500, 127, 9, 3000], hq, hk, d, pad=2, seed=hi, qo_len=hi)
    m = p.tree_masks(kind)
    check(p, p.tree(m), m)


def test_agrees_with_a_bf16_cache():
    """Values that both caches hold exactly: the outputs differ by the roundings of the weights and the output alone."""
    from rows_common import Rows
    p = Fp4Rows([4] * 3, [1000, 60, 333], 32, 4, 128, uniform=True, k_scale=1.0, v_scale=1.0)
    r = Rows([4] * 3, [1000, 60, 333], 32, 4, 128, uniform=True)
    assert torch.equal(p.q, r.q) and torch.equal(p.table, r.table)
    r.pool = p.values().to(torch.bfloat16)   # 6 significant bits at most
    a, b = p.prompt(T.TRTV_F32).double(), r.prompt(T.TRTV_F32).double()
    check(p, p.dense())
    mag = p.attention()[1]
    assert ((a - b).abs() <= (2.0 ** -8 + 2.0 ** -10) * mag + 1e-6).all()


def test_largest_codes_and_scales():
    """Codes of +-6 under scales of 448 next to blocks of zeros and of the smallest scale."""
    p = Fp4Rows([4] * 2, [300, 1000], 16, 2, 128, uniform=True, seed=3, k_scale=2.0 ** -12, v_scale=2.0 ** -6)
    codes, scales = split(p.pool, 128)
    ok = (scales.view(torch.uint8) & 0x7F) != 0x7F     # not the NaN rows
    g = torch.Generator(device="cuda").manual_seed(1)
    pick = torch.randint(0, 4, scales.shape, generator=g, device="cuda")
    new = torch.where(pick == 0, 0x7E, torch.where(pick == 1, 0, torch.where(pick == 2, 1, scales.int()))).to(torch.uint8)
    scales.copy_(torch.where(ok, new, scales))
    p.q.mul_(0.25)
    # scores: sums of 128 products of up to 2688 * 2^-12 * |q|, off by 128 * 2^-24 of sum |q k| sm_scale, under 2^-13
    check(p, p.dense())


def test_masked_places_may_hold_anything():
    """Later tokens' cells (NaN scales) do not reach earlier rows."""
    p = Fp4Rows([200], [100], 8, 2, 128, seed=5)
    ref, _ = p.attention()
    clean = p.prompt()
    codes, scales = split(p.pool, 128)
    for t in range(150, 200):
        c = 100 + t
        s = int(p.table[0, c // 128]) * p.stride
        scales[s, c % 128 // 32, :, c % 32] = 0x7F
    out = p.prompt()
    torch.cuda.synchronize()
    assert torch.equal(out[:128], clean[:128])   # tiles that end before the NaN keys


def test_bad_lengths_and_pages():
    p = Fp4Rows([4] * 4, [100, 20, 300, 60], 32, 4, 128, uniform=True)
    p.kv_lens[1] = 3          # less than its tokens
    p.kv_lens[2] = 128 * p.mp + 1
    out = p.dense()
    check(p, out, err=T.DEVERR_KV_LEN, rows=torch.cat([torch.arange(0, 4), torch.arange(12, 16)]).cuda())
    assert (out[4:12] == 0).all()
    p = Fp4Rows([4] * 2, [100, 20], 32, 4, 128, uniform=True)
    p.good_table = p.table.clone()
    p.table[1, 0] = p.slots
    p.pool[0:2] = 0
    out = p.dense()
    check(p, out, err=T.DEVERR_PAGE_ID, rows=slice(0, 4))
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("n", [1, 4, 8])
def test_captured_and_replayed_with_other_lengths(n):
    p = Fp4Rows([n] * 4, [1000, 500, 300, 900], 32, 4, 128, uniform=True)
    nb = T.trtv_workspace_bytes(p.geom)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    out = torch.zeros(p.rows, p.hq, p.d, dtype=torch.bfloat16, device="cuda")

    def step():
        T.trtv_verify_dense(p.geom, p.q, p.pool, p.table, p.kv_lens, out, T.TRTV_BF16, ws, nb)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for lens in ([1000, 500, 300, 900], [n, 129, 128, 256 + n], [700, n, n + 1, 1]):
        lens = [max(n, x) for x in lens]
        p.kv_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        p.kv, p.ctx = lens, [x - n for x in lens]
        graph.replay()
        check(p, out)


def test_two_streams_with_a_workspace_each():
    a = Fp4Rows([1] * 8, [3000 + i for i in range(8)], 32, 4, 128, uniform=True, seed=1)
    b = Fp4Rows([4] * 8, [2000 + i for i in range(8)], 32, 4, 128, uniform=True, seed=2)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(5):
        with torch.cuda.stream(s1):
            x = a.dense()
        with torch.cuda.stream(s2):
            y = b.dense()
        outs.append((x, y))
    torch.cuda.synchronize()
    for x, y in outs:
        check(a, x)
        check(b, y)
        assert torch.equal(x, outs[0][0]) and torch.equal(y, outs[0][1])
