"""Problems over E2M1 caches: codes with an E4M3 scale for every 16 dims of a head."""
import torch

import speculative_decode_verify_kv_gb300 as T
from rows_common import GROUPS, SUB, Rows

LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def level_values(dev="cpu"):
    """Value of each of the 16 codes."""
    return torch.tensor(LEVELS + tuple(-x for x in LEVELS), dtype=torch.float64, device=dev)


def quantise(x, scale):
    """[..., d] values in binary32 -> code bytes [..., d / 2] and scale bytes [..., d / 16], step by step in binary32."""
    t = (x.float() / torch.tensor(scale, dtype=torch.float32, device=x.device)).unflatten(-1, (-1, 16))
    top = t.abs().amax(-1)                                  # (a NaN stays one)
    s = (top / 6).clamp(max=448).to(torch.float8_e4m3fn)
    u = t / s.float()[..., None]
    a = u.abs()
    code = torch.zeros_like(a, dtype=torch.uint8)
    for mid, to_upper in zip((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0), (False, True, False, True, False, True, False)):
        code += ((a >= mid) if to_upper else (a > mid)).to(torch.uint8)   # ties to the even code
    code |= (u < 0).to(torch.uint8) << 3
    code = torch.where(s.float()[..., None] > 0, code, torch.zeros_like(code)).flatten(-2)
    return code[..., 0::2] | code[..., 1::2] << 4, s.view(torch.uint8)


def join(codes, scales):
    """[..., 32, d / 2] and [..., 32, d / 16] -> a head's block [..., 18 d]."""
    return torch.cat([codes.flatten(-2), scales.flatten(-2)], -1)


def split(pool, d):
    return pool[..., :16 * d].unflatten(-1, (SUB, d // 2)), pool[..., 16 * d:].unflatten(-1, (SUB, d // 16))


def values_of(pool, d):
    """[buffers, 4, hk, 18 d] bytes -> [buffers, 4, hk, 32, d] in 64 bits, the tensor's scale left out."""
    codes, scales = split(pool, d)
    lv = level_values(pool.device)
    x = torch.stack([lv[(codes & 15).long()], lv[(codes >> 4).long()]], -1).flatten(-2)
    f = scales.contiguous().view(torch.float8_e4m3fn).double()
    return (x.unflatten(-1, (-1, 16)) * f[..., None]).flatten(-2)


class Fp4Rows(Rows):
    """Rows over an E2M1 cache; cache rows at or past kv_len, unused slots and other layers' buffers hold NaN scales."""

    def __init__(self, *args, k_scale=5.0 / 2688, v_scale=6.0 / 2688, **kw):
        super().__init__(*args, **kw)
        self.k_scale, self.v_scale = k_scale, v_scale
        pool = self.pool.float()
        out = torch.empty(pool.shape[0], GROUPS, self.hk, 18 * self.d, dtype=torch.uint8, device=pool.device)
        for kv, scale in ((0, k_scale), (1, v_scale)):
            out[kv::self.stride] = join(*quantise(pool[kv::self.stride], scale))
        for other in range(2, self.stride):
            out[other::self.stride] = 255
        self.pool = out
        self.geom.kv_dtype = T.TRTV_FP4_E2M1
        self.geom.k_scale, self.geom.v_scale = k_scale, v_scale
        self.k_scale, self.v_scale = self.geom.k_scale, self.geom.v_scale   # as binary32 holds them

    def values(self, pool=None):
        return values_of(self.pool if pool is None else pool, self.d)

    def dense(self, out_dtype=T.TRTV_BF16):
        nb = T.trtv_workspace_bytes(self.geom)
        assert nb > 0
        ws = torch.full((nb,), 255, dtype=torch.uint8, device=self.dev)
        out = torch.full((self.rows, self.hq, self.d), 7.0, device=self.dev,
                         dtype=torch.float32 if out_dtype == T.TRTV_F32 else torch.bfloat16)
        T.trtv_verify_dense(self.geom, self.q, self.pool, self.table, self.kv_lens, out, out_dtype, ws, nb)
        return out

    def read(self):
        k, v = (torch.full((self.rows, self.hk, self.d), 7.0, dtype=torch.bfloat16, device=self.dev) for _ in range(2))
        T.trtv_read_kv(self.geom, self.pool, self.table, self.kv_lens, self.indptr, k, v)
        return k, v


def check(p, out, mask=None, err=0, rows=None):
    """Attention against the 64-bit reference.  The weights enter the second product as f16 (each off by at most
    2^-11 of itself, together 2^-11 sum w |v|; one more 2^-11 covers the 32-bit scores: 128 products of order one,
    their sums and the exponential, off by under 2^-13, the weights that f16 cannot hold, under 2^-32 of the largest,
    and the 32-bit sums), the output is rounded once (bf16: 2^-8 |o|)."""
    torch.cuda.synchronize()
    assert T.trtv_get_device_error() == err
    ref, mag = p.attention(mask)
    rows = slice(0, p.toks) if rows is None else rows
    got = out.double()
    tol = 2 * 2.0 ** -11 * mag + (2.0 ** -8 * ref.abs() if out.dtype == torch.bfloat16 else 0) + 1e-6
    off = (got - ref).abs()[rows]
    assert torch.isfinite(got[rows]).all()
    worst = (off / tol[rows]).max().item() if off.numel() else 0
    assert worst <= 1, f"{worst} of the tolerance, {off.max().item()} off"
    assert (out[p.toks:] == 7).all()  # rows behind the last request's are left as they were


