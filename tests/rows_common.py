"""Problems and 64-bit references of the packed-row calls (staging with norm
and rotation, prompt attention, tree attention, tree commit)."""
import math

import torch

import speculative_decode_verify_kv_gb300 as T

PAGE, GROUPS, SUB = 128, 4, 32


class Rows:
    """Packed requests over a paged pool; everything on the device.  Cache rows
    at or past kv_len, unused slots and other layers' buffers hold NaN."""

    def __init__(self, new, ctx, hq, hk, d, fp8=False, stride=2, pad=0, seed=0, dev="cuda", uniform=False, qo_len=None,
                 num_ctas=0, extra_pages=0):
        g = torch.Generator().manual_seed(seed)
        self.new, self.ctx = list(new), list(ctx)
        self.B, self.hq, self.hk, self.d, self.fp8, self.stride = len(new), hq, hk, d, fp8, stride
        self.kv = [n + c for n, c in zip(new, ctx)]
        self.toks = sum(new)
        self.rows = self.toks + pad
        pages = [max(0, (x + PAGE - 1) // PAGE) for x in self.kv]
        self.mp = max(1, max(pages)) + extra_pages
        self.slots = sum(pages) + 2
        self.k_scale, self.v_scale = (4.0 / 448, 5.0 / 448) if fp8 else (1.0, 1.0)
        perm = torch.randperm(self.slots, generator=g)
        table = torch.zeros(self.B, self.mp, dtype=torch.int32)
        pool = torch.full((self.slots * stride, GROUPS, hk, SUB, d), math.nan)
        at = 0
        for b, n in enumerate(pages):
            ids = perm[at:at + n]
            at += n
            table[b, :n] = ids.int()
            for kv in (0, 1):
                x = torch.randn(n, GROUPS, SUB, hk, d, generator=g).reshape(n * PAGE, hk, d)
                x[self.kv[b]:] = math.nan
                pool[ids * stride + kv] = x.view(n, GROUPS, SUB, hk, d).transpose(2, 3)
        if fp8:
            k = torch.arange(self.slots) * stride
            pool[k] /= self.k_scale
            pool[k + 1] /= self.v_scale
            pool = pool.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)  # (NaN stays)
        else:
            pool = pool.to(torch.bfloat16)
        indptr = [0]
        for n in new:
            indptr.append(indptr[-1] + n)
        self.indptr = None if uniform else torch.tensor(indptr, dtype=torch.int32, device=dev)
        self.table = table.to(dev)
        self.pool = pool.to(dev)
        self.kv_lens = torch.tensor(self.kv, dtype=torch.int32, device=dev)
        self.q = torch.randn(self.rows, hq, d, generator=g).to(torch.bfloat16).to(dev)
        self.qo_len = qo_len or max(1, max(new))
        self.geom = T.Geom(batch=self.B, qo_len=self.qo_len, num_q_heads=hq, num_kv_heads=hk, head_dim=d,
                           max_pages_per_req=self.mp, num_slots=self.slots, slot_stride=stride,
                           kv_dtype=T.TRTV_FP8_E4M3 if fp8 else T.TRTV_BF16, sm_scale=1 / math.sqrt(d),
                           k_scale=self.k_scale, v_scale=self.v_scale, num_ctas=num_ctas)
        self.gen, self.dev = g, dev
        self.good_table = None  # what the references read where a test spoils the table

    def start(self, b):
        return sum(self.new[:b])

    def values(self, pool=None):
        """The pool as 64-bit values (E4M3 codes unscaled)."""
        pool = self.pool if pool is None else pool
        return (pool.view(torch.float8_e4m3fn) if self.fp8 else pool).double()

    def cache(self, b, kv, pool=None):
        """[kv_len, hk, d] of request b in 64 bits, scaled."""
        n = (self.kv[b] + PAGE - 1) // PAGE
        table = self.table if self.good_table is None else self.good_table
        x = self.values(pool)[table[b, :n].long() * self.stride + kv]
        x = x.permute(0, 1, 3, 2, 4).reshape(n * PAGE, self.hk, self.d)[:self.kv[b]]
        return x * (self.v_scale if kv else self.k_scale)

    def attention(self, mask=None):
        """64-bit reference and the same sum over |v| (what a relative error of the weights is measured by);
        mask: bool [rows, qo_len] or None (causal)."""
        out = torch.zeros(self.rows, self.hq, self.d, dtype=torch.float64, device=self.dev)
        mag = torch.zeros_like(out)
        G = self.hq // self.hk
        for b in range(self.B):
            n, c, r = self.new[b], self.ctx[b], self.start(b)
            if n == 0 or c < 0:
                continue
            K, V = (self.cache(b, i).repeat_interleave(G, 1) for i in (0, 1))
            x = torch.einsum("thd,phd->htp", self.q[r:r + n].double(), K) * self.geom.sm_scale
            if mask is None:
                see = torch.arange(n + c, device=self.dev)[None] <= c + torch.arange(n, device=self.dev)[:, None]
            else:
                see = torch.cat([torch.ones(n, c, dtype=torch.bool, device=self.dev), mask[r:r + n, :n]], 1)
            x = x.masked_fill(~see[None], -math.inf)
            top = x.amax(-1, keepdim=True)
            w = torch.exp(x - torch.where(top == -math.inf, torch.zeros_like(top), top))
            s = w.sum(-1, keepdim=True)
            w = torch.where(s > 0, w / s, torch.zeros_like(w))
            out[r:r + n] = torch.einsum("htp,phd->thd", w, V)
            mag[r:r + n] = torch.einsum("htp,phd->thd", w, V.abs())
        return out, mag

    def workspace(self):
        nb = T.trtv_workspace_bytes_rows(self.geom)
        assert nb > 0
        return torch.full((nb,), 255, dtype=torch.uint8, device=self.dev), nb

    def prompt(self, out_dtype=T.TRTV_BF16, fill=7.0, stream=None):
        ws, nb = self.workspace()
        out = torch.full((self.rows, self.hq, self.d), fill, device=self.dev,
                         dtype=torch.float32 if out_dtype == T.TRTV_F32 else torch.bfloat16)
        T.trtv_prompt_attn(self.geom, self.q, self.pool, self.table, self.kv_lens, self.indptr, out, out_dtype, ws, nb,
                           stream)
        return out

    def tree(self, mask, out_dtype=T.TRTV_BF16, fill=7.0, stream=None):
        ws, nb = self.workspace()
        out = torch.full((self.rows, self.hq, self.d), fill, device=self.dev,
                         dtype=torch.float32 if out_dtype == T.TRTV_F32 else torch.bfloat16)
        T.trtv_verify_tree(self.geom, self.q, self.pool, self.table, self.kv_lens, self.indptr, pack(mask, self.qo_len),
                           out, out_dtype, ws, nb, stream)
        return out

    def tree_masks(self, kind="tree"):
        """bool [rows, qo_len]; kinds: tree (random parents), chain, random, none, junk (bits past n set)."""
        m = torch.zeros(self.rows, self.qo_len, dtype=torch.bool)
        for b in range(self.B):
            r = self.start(b)
            for t in range(self.new[b]):
                if kind == "chain":
                    m[r + t, :t + 1] = True
                elif kind in ("random", "junk"):
                    m[r + t, :self.new[b]] = torch.rand(self.new[b], generator=self.gen) < 0.5
                    if kind == "junk":
                        m[r + t, self.new[b]:] = True
                elif kind == "tree":
                    if t:
                        m[r + t] = m[r + int(torch.randint(max(0, t - 5), t, (1,), generator=self.gen))]
                    m[r + t, t] = True
        return m.to(self.dev)


def pack(mask, qo_len):
    words = (qo_len + 31) // 32
    m = torch.zeros(mask.shape[0], words * 32, dtype=torch.int64, device=mask.device)
    m[:, :mask.shape[1]] = mask.long()
    w = (m.view(-1, words, 32) << torch.arange(32, device=mask.device)).sum(-1)
    return w.to(torch.int32)


def rope_table(n, rot, base=1e4):
    a = torch.arange(n, dtype=torch.float64)[:, None] * base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)[None]
    return torch.cat([a.cos(), a.sin()], 1).float()


def norm_rope(x, w, eps, rope, rot, interleaved):
    """64-bit norm and rotation of [rows, heads, d]; rope: [rows, rot] or None."""
    y = x.double()
    if w is not None:
        y = y / torch.sqrt(y.pow(2).mean(-1, keepdim=True) + eps) * w.double()
    if rot:
        h = rot // 2
        i = torch.arange(h, device=y.device)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
        c, s = rope.double()[:, None, :h], rope.double()[:, None, h:]
        z = y.clone()
        z[..., a] = y[..., a] * c - y[..., b] * s
        z[..., b] = y[..., b] * c + y[..., a] * s
        y = z
    return y
