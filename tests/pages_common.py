"""Requests over shared pages, and the page calls done one page after the other on the host."""
import random

import torch

import speculative_decode_verify_kv_gb300 as T

PAGE, GROUPS, SUB = 128, 4, 32


def pages_for(n):
    return (n + PAGE - 1) // PAGE


def walk_fork(ref, rows, lens, num_pages, parent, grow):
    """(new counts, rows of slots, lengths, [(source, target, rows)] copied pages), or None where slots run out."""
    new_ref, out, copies, seen = list(ref), [], [], set()
    free = iter([i for i, r in enumerate(ref) if r == 0])
    for row, n in zip(rows, num_pages):
        for s in row[:n]:
            new_ref[s] -= 1
    for p, g in zip(parent, grow):
        length, held = (lens[p], rows[p][:num_pages[p]]) if p >= 0 else (0, [])
        slots, keeps = [], p >= 0 and p not in seen
        for j in range(pages_for(length + g)):
            if j < length // PAGE:
                slots.append(held[j])
            elif keeps and j < len(held) and ref[held[j]] == 1:
                slots.append(held[j])
            else:
                keeps = False
                s = next(free, None)
                if s is None:
                    return None
                slots.append(s)
                if j == length // PAGE and length % PAGE:
                    copies.append((held[j], s, length % PAGE))
            new_ref[slots[-1]] += 1
        seen.add(p)
        out.append(slots)
    return new_ref, out, [(lens[p] if p >= 0 else 0) + g for p, g in zip(parent, grow)], copies


def walk_compact(ref):
    used = [i for i, r in enumerate(ref) if r]
    holes = iter([i for i in range(len(used)) if ref[i] == 0])
    to = [-1] * len(ref)
    for i in used:
        to[i] = i if i < len(used) else next(holes)
    return to, len(used)


class Pages:
    """A pool with requests; `holders` counts holds that are no request's."""

    def __init__(self, slots, mp, hk=2, d=128, kv="bf16", stride=2, buffers=2, seed=0):
        self.r = random.Random(seed)
        self.slots, self.mp, self.hk, self.d, self.kv, self.stride, self.buffers = slots, mp, hk, d, kv, stride, buffers
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.block = {"bf16": 64 * d, "fp8": 32 * d, "fp4": 18 * d}[kv]
        self.bytes = torch.randint(0, 256, (slots * stride, GROUPS, hk, self.block), generator=g, device="cuda", dtype=torch.uint8)
        self.ref = [0] * slots
        self.rows, self.lens, self.num = [], [], []

    def add(self, length, spare=0, share=None, scattered=True):
        """A request of `length` tokens in free slots; share: the full pages of that request first."""
        row = [] if share is None else self.rows[share][:min(self.lens[share], length) // PAGE]
        for s in row:
            self.ref[s] += 1
        while len(row) < pages_for(length) + spare:
            free = [i for i, x in enumerate(self.ref) if x == 0]
            s = self.r.choice(free) if scattered else free[0]
            self.ref[s] = 1
            row.append(s)
        self.rows.append(row)
        self.lens.append(length)
        self.num.append(len(row))
        return len(self.rows) - 1

    def geom(self, batch, num_slots=None):
        kv = {"bf16": T.TRTV_BF16, "fp8": T.TRTV_FP8_E4M3, "fp4": T.TRTV_FP4_E2M1}[self.kv]
        return T.Geom(batch=batch, qo_len=1, num_q_heads=self.hk, num_kv_heads=self.hk, head_dim=self.d, max_pages_per_req=self.mp,
                      num_slots=num_slots or self.slots, slot_stride=self.stride, kv_dtype=kv, sm_scale=1.0, k_scale=1.0,
                      v_scale=1.0, num_ctas=0)

    def pool(self):
        return self.bytes.view(torch.bfloat16) if self.kv == "bf16" else self.bytes

    def table(self, junk=0):
        t = torch.full((len(self.rows), self.mp), junk, dtype=torch.int32)
        for b, row in enumerate(self.rows):
            t[b, :len(row)] = torch.tensor(row, dtype=torch.int32)
        return t.cuda()

    def parts(self):
        """The pool's rows, [slots, stride, 4, hk, 32, bytes of a row]: one part, or codes and scales."""
        x = self.bytes.view(self.slots, self.stride, GROUPS, self.hk, self.block)
        if self.kv != "fp4":
            return [x.unflatten(-1, (SUB, -1))]
        return [x[..., :16 * self.d].unflatten(-1, (SUB, -1)), x[..., 16 * self.d:].unflatten(-1, (SUB, -1))]

    def copied(self, copies):
        """The pool's bytes after copying the rows of [(source, target, rows)]."""
        keep = self.bytes
        self.bytes = keep.clone()
        for src, dst, n in copies:
            live = (torch.arange(PAGE, device="cuda") < n).view(GROUPS, 1, SUB, 1)
            for x in self.parts():
                x[dst, :self.buffers] = torch.where(live, x[src, :self.buffers], x[dst, :self.buffers])
        want, self.bytes = self.bytes, keep
        return want


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def fork(p, parent, grow=None, in_place=False, num=True, new_num=True, junk=0, stream=None):
    """The call on the device; everything that it could write, and what it held before."""
    n = len(parent)
    geom = p.geom(len(p.rows))
    nb = T.trtv_workspace_bytes_pages(geom, n)
    ws = torch.full((nb,), 255, dtype=torch.uint8, device="cuda")
    ref = ints(p.ref)
    new_ref = ref if in_place else torch.full_like(ref, -7)
    table = torch.full((n, p.mp), -7, dtype=torch.int32, device="cuda")
    lens, pages = ints([-7] * n), ints([-7] * n) if new_num else None
    T.trtv_pages_fork(geom, p.pool(), p.buffers, ref, p.table(junk), ints(p.lens), ints(p.num) if num else None, ints(parent),
                      None if grow is None else ints(grow), new_ref, table, lens, pages, ws, nb, stream)
    return new_ref, table, lens, pages


def check_fork(p, parent, grow=None, **kw):
    grow_ = [0] * len(parent) if grow is None else grow
    want_ref, rows, lens, copies = walk_fork(p.ref, p.rows, p.lens, p.num, parent, grow_)
    want = p.copied(copies)
    ref, table, new_lens, pages = fork(p, parent, grow, **kw)
    torch.cuda.synchronize()
    assert T.trtv_get_device_error() == 0
    assert ref.tolist() == want_ref
    assert table.tolist() == [r + [0] * (p.mp - len(r)) for r in rows]
    assert new_lens.tolist() == lens
    assert pages is None or pages.tolist() == [len(r) for r in rows]
    assert torch.equal(p.bytes, want)
    p.ref, p.rows, p.lens, p.num = want_ref, rows, lens, [len(r) for r in rows]


def compact(p, in_place=False, stream=None):
    geom = p.geom(len(p.rows))
    nb = T.trtv_workspace_bytes_pages(geom, 0)
    ws = torch.full((nb,), 255, dtype=torch.uint8, device="cuda")
    ref, table = ints(p.ref), p.table(junk=-5)
    new_ref, new_table = (ref, table) if in_place else (torch.full_like(ref, -7), torch.full_like(table, -7))
    slot_map, used = torch.full_like(ref, -7), ints([-7])
    T.trtv_pages_compact(geom, p.pool(), p.buffers, ref, table, ints(p.num), slot_map, used, new_ref, new_table, ws, nb, stream)
    return new_ref, new_table, slot_map, used


def check_compact(p, **kw):
    to, used = walk_compact(p.ref)
    src = [i for i, t in enumerate(to) if t >= 0 and t != i]
    keep = p.bytes.clone()
    x = keep.view(p.slots, p.stride, -1)
    if src:
        a, b = torch.tensor(src, device="cuda"), torch.tensor([to[i] for i in src], device="cuda")
        x[b, :p.buffers] = x[a, :p.buffers]
    want_ref = [0] * p.slots
    for i, t in enumerate(to):
        if t >= 0:
            want_ref[t] = p.ref[i]
    rows = [[to[s] for s in row] for row in p.rows]
    ref, table, slot_map, n = compact(p, **kw)
    torch.cuda.synchronize()
    assert T.trtv_get_device_error() == 0
    assert slot_map.tolist() == to and n.tolist() == [used]
    assert ref.tolist() == want_ref
    assert table.tolist() == [r + [0] * (p.mp - len(r)) for r in rows]
    assert torch.equal(p.bytes, keep)
    p.ref, p.rows = want_ref, rows
