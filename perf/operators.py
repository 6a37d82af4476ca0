"""What is measured of the operators around tree verification over the paged KV cache.

Four operators, as a serving step calls them, on the framework's pool layout
(page buffers ``[4, kv_heads, 32, head_dim]``, K page of slot s at buffer
``s * stride``, its V page the next one):

stage   ``trtv_norm_rope_stage``: per-head RMS norm of the new tokens' queries
        and keys, their rotation, and the rows' way into the cache.
prompt  ``trtv_prompt_attn``: causal attention of packed prompts (or chunks of
        prompts) of different lengths over the cache.
tree    ``trtv_verify_tree``: a tree of drafted tokens over the cache.
commit  ``trtv_norm_rope_stage`` of a tree's tokens, then
        ``trtv_tree_commit`` of the accepted path: the part of a tree step
        that writes the cache (the staging puts back the rows that the commit
        moves, so that a pass can be repeated).

``run`` computes the plain form with elementary torch operations in 32 bits,
or, with ``own`` set, makes the framework's calls.
"""
import math
import random

import torch

own = False

PAGE, GROUPS, SUB = 128, 4, 32
EPS = 1e-6
ROPE_BASE = 1e6


# ---------------------------------------------------------------------------
# cases

def listed():
    return [
        # a verify step's new tokens: 64 requests of 4, the default verify geometry; latency counts
        dict(name="stage verify step", op="stage", batch=64, lo=4, hi=4, ctx_lo=1020, ctx_hi=8188, hq=32, hk=4, d=128,
             kv="bf16", stride=2, rot=128, interleaved=False, pad=0, lens=1),
        # packed prompts of different lengths, 64 query heads, half of each head rotated, padded rows at the end
        dict(name="stage prompts", op="stage", batch=12, lo=100, hi=4096, ctx_lo=0, ctx_hi=0, hq=64, hk=4, d=128,
             kv="bf16", stride=2, rot=64, interleaved=False, pad=57, lens=2),
        # prompt chunks into an E4M3 cache whose slots hold other layers' pages too, pairs side by side
        dict(name="stage chunks fp8", op="stage", batch=32, lo=1, hi=512, ctx_lo=0, ctx_hi=4096, hq=32, hk=4, d=128,
             kv="fp8", stride=8, rot=128, interleaved=True, pad=3, lens=3),
        # one short prompt, small heads; latency counts
        dict(name="prompt short d64", op="prompt", batch=1, lo=203, hi=203, ctx_lo=0, ctx_hi=0, hq=8, hk=2, d=64,
             kv="bf16", stride=2, pad=0, lens=4),
        # packed prompts of different lengths
        dict(name="prompt packed", op="prompt", batch=8, lo=100, hi=4000, ctx_lo=0, ctx_hi=0, hq=32, hk=4, d=128,
             kv="bf16", stride=2, pad=17, lens=5),
        # one long prompt
        dict(name="prompt long", op="prompt", batch=1, lo=16384, hi=16384, ctx_lo=0, ctx_hi=0, hq=32, hk=4, d=128,
             kv="bf16", stride=2, pad=0, lens=6),
        # chunks of prompts behind a cached prefix, E4M3 cache
        dict(name="prompt chunks fp8", op="prompt", batch=4, lo=300, hi=512, ctx_lo=2000, ctx_hi=12000, hq=32, hk=4, d=128,
             kv="fp8", stride=2, pad=0, lens=7),
        # a small tree of one request; latency counts
        dict(name="tree one request", op="tree", batch=1, lo=8, hi=8, ctx_lo=900, ctx_hi=900, hq=32, hk=4, d=128,
             kv="bf16", stride=2, pad=0, lens=8),
        # the default verify batch, trees of up to 16 nodes
        dict(name="tree batch", op="tree", batch=64, lo=9, hi=16, ctx_lo=1020, ctx_hi=8176, hq=32, hk=4, d=128,
             kv="bf16", stride=2, pad=5, lens=9),
        # wide groups, long contexts, large trees
        dict(name="tree long contexts", op="tree", batch=16, lo=32, hi=32, ctx_lo=16384, ctx_hi=32000, hq=64, hk=4, d=128,
             kv="bf16", stride=2, pad=0, lens=10),
        # a tree step's cache writes, the default verify batch
        dict(name="commit batch", op="commit", batch=64, lo=16, hi=16, ctx_lo=1020, ctx_hi=8176, hq=32, hk=4, d=128,
             kv="bf16", stride=2, rot=128, interleaved=False, pad=0, lens=11),
        # many requests, large trees, E4M3 cache
        dict(name="commit large fp8", op="commit", batch=256, lo=24, hi=64, ctx_lo=200, ctx_hi=2000, hq=32, hk=4, d=128,
             kv="fp8", stride=2, rot=64, interleaved=False, pad=0, lens=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _padded_cost(c):
    reqs = _requests(c)
    return len(reqs) * max(n for n, _ in reqs) * max(x + n for n, x in reqs) * c["hq"] * c["d"]


def draw(rng):
    op = rng.choice(["stage", "prompt", "tree", "commit"])
    hq, hk = rng.choice([(8, 2), (32, 4), (64, 4), (16, 2), (12, 2), (32, 8), (8, 8)])
    kv = rng.choice(["bf16", "bf16", "fp8"])
    d = 128 if kv == "fp8" else rng.choice([64, 128, 128])
    c = dict(op=op, hq=hq, hk=hk, d=d, kv=kv, stride=rng.choice([2, 2, 3, 8]), pad=rng.choice([0, 0, 1, 37]),
             lens=rng.randrange(1 << 30))
    if op in ("stage", "commit"):
        c["rot"] = rng.choice([32, 64, d])
        c["interleaved"] = rng.random() < 0.5
    if op == "stage":
        hi = _log(rng, 1, 8192)
        c.update(batch=_log(rng, 1, max(1, min(128, 32768 // hi))), hi=hi, lo=rng.randint(1, hi))
        c.update(ctx_lo=0, ctx_hi=_log(rng, 1, 8192))
    elif op == "prompt":
        while True:
            hi = _log(rng, 2, 12000)
            lo, ctx = rng.randint(1, hi), rng.choice([0, 0, _log(rng, 1, 8192)])
            c.update(batch=_log(rng, 1, 16), lo=lo, hi=hi, ctx_lo=ctx // 2, ctx_hi=ctx)
            if _padded_cost(c) <= 4000 ** 2 * 8 * 32 * 128:
                break
    elif op == "tree":
        while True:
            hi = _log(rng, 2, 64)
            ctx = _log(rng, 1, 32000)
            c.update(batch=_log(rng, 1, 128), lo=rng.randint(1, hi), hi=hi, ctx_lo=ctx // 2, ctx_hi=ctx)
            if _padded_cost(c) <= 16 * 32 * 32000 * 64 * 128 and c["batch"] * ctx * hk * d <= 64 * 8192 * 4 * 128:
                break
    else:
        hi = _log(rng, 2, 64)
        ctx = _log(rng, 1, 8000)
        c.update(batch=_log(rng, 1, 128), lo=rng.randint(1, hi), hi=hi, ctx_lo=ctx // 2, ctx_hi=ctx)
    return c


def _requests(c):
    """[(new tokens, cached tokens before them)] of the case's requests."""
    r = random.Random(c["lens"])
    return [(r.randint(c["lo"], c["hi"]), r.randint(c["ctx_lo"], c["ctx_hi"])) for _ in range(c["batch"])]


def _trees(c):
    """Parents of every request's tree nodes (-1: the tree's root hangs on the context), parents first."""
    r = random.Random(c["lens"] + 1)
    trees = []
    for n, _ in _requests(c):
        parents = [-1]
        for t in range(1, n):
            parents.append(r.randrange(max(0, t - 6), t))
        trees.append(parents)
    return trees


def _path(parents, r):
    """An accepted path: from a random node up to the root, in order."""
    node, path = r.randrange(len(parents)), []
    while node >= 0:
        path.append(node)
        node = parents[node]
    return path[::-1]


def work(c):
    reqs = _requests(c)
    toks = sum(n for n, _ in reqs)
    elem = 1 if c["kv"] == "fp8" else 2
    hq, hk, d = c["hq"], c["hk"], c["d"]
    if c["op"] in ("stage", "commit"):
        nbytes = toks * ((2 * hq + 2 * hk) * d * 2 + 2 * hk * d * elem + c["rot"] * 4)
        flops = toks * ((hq + hk) * (4 * d + 3 * c["rot"]))
        if c["op"] == "commit":
            r = random.Random(c["lens"] + 2)
            nbytes += sum(sum(i != j for i, j in enumerate(_path(p, r))) for p in _trees(c)) * 4 * hk * d * elem
        return {"bytes": nbytes, "flops": flops}
    kv = sum(n + x for n, x in reqs)
    nbytes = toks * hq * d * 4 + kv * 2 * hk * d * elem
    if c["op"] == "prompt":
        pairs = sum(n * x + n * (n + 1) // 2 for n, x in reqs)
    else:
        pairs = 0
        for (n, x), parents in zip(reqs, _trees(c)):
            depth = []
            for p in parents:
                depth.append(1 + (depth[p] if p >= 0 else 0))
            pairs += n * x + sum(depth)
    return {"bytes": nbytes, "flops": 4 * d * hq * pairs}


# ---------------------------------------------------------------------------
# inputs

def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    reqs = _requests(c)
    B, hq, hk, d, stride = len(reqs), c["hq"], c["hk"], c["d"], c["stride"]
    n = [a for a, _ in reqs]
    kv = [a + x for a, x in reqs]
    pages = [(x + PAGE - 1) // PAGE for x in kv]
    mp, slots = max(pages), sum(pages) + 3
    toks = sum(n)
    rows = toks + c["pad"]
    s = dict(op=c["op"], kv=c["kv"], B=B, hq=hq, hk=hk, d=d, stride=stride, tmax=max(n), lmax=max(kv), mp=mp, slots=slots,
             toks=toks, rows=rows, scale=1.0 / math.sqrt(d), k_scale=1.0, v_scale=1.0)
    fp8 = c["kv"] == "fp8"
    if fp8:
        s["k_scale"], s["v_scale"] = 5.0 / 448, 6.0 / 448

    def ints(v, dtype=torch.int32):
        return torch.tensor(v, dtype=dtype, device=dev)

    # pages of the requests, in a random order over the pool
    perm = torch.randperm(slots, generator=g, device=dev).to(torch.int32)
    cnt = ints(pages, torch.int64)
    first = torch.cumsum(cnt, 0) - cnt
    j = torch.arange(mp, device=dev)
    at = first[:, None] + torch.minimum(j[None], cnt[:, None] - 1)
    s["table"] = torch.where(j[None] < cnt[:, None], perm[at], perm.new_zeros(())).contiguous()
    s["kv_lens"] = ints(kv)
    indptr = [0]
    for a in n:
        indptr.append(indptr[-1] + a)
    s["indptr"] = ints(indptr)
    pool = torch.randn(slots * stride, GROUPS, hk, SUB, d, generator=g, device=dev, dtype=torch.float32)
    s["pool"] = (pool / s["k_scale"]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else pool.to(torch.bfloat16)
    del pool
    if c["op"] in ("stage", "commit"):
        # the projection's output: a token's query, key and value heads side by side
        qkv = torch.randn(rows, (hq + 2 * hk) * d, generator=g, device=dev, dtype=torch.float32).to(torch.bfloat16)
        s["q"] = qkv[:, :hq * d].view(rows, hq, d)
        s["k"] = qkv[:, hq * d:(hq + hk) * d].view(rows, hk, d)
        s["v"] = qkv[:, (hq + hk) * d:].view(rows, hk, d)
        s["qw"] = (1 + 0.2 * torch.randn(d, generator=g, device=dev)).to(torch.bfloat16)
        s["kw"] = (1 + 0.2 * torch.randn(d, generator=g, device=dev)).to(torch.bfloat16)
        s["rot"], s["interleaved"] = c["rot"], bool(c["interleaved"])
        ang = torch.arange(max(kv) + 1, device=dev, dtype=torch.float64)[:, None] * ROPE_BASE ** (
            -torch.arange(0, c["rot"], 2, device=dev, dtype=torch.float64) / c["rot"])[None]
        s["rope"] = torch.cat([ang.cos(), ang.sin()], 1).to(torch.float32)
        s["positions"] = None
        s["q_out"] = torch.zeros(rows, hq, d, dtype=torch.bfloat16, device=dev)
    else:
        s["q"] = torch.randn(rows, hq, d, generator=g, device=dev, dtype=torch.float32).to(torch.bfloat16)
        s["out"] = torch.zeros(rows, hq, d, dtype=torch.bfloat16, device=dev)
    if c["op"] in ("tree", "commit"):
        trees = _trees(c)
        words = (max(n) + 31) // 32
        masks, pos = [], []
        for (a, x), parents in zip(reqs, trees):
            m, dep = [], []
            for t, p in enumerate(parents):
                m.append((m[p] if p >= 0 else 0) | 1 << t)
                dep.append(dep[p] + 1 if p >= 0 else 0)
            masks += [[v >> 32 * w & 0xFFFFFFFF for w in range(words)] for v in m]
            pos += [x + v for v in dep]
        masks += [[0] * words] * c["pad"]
        s["mask"] = ints(masks, torch.int64).to(torch.int32)  # the low 32 bits
        if c["op"] == "commit":
            r = random.Random(c["lens"] + 2)
            paths = [_path(p, r) for p in trees]
            s["path"] = ints([p + [-1] * (max(n) - len(p)) for p in paths])
            s["path_len"] = ints([len(p) for p in paths])
            s["positions"] = ints(pos + [0] * c["pad"])  # a node's position is the context's length plus its depth
            s["new_lens"] = torch.zeros(B, dtype=torch.int32, device=dev)
    return s


# ---------------------------------------------------------------------------
# the plain forms

def _token_requests(s):
    """(request, index in the request) of every token row."""
    n = (s["indptr"][1:] - s["indptr"][:-1]).long()
    b = torch.repeat_interleave(torch.arange(s["B"], device=n.device), n, output_size=s["toks"])
    return b, torch.arange(s["toks"], device=n.device) - s["indptr"].long()[b]


def _cells(s, b, pos):
    """(K buffer, sub-page, row) of cache positions pos of requests b."""
    return s["table"].long()[b, pos // PAGE] * s["stride"], pos % PAGE // SUB, pos % SUB


def _norm(x, w):
    x = x.float()
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()


def _rotate(y, rope, interleaved):
    half = rope.shape[-1] // 2
    c, sn = rope[:, None, :half], rope[:, None, half:]
    a, b = (y[..., 0:2 * half:2], y[..., 1:2 * half:2]) if interleaved else (y[..., :half], y[..., half:2 * half])
    u, v = a * c - b * sn, b * c + a * sn
    turned = torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)
    return torch.cat([turned, y[..., 2 * half:]], -1)


def _stage(s):
    b, t = _token_requests(s)
    cell = (s["kv_lens"] - (s["indptr"][1:] - s["indptr"][:-1])).long()[b] + t
    pos = cell if s["positions"] is None else s["positions"].long()[:s["toks"]]
    rope = s["rope"][pos]
    m = s["toks"]
    s["q_out"][:m] = _rotate(_norm(s["q"][:m], s["qw"]), rope, s["interleaved"]).to(torch.bfloat16)
    k = _rotate(_norm(s["k"][:m], s["kw"]), rope, s["interleaved"])
    v = s["v"][:m].float()
    buf, grp, row = _cells(s, b, cell)
    pool = s["pool"]
    if s["kv"] == "fp8":
        k = (k / s["k_scale"]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        v = (v / s["v_scale"]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    pool[buf, grp, :, row] = k.to(pool.dtype)
    pool[buf + 1, grp, :, row] = v.to(pool.dtype)


def _commit(s):
    n = (s["indptr"][1:] - s["indptr"][:-1]).long()
    start = s["kv_lens"].long() - n
    width = s["path"].shape[1]
    i = torch.arange(width, device=n.device)[None].expand(s["B"], width)
    keep = i < s["path_len"][:, None]
    b = torch.arange(s["B"], device=n.device)[:, None].expand_as(i)[keep]
    src = _cells(s, b, (start[:, None] + s["path"].long())[keep])
    dst = _cells(s, b, (start[:, None] + i)[keep])
    pool = s["pool"]
    for kv in (0, 1):
        pool[dst[0] + kv, dst[1], :, dst[2]] = pool[src[0] + kv, src[1], :, src[2]]
    s["new_lens"].copy_(start + s["path_len"])


def _attend(s):
    """Scores of all requests at once, padded to the longest: [B, hk, tmax * group, lmax]."""
    B, hk, d, grp = s["B"], s["hk"], s["d"], s["hq"] // s["hk"]
    T, L, dev = s["tmax"], s["lmax"], s["q"].device
    pos = torch.arange(L, device=dev)
    buf, sub, row = _cells(s, torch.arange(B, device=dev)[:, None], pos[None].expand(B, L))

    def cache(kv, scale):
        x = s["pool"][buf + kv, sub, :, row]
        x = x.view(torch.float8_e4m3fn).float() * scale if s["kv"] == "fp8" else x.float()
        return x.masked_fill_((pos[None] >= s["kv_lens"][:, None])[..., None, None], 0).transpose(1, 2)

    n = (s["indptr"][1:] - s["indptr"][:-1]).long()
    b, t = _token_requests(s)
    q = torch.zeros(B, T, s["hq"], d, device=dev)
    q[b, t] = s["q"][:s["toks"]].float()
    q = q.view(B, T, hk, grp, d).permute(0, 2, 1, 3, 4).reshape(B, hk, T * grp, d)
    x = torch.matmul(q, cache(0, s["k_scale"]).transpose(2, 3)).mul_(s["scale"])
    tt = torch.arange(T, device=dev)
    start = s["kv_lens"].long() - n
    if s["op"] == "prompt":
        see = pos[None, None] <= (start[:, None] + tt[None])[..., None]
    else:
        mask = torch.zeros(B, T, s["mask"].shape[1], dtype=torch.int32, device=dev)
        mask[b, t] = s["mask"][:s["toks"]]
        j = pos[None] - start[:, None]  # which tree node a position is, per request
        jc = j.clamp(0, T - 1)
        word = torch.gather(mask, 2, (jc // 32)[:, None].expand(B, T, L))
        see = (j < 0)[:, None] | ((word >> (jc % 32)[:, None].int() & 1).bool() & (j < n[:, None])[:, None])
    x = x.view(B, hk, T, grp, L)
    x.masked_fill_(~see[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x.sub_(top.masked_fill_(top == -math.inf, 0)).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, hk, T * grp, L), cache(1, s["v_scale"])).view(B, hk, T, grp, d)
    o = torch.where(total > 0, o / total, o.new_zeros(()))
    o = o.permute(0, 2, 1, 3, 4).reshape(B, T, s["hq"], d)
    s["out"][:s["toks"]] = o[b, t].to(torch.bfloat16)


# ---------------------------------------------------------------------------
# the framework's calls

def _handle(s):
    """What a user's program keeps: the geometry and the workspace."""
    if "geom" not in s:
        import speculative_decode_verify_kv_gb300 as trtv
        s["geom"] = trtv.Geom(batch=s["B"], qo_len=s["tmax"], num_q_heads=s["hq"], num_kv_heads=s["hk"], head_dim=s["d"],
                              max_pages_per_req=s["mp"], num_slots=s["slots"], slot_stride=s["stride"],
                              kv_dtype=trtv.TRTV_FP8_E4M3 if s["kv"] == "fp8" else trtv.TRTV_BF16, sm_scale=s["scale"],
                              k_scale=s["k_scale"], v_scale=s["v_scale"], num_ctas=0)
        s["trtv"] = trtv
        if s["op"] in ("prompt", "tree"):
            s["ws_bytes"] = trtv.trtv_workspace_bytes_rows(s["geom"])
            s["ws"] = torch.empty(s["ws_bytes"], dtype=torch.uint8, device=s["q"].device)
    return s["trtv"], s["geom"]


def run(s):
    if own:
        trtv, geom = _handle(s)
        if s["op"] in ("stage", "commit"):
            trtv.trtv_norm_rope_stage(geom, s["q"], s["k"], s["v"], s["qw"], s["kw"], EPS, s["rope"], s["rot"],
                                      s["interleaved"], s["positions"], s["indptr"], s["q_out"], s["pool"], s["table"],
                                      s["kv_lens"])
            if s["op"] == "commit":
                trtv.trtv_tree_commit(geom, s["pool"], s["table"], s["kv_lens"], s["indptr"], s["path"], s["path_len"],
                                      s["new_lens"])
        elif s["op"] == "prompt":
            trtv.trtv_prompt_attn(geom, s["q"], s["pool"], s["table"], s["kv_lens"], s["indptr"], s["out"],
                                  trtv.TRTV_BF16, s["ws"], s["ws_bytes"])
        else:
            trtv.trtv_verify_tree(geom, s["q"], s["pool"], s["table"], s["kv_lens"], s["indptr"], s["mask"], s["out"],
                                  trtv.TRTV_BF16, s["ws"], s["ws_bytes"])
    elif s["op"] in ("stage", "commit"):
        _stage(s)
        if s["op"] == "commit":
            _commit(s)
    else:
        _attend(s)
    if s["op"] in ("prompt", "tree"):
        return {"out": s["out"]}
    # E4M3 codes are returned as E4M3 values
    outs = {"q": s["q_out"], "pool": s["pool"].view(torch.float8_e4m3fn) if s["kv"] == "fp8" else s["pool"]}
    if s["op"] == "commit":
        outs["new_lens"] = s["new_lens"]
    return outs


# ---------------------------------------------------------------------------
# 64 bits

def exact(c, seed):
    if 8 * work(c)["flops"] > 4e13 or (c["op"] in ("stage", "commit") and work(c)["bytes"] > 4e9):
        return None
    s = prepare(c, seed)
    reqs, hq, hk, d = _requests(c), c["hq"], c["hk"], c["d"]
    table = s["table"].long()
    fp8 = c["kv"] == "fp8"
    pool = s["pool"].view(torch.float8_e4m3fn).double() if fp8 else None
    if c["op"] in ("prompt", "tree"):
        out = torch.zeros(s["rows"], hq, d, dtype=torch.float64, device="cuda")
        r0 = 0
        for i, (n, x) in enumerate(reqs):
            L = n + x
            ids = table[i, :(L + PAGE - 1) // PAGE] * c["stride"]

            def flat(buf, scale):
                pages = (pool if fp8 else s["pool"])[buf].double() * scale  # [pages, 4, hk, 32, d]
                return pages.permute(2, 0, 1, 3, 4).reshape(hk, -1, d)[:, :L]

            K, V = flat(ids, s["k_scale"]), flat(ids + 1, s["v_scale"])
            q = s["q"][r0:r0 + n].double()
            if c["op"] == "tree":
                words = s["mask"][r0:r0 + n].long() & 0xFFFFFFFF
                bits = torch.stack([words[:, k // 32] >> (k % 32) & 1 for k in range(n)], 1).bool()
                see = torch.cat([torch.ones(n, x, dtype=torch.bool, device="cuda"), bits], 1)
            for t0 in range(0, n, 2048):
                t1 = min(n, t0 + 2048)
                ok = see[t0:t1] if c["op"] == "tree" else (
                    torch.arange(L, device="cuda")[None] <= torch.arange(x + t0, x + t1, device="cuda")[:, None])
                for h in range(hq):
                    kh = h // (hq // hk)
                    logit = (q[t0:t1, h] @ K[kh].T * s["scale"]).masked_fill(~ok, -math.inf)
                    out[r0 + t0:r0 + t1, h] = torch.softmax(logit, -1) @ V[kh]
            r0 += n
        return {"out": out}
    # stage and commit, token rows laid out request by request
    m = s["toks"]
    req = torch.cat([torch.full((n,), i, device="cuda") for i, (n, _) in enumerate(reqs)])
    cell = torch.cat([torch.arange(x, x + n, device="cuda") for n, x in reqs])
    angle_row = s["rope"].double()[cell if s["positions"] is None else s["positions"][:m].long()]

    def normed(x, w):
        x = x[:m].double()
        y = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / d + EPS) * w.double()
        half = c["rot"] // 2
        first = torch.arange(half, device="cuda")
        i0, i1 = (2 * first, 2 * first + 1) if c["interleaved"] else (first, first + half)
        co, si = angle_row[:, None, :half], angle_row[:, None, half:]
        z = y.clone()
        z[..., i0] = y[..., i0] * co - y[..., i1] * si
        z[..., i1] = y[..., i1] * co + y[..., i0] * si
        return z

    q = torch.zeros(s["rows"], hq, d, dtype=torch.float64, device="cuda")
    q[:m] = normed(s["q"], s["qw"])
    new = [normed(s["k"], s["kw"]) / s["k_scale"], s["v"][:m].double() / s["v_scale"]]
    values = pool if fp8 else s["pool"].double()
    place = (table[req, cell // PAGE] * c["stride"], cell % PAGE // SUB, cell % SUB)
    for kv in (0, 1):
        values[place[0] + kv, place[1], :, place[2]] = new[kv].clamp(-448, 448) if fp8 else new[kv]
    if c["op"] == "stage":
        return {"q": q, "pool": values}
    r0, lens = 0, []
    for i, ((n, x), k) in enumerate(zip(reqs, s["path_len"].tolist())):
        took = r0 + s["path"][i, :k].long()
        to = tuple(p[r0:r0 + k] for p in place)
        for kv in (0, 1):
            values[to[0] + kv, to[1], :, to[2]] = new[kv][took].clamp(-448, 448) if fp8 else new[kv][took]
        lens.append(x + k)
        r0 += n
    return {"q": q, "pool": values, "new_lens": torch.tensor(lens, dtype=torch.int32, device="cuda")}
