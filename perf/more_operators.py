"""Workloads of a speculative step over a paged cache: rotating and appending
keys and values, attention for a tree of drafted tokens, verification of the
drafts, and keeping the accepted rows.

Each workload has a plain form (elementary torch operations in 32 bits, 64
where angles, long sums and borders need them, rounded once at the end) and,
with ``own`` set, the calls that a user of libfusekv makes.  ``exact`` states
the results in 64 bits.
"""

import math
import random

import torch

own = False

HEADS = {                    # query heads, KV heads, head dim, RoPE base
    "qwen3_8b": (32, 8, 128, 1e6),
    "llama3_8b": (32, 8, 128, 5e5),
    "llama3_70b": (64, 8, 128, 5e5),
    "mha": (8, 8, 128, 1e4),
    "narrow": (16, 4, 64, 1e4),
    "tiny": (4, 2, 64, 1e4),
}
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}

# rotary positions: layout, share of the head, scaling (kind, factor, original length, low, high, mscale)
ROPES = {
    "half": ("half", 1.0, ("none", 1.0, 0, 0.0, 0.0, 1.0)),
    "interleaved": ("interleaved", 1.0, ("none", 1.0, 0, 0.0, 0.0, 1.0)),
    "part": ("half", 0.5, ("none", 1.0, 0, 0.0, 0.0, 1.0)),
    "part_interleaved": ("interleaved", 0.25, ("linear", 4.0, 0, 0.0, 0.0, 1.0)),
    "llama3": ("half", 1.0, ("llama3", 8.0, 8192, 1.0, 4.0, 1.0)),
    "yarn": ("half", 1.0, ("yarn", 4.0, 32768, 1.0, 32.0, 0.1 * math.log(4.0) + 1.0)),
}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _case(op, **kw):
    c = dict(op=op, heads="qwen3_8b", dtype="bf16", rope="half", sequences=1, ctx=(512, 512),
             new=(1, 1), width=1, block_size=16, layers=1, tree=True, vocab=0, sampled=True, shape=0)
    c.update(kw)
    out = {}
    for k, v in c.items():
        out.update({k + "_lo": v[0], k + "_hi": v[1]} if isinstance(v, tuple) else {k: v})
    return out


def listed():
    return [
        # the next token of 64 running sequences joins the cache: latency counts
        _case("append", name="append, 64 next tokens", sequences=64, ctx=(100, 9000), shape=1),
        # a whole prompt's projections, rotated for a long context, go to their pages: bandwidth counts
        _case("append", name="append, prompt of 10368", heads="llama3_8b", rope="llama3", ctx=(0, 0),
              new=(10368, 10368), tree=False, shape=2),
        # fp32 layer, pairs side by side in a quarter of the head, ragged chunks of prompts
        _case("append", name="append, f32 part of the head", heads="tiny", dtype="f32",
              rope="part_interleaved", sequences=9, ctx=(0, 700), new=(1, 333), tree=False,
              block_size=24, shape=3),
        # one user's next token over 4096 tokens: latency counts
        _case("tree", name="next token over 4096", ctx=(4096, 4096), shape=4),
        # 16 sequences of a batch, each with a tree of about 16 drafts
        _case("tree", name="16 trees over 0.5 to 8k", heads="llama3_8b", sequences=16, ctx=(512, 8192),
              new=(9, 20), width=4, shape=5),
        # eight long contexts of the Llama-3-70B shape, full trees of 64 nodes: arithmetic counts
        _case("tree", name="8 trees of 64 over 33k", heads="llama3_70b", sequences=8,
              ctx=(33000, 33000), new=(64, 64), width=8, block_size=64, shape=6),
        # the fp32 layer of the small configuration
        _case("tree", name="f32 trees", heads="tiny", dtype="f32", sequences=5, ctx=(0, 300),
              new=(1, 12), width=3, block_size=24, shape=7),
        # one sequence's chain of drafts
        _case("verify", name="verify one chain", new=(8, 8), vocab=32000, shape=8),
        # a batch of trees whose drafts were sampled, a large vocabulary of odd size
        _case("verify", name="verify 64 sampled trees", sequences=64, new=(6, 16), width=3,
              vocab=150001, shape=9),
        # drafts looked up in the retrieved chunks: certain, not sampled
        _case("verify", name="verify 16 looked-up drafts", sequences=16, new=(2, 12), width=2,
              vocab=128000, sampled=False, shape=10),
        # the drafts of a step join the cache, the accepted ones stay: a small batch
        _case("accept", name="append 8 trees and keep", heads="llama3_8b", sequences=8, ctx=(64, 4000),
              new=(5, 24), width=4, shape=11),
        # the same for many sequences and several layers
        _case("accept", name="append 96 trees and keep, 8 layers", sequences=96, ctx=(10, 2000),
              new=(8, 32), width=4, layers=8, block_size=32, shape=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _span(rng, lo, hi):
    a, b = sorted((_log(rng, lo, hi), _log(rng, lo, hi)))
    return (a, b)


def draw(rng):
    shape = rng.randrange(1 << 30)
    op = rng.choice(["append", "append", "tree", "tree", "tree", "verify", "verify", "accept"])
    dtype = rng.choice(["bf16"] * 5 + ["f32"])
    kw = dict(dtype=dtype, heads=rng.choice(sorted(HEADS)) if dtype == "bf16" else "tiny", shape=shape,
              block_size=rng.choice([16, 16, 32, 64, 24, 5]), sequences=_log(rng, 1, 64),
              width=rng.choice([1, 2, 3, 4, 8]))
    if op == "verify":
        kw.update(new=_span(rng, 1, 16), vocab=_log(rng, 1000, 150000), sampled=rng.random() < 0.6)
    elif op == "append" and rng.random() < 0.5:                 # prompts
        kw.update(rope=rng.choice(sorted(ROPES)), ctx=_span(rng, 1, 60000), tree=False,
                  sequences=_log(rng, 1, 16), new=_span(rng, 1, 600), width=1)
    elif op in ("append", "accept"):
        kw.update(rope=rng.choice(sorted(ROPES)), ctx=_span(rng, 1, 4000), new=_span(rng, 1, 64))
        if op == "accept":
            kw.update(layers=rng.choice([1, 1, 2, 4]))
    else:
        kw.update(ctx=_span(rng, 1, 33000 if dtype == "bf16" else 1000), new=_span(rng, 1, 64))
    c = _case(op, **kw)
    # no more than the largest listed ones: keys times rows of a tree, tokens of a cache
    while c["sequences"] > 1 and (
            op == "tree" and c["sequences"] * c["ctx_hi"] > (264000 if dtype == "bf16" else 4000) or
            c["layers"] * c["sequences"] * (c["ctx_hi"] + c["new_hi"]) > 600000):
        c["sequences"] -= 1
    return c


# ---------------------------------------------------------------------------
# structure: lengths and trees follow from the case alone, values from the seed
# ---------------------------------------------------------------------------

class State:
    pass


def _plan(c):
    """[(tokens held, new rows, parents)] of a case's sequences."""
    r = random.Random(c["shape"])
    out = []
    for _ in range(c["sequences"]):
        ctx, n = r.randint(c["ctx_lo"], c["ctx_hi"]), r.randint(c["new_lo"], c["new_hi"])
        # a node's parent is one of the `width` nodes before it: several children, several depths
        par = [-1] + [max(0, i - 1 - r.randrange(c["width"])) for i in range(1, n)]
        out.append((ctx, n, par if c["tree"] else list(range(-1, n - 1))))
    return out


def _path(par, r):
    """A way down from the root, as verification leaves it."""
    path = [0]
    for i in range(1, len(par)):
        if par[i] == path[-1] and r.random() < 0.7:
            path.append(i)
    return path


def _depths(par):
    d = []
    for i, p in enumerate(par):
        d.append(0 if p < 0 else d[p] + 1)
    return d


def work(case):
    c = case
    Hq, Hkv, d, _ = HEADS[c["heads"]]
    es = 2 if c["dtype"] == "bf16" else 4
    plan = _plan(c)
    rows = sum(n for _, n, _ in plan)
    if c["op"] == "tree":
        byt = sum((ctx + n) * Hkv * d * 2 * es for ctx, n, _ in plan) + 2 * rows * Hq * d * es
        return {"bytes": byt, "flops": sum(4 * n * Hq * d * (ctx + n) for ctx, n, _ in plan)}
    if c["op"] == "verify":
        # a row of the target's probabilities (and of the draft's) a sequence, and the drafts' own
        per = 2 if c["sampled"] else 1
        return {"bytes": 4 * per * (c["vocab"] * len(plan) + rows) + 12 * rows, "flops": 0}
    byt = c["layers"] * rows * d * es * (2 * Hq + 4 * Hkv)
    if c["op"] == "accept":
        r = random.Random(c["shape"] + 1)
        moved = sum(i != j for _, _, p in plan for j, i in enumerate(_path(p, r)))
        byt = c["layers"] * d * es * (4 * Hkv * rows + 4 * Hkv * moved)
    return {"bytes": byt, "flops": 0}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _thetas(base, rot, scaling):
    """Frequencies of the pairs in 64 bits, scaled."""
    kind, f, orig, low, high, _ = scaling
    out = []
    for j in range(rot // 2):
        th = base ** (-2.0 * j / rot)
        if kind == "linear":
            th /= f
        elif kind == "llama3":
            turns = orig * th / (2 * math.pi)                  # of the original length
            mix = min(1.0, max(0.0, (turns - low) / (high - low)))
            th = (1 - mix) * th / f + mix * th
        elif kind == "yarn":
            at = lambda b: rot * math.log(orig / (b * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
            a, b = max(0, math.floor(at(high))), min(rot - 1, math.ceil(at(low)))
            ramp = min(1.0, max(0.0, (j - a) / max(b - a, 0.001)))
            th = (1 - ramp) * th + ramp * th / f
        out.append(th)
    return out


def _pages(c, plan, g, dev):
    """Pages of the sequences in random order: tables, and slot -> pool row."""
    bs = c["block_size"]
    need = [-(-(ctx + n) // bs) for ctx, n, _ in plan]
    total = sum(need) + 3
    perm = torch.randperm(total, generator=g, device=dev).int()
    tab = torch.full((len(plan), max(need)), -1, dtype=torch.int32, device=dev)
    at = 0
    for s, k in enumerate(need):
        tab[s, :k] = perm[at:at + k]
        at += k
    return tab, total


def _slots(s, of, pos, bs):
    """Pool rows of slots `pos` of sequences `of`."""
    return s.tables[of, pos // bs].long() * bs + pos % bs


def _prepare_cache(c, seed):
    s = State()
    s.c, dev = c, "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    Hq, Hkv, d, base = HEADS[c["heads"]]
    dt, bs = TORCH[c["dtype"]], c["block_size"]
    s.plan = plan = _plan(c)
    n = [x[1] for x in plan]
    R = sum(n)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    s.tables, s.n_pages = _pages(c, plan, g, dev)
    s.lens0, s.lens = i32([x[0] for x in plan]), i32([x[0] for x in plan])
    s.rows = i32([sum(n[:i]) for i in range(len(n) + 1)])
    s.parents = i32([p for x in plan for p in x[2]]) if c["tree"] else None
    make = lambda *z: torch.randn(*z, generator=g, device=dev).to(dt)  # noqa: E731
    s.of = torch.repeat_interleave(torch.arange(len(n), device=dev), s.rows.diff().long())
    s.node = torch.arange(R, device=dev) - s.rows[s.of].long()
    s.depth = torch.tensor([q for x in plan for q in _depths(x[2])], device=dev) if c["tree"] else s.node
    s.max_new = max(n)
    if c["op"] == "tree":
        s.kp, s.vp = make(s.n_pages, bs, Hkv, d), make(s.n_pages, bs, Hkv, d)
        s.Q = make(R, Hq, d) * 1.5
        s.O = torch.zeros_like(s.Q)
        # who is whose ancestor, padded to the largest tree
        N = s.max_new
        anc = torch.zeros(len(n), N, N, dtype=torch.bool)
        for k, (_, m, par) in enumerate(plan):
            for i in range(m):
                anc[k, i, i] = True
                if par[i] >= 0:
                    anc[k, i] |= anc[k, par[i]]
        s.anc = anc.to(dev)
    else:
        L = c["layers"]
        # one fused projection: query, key and value heads side by side in a row
        s.qkv = [make(R, Hq + 2 * Hkv, d) for _ in range(L)]
        s.pools = [(make(s.n_pages, bs, Hkv, d), make(s.n_pages, bs, Hkv, d)) for _ in range(L)]
        s.Qr = torch.zeros(R, Hq, d, dtype=dt, device=dev)
        layout, part, scaling = ROPES[c["rope"]]
        s.rot = int(d * part)
        s.theta = torch.tensor(_thetas(base, s.rot, scaling), dtype=torch.float64, device=dev)
        if c["op"] == "accept":
            r = random.Random(c["shape"] + 1)
            paths = [_path(x[2], r) for x in plan]
            s.count = i32([len(p) for p in paths])
            s.path = i32([p + [-1] * (s.max_new - len(p)) for p in paths])
            s.kept_of = torch.tensor([k for k, p in enumerate(paths) for _ in p], device=dev)
            s.kept_to = torch.tensor([i for p in paths for i in range(len(p))], device=dev)
            s.kept_from = torch.tensor([i for p in paths for i in p], device=dev)
    if own:
        _handles_cache(s, Hq, Hkv, d, base, bs)
    return s


def _handles_cache(s, Hq, Hkv, d, base, bs):
    from rag_kv_cache_rerotate_gb300 import fusekv as fk
    c = s.c
    kind = fk.FUSE_BF16 if c["dtype"] == "bf16" else fk.FUSE_F32
    s.desc = fk.layer_desc(Hq * d, Hq, Hkv, d, base, kind)
    s.seqs = fk.Sequences(s.tables, s.lens, s.rows, block_size=bs, n_pool_blocks=s.n_pages,
                          max_new=s.max_new)
    if c["op"] == "tree":
        s.ws = fk.alloc_tree_workspace(s.desc, s.seqs)
        return
    layout, _, (scaling, f, orig, low, high, mscale) = ROPES[c["rope"]]
    s.rope = fk.rope_desc(fk.FUSE_ROPE_INTERLEAVED if layout == "interleaved" else fk.FUSE_ROPE_HALF,
                          rot_dim=s.rot, mscale=mscale, factor=f, original_len=orig, low=low, high=high,
                          scaling={"none": fk.FUSE_ROPE_PLAIN, "linear": fk.FUSE_ROPE_LINEAR,
                                   "llama3": fk.FUSE_ROPE_LLAMA3, "yarn": fk.FUSE_ROPE_YARN}[scaling])
    s.handle = fk.PagePools([p[0] for p in s.pools], [p[1] for p in s.pools], kind, bs)
    s.ws = fk.alloc_cache_workspace()


def _prepare_verify(c, seed):
    s = State()
    s.c, dev = c, "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    s.plan = plan = _plan(c)
    n = [x[1] for x in plan]
    R, V = sum(n), c["vocab"]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    s.rows = i32([sum(n[:i]) for i in range(len(n) + 1)])
    s.parents = i32([p for x in plan for p in x[2]])
    s.max_new = max(n)
    # the drafter's distribution is the target's, blurred; few tokens hold most of it
    s.P = torch.empty(R, V, device=dev)
    s.Qd = torch.empty(R, V, device=dev)
    for a in range(0, R, 64):
        b = min(R, a + 64)
        z = 4.0 * torch.randn(b - a, V, generator=g, device=dev)
        s.P[a:b] = torch.softmax(z, -1)
        s.Qd[a:b] = torch.softmax(z + 0.8 * torch.randn(b - a, V, generator=g, device=dev), -1)
    # each draft comes from the row of its parent
    above = torch.tensor([o + max(p, 0) for o, x in zip(s.rows.tolist(), plan) for p in x[2]], device=dev)
    s.tokens = torch.empty(R, dtype=torch.int32, device=dev)
    for a in range(0, R, 64):
        b = min(R, a + 64)
        w = s.Qd[above[a:b]]
        if not c["sampled"]:
            w = w * w                                           # a search prefers the likely ones
        e = -torch.log(torch.rand(b - a, V, generator=g, device=dev).clamp_min(1e-30))
        s.tokens[a:b] = (w / e).argmax(-1).int()
    s.u = torch.rand(R, generator=g, device=dev)
    s.u_next = torch.rand(len(n), generator=g, device=dev)
    if not c["sampled"]:
        s.Qd = None
    s.path = torch.empty(len(n), s.max_new, dtype=torch.int32, device=dev)
    s.count = torch.empty(len(n), dtype=torch.int32, device=dev)
    s.next = torch.empty(len(n), dtype=torch.int32, device=dev)
    if own:
        from rag_kv_cache_rerotate_gb300 import fusekv as fk
        s.ws = fk.alloc_cache_workspace()
    return s


def prepare(case, seed):
    return _prepare_verify(case, seed) if case["op"] == "verify" else _prepare_cache(case, seed)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _turn(x, cos, sin, layout, rot):
    """Rows [n, heads, d] in 32 bits, their first `rot` channels rotated."""
    y, rest = x[..., :rot], x[..., rot:]
    if layout == "interleaved":
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, rest], -1)


def _plain_append(s):
    c = s.c
    Hq, Hkv, d, _ = HEADS[c["heads"]]
    layout, _, scaling = ROPES[c["rope"]]
    s.lens.copy_(s.lens0)
    pos = s.lens[s.of].double() + s.depth
    ang = pos[:, None] * s.theta
    cos, sin = ((scaling[5] * f).float()[:, None] for f in (ang.cos(), ang.sin()))
    at = _slots(s, s.of, s.lens[s.of].long() + s.node, c["block_size"])
    for x, (kp, vp) in zip(s.qkv, s.pools):
        x = x.float()
        if c["op"] == "append":
            s.Qr.copy_(_turn(x[:, :Hq], cos, sin, layout, s.rot))
        kp.view(-1, Hkv, d)[at] = _turn(x[:, Hq:Hq + Hkv], cos, sin, layout, s.rot).to(kp.dtype)
        vp.view(-1, Hkv, d)[at] = x[:, Hq + Hkv:].to(vp.dtype)
    if c["op"] == "append":
        return {"Q": s.Qr, "pools": s.pools}
    src = _slots(s, s.kept_of, s.lens[s.kept_of].long() + s.kept_from, c["block_size"])
    dst = _slots(s, s.kept_of, s.lens[s.kept_of].long() + s.kept_to, c["block_size"])
    for pair in s.pools:
        for p in pair:
            p.view(-1, Hkv, d)[dst] = p.view(-1, Hkv, d)[src]
    s.lens += s.count
    return {"pools": s.pools, "lens": s.lens}


def _plain_tree(s):
    c = s.c
    Hq, Hkv, d, _ = HEADS[c["heads"]]
    B, N, G = c["sequences"], s.max_new, Hq // Hkv
    T = max(x[0] + x[1] for x in s.plan)
    dev = s.Q.device
    t = torch.arange(T, device=dev)
    n = s.rows.diff().long()
    last = (s.lens.long() + n - 1)[:, None]
    at = _slots(s, torch.arange(B, device=dev)[:, None], torch.minimum(t[None], last), c["block_size"])
    k = s.kp.view(-1, Hkv, d)[at].float().permute(0, 2, 3, 1)                 # [B, Hkv, d, T]
    v = s.vp.view(-1, Hkv, d)[at].float().permute(0, 2, 1, 3)
    i = torch.minimum(torch.arange(N, device=dev)[None], n[:, None] - 1)
    q = s.Q[s.rows[:-1, None].long() + i].float().view(B, N, Hkv, G, d).permute(0, 2, 1, 3, 4)
    w = (q.reshape(B, Hkv, N * G, d) @ k / math.sqrt(d)).view(B, Hkv, N, G, T)
    rel = t[None] - s.lens[:, None].long()                                    # [B, T]
    own_key = s.anc.gather(2, rel.clamp(0, N - 1)[:, None].expand(B, N, T))
    seen = (rel < 0)[:, None] | (own_key & (rel < n[:, None])[:, None])       # [B, N, T]
    w = torch.where(seen[:, None, :, None], w, -math.inf)
    w = w.sub_(w.amax(-1, keepdim=True)).exp_()
    z = w.sum(-1, keepdim=True)
    o = (w.view(B, Hkv, N * G, T) @ v).view(B, Hkv, N, G, d) / z
    return o.permute(0, 2, 1, 3, 4).reshape(B, N, Hq, d)[s.of, s.node].to(s.Q.dtype)


def _plain_verify(s):
    """All sequences go through their nodes together; probabilities in 64 bits
    where sums and borders decide."""
    dev, B = s.P.device, s.c["sequences"]
    first, n = s.rows[:-1].long(), s.rows.diff().long()
    cur = torch.zeros(B, dtype=torch.long, device=dev)
    A, S = torch.zeros(B, dtype=torch.float64, device=dev), torch.ones(B, dtype=torch.float64, device=dev)
    gone = torch.zeros(B, s.P.shape[1], dtype=torch.bool, device=dev)
    me = torch.arange(B, device=dev)
    path, count = s.path.fill_(-1), s.count.fill_(1)
    path[:, 0] = 0
    for i in range(1, s.max_new):
        row = (first + i).clamp_max(s.P.shape[0] - 1)
        child = (i < n) & (s.parents[row] == cur)
        x, at = s.tokens[row].long(), first + cur
        p, u = s.P[at, x].double(), s.u[row].double()
        if s.Qd is not None:
            q = s.Qd[at, x].double()
            r = (p - A * q).clamp_min(0)
            yes = child & (r > 0) & (u * S * q < r)
        else:
            r = torch.where(gone[me, x], 0, p)
            yes = child & (r > 0) & (u * S < r)
        no = child & ~yes
        if s.Qd is not None:
            A = torch.where(no, A + S, A)
            left = (s.P[at].double() - A[:, None] * s.Qd[at].double()).clamp_min_(0).sum(-1)
            S = torch.where(no, left, S)
        else:
            gone[me, x] = gone[me, x] | no
            S = torch.where(no, S - r, S)
        # an accepted draft starts afresh with its own row
        A, S = torch.where(yes, 0, A), torch.where(yes, 1, S)
        gone &= ~yes[:, None]
        path[me, count.long().clamp_max(s.max_new - 1)] = torch.where(
            yes, i, path[me, count.long().clamp_max(s.max_new - 1)].long()).int()
        count += yes.int()
        cur = torch.where(yes, i, cur)
    p = s.P[first + cur].double()
    r = (p - A[:, None] * s.Qd[first + cur].double()).clamp_min(0) if s.Qd is not None else p.masked_fill(gone, 0)
    r = torch.where(r.sum(-1, keepdim=True) > 0, r, p)
    cum = r.cumsum(-1)
    nxt = (cum <= s.u_next.double()[:, None] * cum[:, -1:]).sum(-1)
    s.next.copy_(nxt)
    return {"path": path, "count": count, "next": s.next}


def run(state):
    s = state
    op = s.c["op"]
    if not own:
        return {"verify": _plain_verify, "tree": _plain_tree}.get(op, _plain_append)(s)
    from rag_kv_cache_rerotate_gb300 import fusekv as fk
    if op == "verify":
        fk.verify_tree(s.rows, s.parents, s.tokens, s.P, s.Qd, s.u, s.u_next, s.path, s.count, s.next, s.ws)
        return {"path": s.path, "count": s.count, "next": s.next}
    if op == "tree":
        fk.attend_tree(s.desc, s.seqs, s.parents, s.Q, s.kp, s.vp, s.O, s.ws)
        return s.O
    Hq, Hkv = s.desc.n_q_heads, s.desc.n_kv_heads
    s.lens.copy_(s.lens0)
    for x, (kp, vp) in zip(s.qkv, s.pools):
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        if op == "append":
            fk.cache_append(s.desc, s.rope, s.seqs, s.parents, q, k, v, s.Qr, None, kp, vp, s.ws)
        else:
            fk.cache_append(s.desc, s.rope, s.seqs, s.parents, None, k, v, None, None, kp, vp, s.ws)
    if op == "append":
        return {"Q": s.Qr, "pools": s.pools}
    fk.cache_keep(s.desc, s.handle, s.seqs, s.path, s.count, s.ws)
    return {"pools": s.pools, "lens": s.lens}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_cache(c, seed):
    s = _prepare_cache(c, seed)
    Hq, Hkv, d, _ = HEADS[c["heads"]]
    layout, _, scaling = ROPES[c["rope"]]
    f, bs = torch.float64, c["block_size"]
    tab = s.tables.tolist()
    Q = torch.empty(s.Qr.shape, dtype=f, device="cuda")
    pools = [(k.to(f), v.to(f)) for k, v in s.pools]
    r = random.Random(c["shape"] + 1)
    lens, row = [], 0
    for q, (ctx, n, par) in enumerate(s.plan):
        deep = _depths(par) if c["tree"] else range(n)
        at = lambda i: (torch.tensor([tab[q][(ctx + j) // bs] for j in i], device="cuda"),  # noqa: E731
                        torch.tensor([(ctx + j) % bs for j in i], device="cuda"))
        page, off = at(range(n))
        # a rotation is a product with a number of modulus mscale
        pos = torch.tensor([ctx + j for j in deep], dtype=f, device="cuda")
        z = torch.polar(torch.full((n, s.rot // 2), scaling[5], dtype=f, device="cuda"), torch.outer(pos, s.theta))
        for x, (kp, vp) in zip(s.qkv, pools):
            x = x[row:row + n].to(f)
            y = x[:, :Hq + Hkv, :s.rot]
            if layout == "interleaved":
                w = torch.view_as_complex(y.reshape(n, Hq + Hkv, -1, 2).contiguous()) * z[:, None]
                w = torch.view_as_real(w).reshape(n, Hq + Hkv, -1)
            else:
                w = torch.complex(y[..., :s.rot // 2], y[..., s.rot // 2:]) * z[:, None]
                w = torch.cat([w.real, w.imag], -1)
            x[:, :Hq + Hkv, :s.rot] = w
            Q[row:row + n] = x[:, :Hq]
            kp[page, off], vp[page, off] = x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        row += n
        if c["op"] == "accept":
            path = _path(par, r)
            (a, b), (e, g) = at(path), at(range(len(path)))
            for pair in pools:
                for p in pair:
                    p[e, g] = p[a, b]
            lens.append(ctx + len(path))
    if c["op"] == "append":
        return {"Q": Q, "pools": pools}
    return {"pools": pools, "lens": torch.tensor(lens, dtype=torch.int32, device="cuda")}


def _exact_tree(c, seed):
    s = _prepare_cache(c, seed)
    Hq, Hkv, d, _ = HEADS[c["heads"]]
    f, bs = torch.float64, c["block_size"]
    if work(c)["flops"] > 5e12:                                 # over 20 seconds in 64 bits
        return None
    out = torch.empty(s.Q.shape, dtype=f, device="cuda")
    row = 0
    for q, (ctx, n, par) in enumerate(s.plan):
        t = torch.arange(ctx + n, device="cuda")
        page = s.tables[q].long()[torch.div(t, bs, rounding_mode="floor")]
        seen = torch.zeros(n, ctx + n, dtype=torch.bool)
        seen[:, :ctx] = True
        for i in range(n):
            j = i
            while j >= 0:
                seen[i, ctx + j] = True
                j = par[j]
        seen = seen.cuda()
        for h in range(Hkv):
            k, v = s.kp[page, t % bs, h].to(f), s.vp[page, t % bs, h].to(f)
            for e in range(h * Hq // Hkv, (h + 1) * Hq // Hkv):
                z = s.Q[row:row + n, e].to(f) @ k.T * d ** -0.5
                out[row:row + n, e] = torch.softmax(z.masked_fill(~seen, -math.inf), -1) @ v
        row += n
    return out


def _exact_verify(c, seed):
    """One sequence after another, the residuals taken in turn as they are defined."""
    s = _prepare_verify(c, seed)
    path, count, nxt = [], [], []
    tok, u, un = s.tokens.tolist(), s.u.double().tolist(), s.u_next.double().tolist()
    for b, (o, (_, n, par)) in enumerate(zip(s.rows.tolist(), s.plan)):
        way = [0]
        p = s.P[o].double()
        r, S = p, 1.0
        for i in range(1, n):
            if par[i] != way[-1]:
                continue
            x = tok[o + i]
            q = torch.zeros_like(p) if s.Qd is None else s.Qd[o + way[-1]].double()
            if s.Qd is None:
                q[x] = 1.0
            rx, qx = r[x].item(), q[x].item()
            if rx > 0 and u[o + i] * S * qx < rx:
                way.append(i)
                p = s.P[o + i].double()
                r, S = p, 1.0
            elif s.Qd is None:
                r = r.clone()
                r[x] = 0
                S -= rx
            else:
                r = torch.relu(r - S * q)
                S = r.sum().item()
        if r.sum().item() <= 0:
            r = p
        cum = torch.cumsum(r, 0)
        nxt.append(int(torch.searchsorted(cum, cum[-1] * un[b], right=True)))
        path.append(way + [-1] * (s.max_new - len(way)))
        count.append(len(way))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    return {"path": i32(path), "count": i32(count), "next": i32(nxt)}


def exact(case, seed):
    if case["op"] == "tree":
        return _exact_tree(case, seed)
    return _exact_verify(case, seed) if case["op"] == "verify" else _exact_cache(case, seed)
