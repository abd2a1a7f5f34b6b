"""Workloads of the cache operators: attention of new tokens over chunk caches
held in 4 or 8 bits, causal attention over whole packed prompts, and the
upkeep of a paged cache (copy, fork, compact, free).

Each workload has a plain form (elementary torch operations in 32 bits,
rounded once at the end) and, with ``own`` set, the calls that a user of
libfusekv makes.  ``exact`` states the results in 64 bits.
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


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _flat(c):
    """Spans (low, high) as two plain values of the case."""
    out = {}
    for k, v in c.items():
        out.update({k + "_lo": v[0], k + "_hi": v[1]} if isinstance(v, tuple) else {k: v})
    return out


def _attend(**kw):
    c = dict(op="attend", heads="qwen3_8b", dtype="bf16", storage="u4", layout="contiguous",
             requests=1, chunks=(8, 8), chunk_len=(512, 512), query=(64, 64), ratio=0.15, new=1,
             block_size=16, shape=0)
    c.update(kw)
    return _flat(c)


def _prompt(**kw):
    c = dict(op="prompt", heads="qwen3_8b", dtype="bf16", sequences=1, length=(512, 512), shape=0)
    c.update(kw)
    return _flat(c)


def _pages(op, **kw):
    c = dict(op=op, heads="llama3_8b", dtype="bf16", layers=1, blocks=1024, block_size=16,
             sequences=8, length=(256, 2048), fan=2, moves=64, shape=0)
    c.update(kw)
    return _flat(c)


def listed():
    return [
        # one user's next token over a Qwen3-8B layer's eight retrieved chunks: latency counts
        _attend(name="next token, 8 x 512, u4"),
        # a batch of 16 ragged requests whose chunks sit in a paged pool of 16-token blocks
        _attend(name="next tokens, 16 paged, u4", heads="llama3_8b", layout="paged", requests=16,
                chunks=(4, 16), chunk_len=(128, 512), query=(32, 128), ratio=0.20, shape=3),
        # eight long-context requests of the Llama-3-70B shape: bandwidth counts
        _attend(name="next tokens, 8 x 33k, u4", heads="llama3_70b", requests=8, chunks=(32, 32),
                chunk_len=(1024, 1024), query=(256, 256), ratio=0.10, shape=4),
        # four drafted tokens verified at once over int8 codes of odd lengths
        _attend(name="4 drafted tokens, u8", storage="u8", requests=4, chunks=(5, 9),
                chunk_len=(77, 701), query=(17, 99), ratio=0.12, new=4, shape=5),
        # the fp32 layer of the small configuration, ragged
        _attend(name="next token, f32, u4", heads="tiny", dtype="f32", requests=2, chunks=(3, 4),
                chunk_len=(33, 64), query=(16, 16), ratio=0.30, shape=6),
        # retrieved chunks, each attending to itself alone, to build their caches
        _prompt(name="chunk prefill, ragged", heads="llama3_8b", sequences=16, length=(128, 512),
                shape=7),
        # a whole prompt without reuse: 20 chunks of 512 and the query
        _prompt(name="whole prompt, 10368", length=(10368, 10368), shape=8),
        # two long prompts of odd lengths, 64 query heads
        _prompt(name="two prompts, 8 to 16k", heads="llama3_70b", sequences=2,
                length=(8191, 16411), shape=9),
        # short prompts with a head dimension of 64
        _prompt(name="short prompts, d 64", heads="narrow", sequences=9, length=(1, 333), shape=10),
        # pages moved within every layer's pool, as a scheduler orders
        _pages("copy", name="copy 64 pages, 16 layers", layers=16, blocks=256, moves=64, shape=11),
        # parallel samples branch off running sequences, then are dropped
        _pages("fork", name="fork 12 x 3 and drop", blocks=4096, sequences=12, length=(65, 4001),
               fan=3, shape=12),
        # a fragmented pool is packed to its front
        _pages("compact", name="compact 4096 blocks", layers=2, blocks=4096, sequences=20,
               length=(100, 3000), fan=2, shape=13),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _span(rng, lo, hi):
    a, b = sorted((_log(rng, lo, hi), _log(rng, lo, hi)))
    return (a, b)


def draw(rng):
    shape = rng.randrange(1 << 30)
    op = rng.choice(["attend", "attend", "attend", "prompt", "prompt", "copy", "fork", "compact"])
    if op == "attend":
        dtype = rng.choice(["bf16"] * 5 + ["f32"])
        storage = rng.choice(["u4", "u4", "u4", "u8", dtype])
        c = _attend(heads=rng.choice(sorted(HEADS)) if dtype == "bf16" else "tiny", dtype=dtype,
                    storage=storage, layout=rng.choice(["contiguous", "paged"]),
                    requests=_log(rng, 1, 16), chunks=_span(rng, 1, 32),
                    chunk_len=_span(rng, 16, 1024), query=_span(rng, 8, 256),
                    ratio=round(rng.uniform(0.0, 0.3), 3), new=rng.choice([1, 1, 1, 2, 4, 8]),
                    block_size=rng.choice([16, 16, 32, 24]), shape=shape)
        limit = 200000 if dtype == "bf16" else 20000
        while c["requests"] > 1 and c["requests"] * c["chunks_hi"] * c["chunk_len_hi"] > limit:
            c["requests"] -= 1
        return c
    if op == "prompt":
        dtype = rng.choice(["bf16"] * 7 + ["f32"])
        c = _prompt(heads=rng.choice(sorted(HEADS)) if dtype == "bf16" else "tiny", dtype=dtype,
                    sequences=_log(rng, 1, 16),
                    length=_span(rng, 1, 12000 if dtype == "bf16" else 700), shape=shape)
        while c["sequences"] > 1 and c["sequences"] * c["length_hi"] ** 2 > 2.0e8:
            c["sequences"] -= 1
        return c
    c = _pages(op, heads=rng.choice(["qwen3_8b", "narrow", "tiny"]), dtype=rng.choice(["bf16", "f32"]),
               layers=_log(rng, 1, 8), blocks=_log(rng, 64, 4096), block_size=rng.choice([16, 32, 24]),
               fan=rng.choice([1, 2, 3, 4]), shape=shape)
    while c["layers"] > 1 and c["layers"] * c["blocks"] * c["block_size"] > 65536:
        c["layers"] -= 1
    room = c["blocks"] * c["block_size"] // 2
    c["length_lo"], c["length_hi"] = _span(rng, 1, max(2, room // 8))
    c["sequences"] = max(1, min(_log(rng, 1, 24), room // (c["length_hi"] + c["block_size"])))
    c["moves"] = _log(rng, 1, c["blocks"] // 2)
    return c


# ---------------------------------------------------------------------------
# structure: lengths follow from the case alone, values from the seed
# ---------------------------------------------------------------------------

def _requests(c):
    """[(chunk lengths, query tokens, selected tokens)] of an attend case."""
    r = random.Random(c["shape"])
    out = []
    for _ in range(c["requests"]):
        lens = [r.randint(c["chunk_len_lo"], c["chunk_len_hi"]) for _ in range(r.randint(c["chunks_lo"], c["chunks_hi"]))]
        n = sum(lens)
        out.append((lens, max(c["new"], r.randint(c["query_lo"], c["query_hi"])), int(c["ratio"] * n + 1e-9)))
    return out


def _lengths(c):
    r = random.Random(c["shape"])
    return [r.randint(c["length_lo"], c["length_hi"]) for _ in range(c["sequences"])]


def _bits(storage):
    return {"u4": 4, "u8": 8, "bf16": 16, "f32": 32}[storage]


def work(case):
    c = case
    Hq, Hkv, d, _ = HEADS[c["heads"]]
    es = _bits(c["dtype"]) // 8
    if c["op"] == "attend":
        quant = c["storage"] in ("u4", "u8")
        byt = flo = 0
        for lens, nq, k in _requests(c):
            n = sum(lens)
            # selected tokens are read from the side rows instead of the codes
            byt += (n - k) * Hkv * (2 * d * _bits(c["storage"]) // 8 + (4 if quant else 0))
            byt += len(lens) * Hkv * d * 4 if quant else 0
            byt += (k + nq) * Hkv * 2 * d * es + 2 * c["new"] * Hq * d * es + 4 * k
            flo += 4 * c["new"] * Hq * d * (n + nq)
        return {"bytes": byt, "flops": flo}
    if c["op"] == "prompt":
        T = sum(_lengths(c))
        return {"bytes": T * d * es * (2 * Hq + 2 * Hkv),
                "flops": sum(2 * Hq * d * n * (n + 1) for n in _lengths(c))}
    page = 2 * c["block_size"] * Hkv * d * es * c["layers"]
    if c["op"] == "copy":
        return {"bytes": 2 * page * c["moves"] + 8 * c["moves"], "flops": 0}
    nb = [-(-n // c["block_size"]) for n in _lengths(c)]
    if c["op"] == "fork":
        part = sum(1 for n in _lengths(c) if n % c["block_size"]) * c["fan"]
        return {"bytes": 2 * page * part + 4 * (2 * c["blocks"] + 6 * c["fan"] * sum(nb)), "flops": 0}
    live = min(1.0, sum(nb) / c["blocks"])
    return {"bytes": int(2 * page * c["blocks"] * live * (1 - live)) + 4 * (2 * c["blocks"] + 2 * sum(nb)),
            "flops": 0}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

class State:
    pass


def _groups(lens, device):
    return torch.repeat_interleave(torch.arange(len(lens), device=device),
                                   torch.tensor(lens, device=device))


def _kivi(x, bits, group):
    """Codes, scale and zero over the groups that `group` (x -> reduced min, max) forms."""
    mn, mx = group(x)
    L = (1 << bits) - 1
    span = mx - mn
    q = torch.where(span > 0, torch.round((x - mn) / torch.where(span > 0, span, 1) * L), 0)
    return q.to(torch.uint8), (span / L).half(), mn.half()


def _store(x, storage, chunk_of, n_chunks, per_channel):
    """One side (keys or values) of the chunk caches in their storage form."""
    if storage in TORCH:
        return x.to(TORCH[storage]), None, None
    bits = _bits(storage)
    if per_channel:
        idx = chunk_of[:, None, None].expand_as(x)
        lo = torch.zeros(n_chunks, *x.shape[1:], device=x.device).scatter_reduce_(0, idx, x, "amin", include_self=False)
        hi = torch.zeros(n_chunks, *x.shape[1:], device=x.device).scatter_reduce_(0, idx, x, "amax", include_self=False)
        q, _, _ = _kivi(x, bits, lambda _: (lo[chunk_of], hi[chunk_of]))
        s, z = ((hi - lo) / ((1 << bits) - 1)).half(), lo.half()
    else:
        q, s, z = _kivi(x, bits, lambda v: (v.amin(-1, keepdim=True), v.amax(-1, keepdim=True)))
        s, z = s[..., 0], z[..., 0]
    if bits == 4:
        q = q[..., 0::2] | (q[..., 1::2] << 4)
    return q.contiguous(), s.contiguous(), z.contiguous()


def _prepare_attend(c, seed):
    s = State()
    s.c = c
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    Hq, Hkv, d, base = HEADS[c["heads"]]
    dt = TORCH[c["dtype"]]
    req = _requests(c)
    lens = [n for r in req for n in r[0]]
    nc, T = len(lens), sum(lens)
    randn = lambda *z: torch.randn(*z, generator=g, device=dev)  # noqa: E731
    s.lens, s.n_ctx = lens, [sum(r[0]) for r in req]
    s.n_query, s.k = [r[1] for r in req], [r[2] for r in req]
    # keys have channels of their own mean and spread; queries point at some of them
    spread = torch.exp(0.4 * randn(1, Hkv, d))
    K = randn(T, Hkv, d) * spread + 0.5 * randn(1, Hkv, d)
    V = randn(T, Hkv, d) * torch.exp(0.3 * randn(T, 1, 1))
    s.chunk_of = _groups(lens, dev)
    kq, s.ks, s.kz = _store(K, c["storage"], s.chunk_of, nc, True)
    vq, vs, vz = _store(V, c["storage"], s.chunk_of, nc, False)
    del K, V
    bs = c["block_size"]
    if c["layout"] == "paged":
        blocks = [-(-n // bs) for n in lens]
        perm = torch.randperm(sum(blocks), generator=g, device=dev)
        first = torch.tensor([sum(blocks[:i]) for i in range(nc)], device=dev)
        start = torch.tensor([sum(lens[:i]) for i in range(nc)], device=dev)
        r = torch.arange(T, device=dev) - start[s.chunk_of]
        s.slot = perm[first[s.chunk_of] + r // bs] * bs + r % bs
        s.table, s.table0, s.n_blocks = perm.int(), [sum(blocks[:i]) for i in range(nc)], sum(blocks)

        def pool(x):
            p = torch.zeros(s.n_blocks * bs, *x.shape[1:], dtype=x.dtype, device=dev)
            p[s.slot] = x
            return p
        kq, vq = pool(kq), pool(vq)
        vs, vz = (pool(vs), pool(vz)) if vs is not None else (None, None)
    else:
        s.slot = torch.arange(T, device=dev)
    s.K, s.V, s.vs, s.vz = kq, vq, vs, vz
    R = [k + q for k, q in zip(s.k, s.n_query)]
    s.Ks, s.Vs = randn(sum(R), Hkv, d).to(dt), randn(sum(R), Hkv, d).to(dt)
    s.Q = (1.5 * randn(len(req) * c["new"], Hq, d)).to(dt)
    s.idx = torch.cat([torch.randperm(n, generator=g, device=dev)[:k].sort().values
                       for n, k in zip(s.n_ctx, s.k)]).int()
    # where each request's tokens lie, padded to the longest request
    pos, ctx0, row0, pads, sides, offs = [], 0, 0, [], [], []
    for (ls, _, _), n, rr in zip(req, s.n_ctx, R):
        pads.append(ctx0 + torch.arange(max(s.n_ctx), device=dev).clamp(max=n - 1))
        sides.append(row0 + torch.arange(max(R), device=dev).clamp(max=rr - 1))
        ctx0, row0 = ctx0 + n, row0 + rr
        o = 0
        for n_i in ls:
            offs.append(o)
            o += n_i
    s.pad, s.side = torch.stack(pads), torch.stack(sides)
    s.off = torch.tensor(offs, device=dev)
    s.sel_req = _groups(s.k, dev)
    t = lambda x: torch.tensor(x, device=dev)  # noqa: E731
    s.t_ctx, s.t_side = t(s.n_ctx), t([r - c["new"] for r in R])
    s.theta = torch.tensor([base ** (-2.0 * j / d) for j in range(d // 2)], dtype=torch.float64, device=dev)
    s.O = torch.zeros_like(s.Q)
    s.offs = offs
    if own:
        _handles_attend(s, d, Hq, Hkv, base, bs)
    return s


def _handles_attend(s, d, Hq, Hkv, base, bs):
    from rag_kv_cache_rerotate_gb300 import fusekv as fk
    c = s.c
    kind = {"u4": fk.FUSE_U4_ASYM, "u8": fk.FUSE_U8_ASYM, "bf16": fk.FUSE_BF16, "f32": fk.FUSE_F32}
    s.desc = fk.layer_desc(Hq * d, Hq, Hkv, d, base, kind[c["dtype"]])
    plan = fk.plan_requests(s.n_ctx, s.n_query, 0.0)
    s.reqs = fk.requests_with_k(plan, s.k)
    paged, quant = c["layout"] == "paged", s.ks is not None
    rb = s.K[0].numel() * s.K.element_size()
    entries, start, row = [], 0, 0
    chunk = 0
    for r, (ls, nq, _) in enumerate(_requests(c)):
        for n in ls:
            e = fk.Chunk()
            e.k, e.v = s.K.data_ptr(), s.V.data_ptr()
            if paged:
                e.block_table = s.table.data_ptr() + 4 * s.table0[chunk]
            else:
                e.k += start * rb
                e.v += start * rb
            if quant:
                at = 0 if paged else start * Hkv * 2
                e.k_scale, e.k_zero = s.ks[chunk].data_ptr(), s.kz[chunk].data_ptr()
                e.v_scale, e.v_zero = s.vs.data_ptr() + at, s.vz.data_ptr() + at
            e.dst_row, e.pos, e.len = row + s.offs[chunk], s.offs[chunk], n
            entries.append(e)
            start, chunk = start + n, chunk + 1
        row += s.n_ctx[r] + nq
    s.chunks = fk.ChunkTable(entries, fk.FUSE_KV_PAGED if paged else fk.FUSE_KV_CONTIGUOUS,
                             kind[c["storage"]], block_size=bs if paged else 0,
                             n_pool_blocks=s.n_blocks if paged else 0,
                             keep=[s.K, s.V, s.ks, s.kz, s.vs, s.vz])
    s.ws = fk.alloc_attend_workspace(s.desc, s.chunks, s.reqs, c["new"])


def _prepare_prompt(c, seed):
    s = State()
    s.c = c
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    Hq, Hkv, d, base = HEADS[c["heads"]]
    s.n = _lengths(c)
    T, top = sum(s.n), max(s.n)
    make = lambda h, a: (a * torch.randn(T, h, d, generator=g, device=dev)).to(TORCH[c["dtype"]])  # noqa: E731
    s.Q, s.K, s.V = make(Hq, 1.5), make(Hkv, 1.0), make(Hkv, 1.0)
    s.O = torch.zeros_like(s.Q)
    start = torch.tensor([sum(s.n[:i]) for i in range(len(s.n))], device=dev)
    t_n = torch.tensor(s.n, device=dev)
    s.pad = start[:, None] + torch.minimum(torch.arange(top, device=dev)[None], t_n[:, None] - 1)
    seq = _groups(s.n, dev)
    s.back = seq * top + torch.arange(T, device=dev) - start[seq]
    if own:
        from rag_kv_cache_rerotate_gb300 import fusekv as fk
        s.desc = fk.layer_desc(Hq * d, Hq, Hkv, d, base,
                               fk.FUSE_BF16 if c["dtype"] == "bf16" else fk.FUSE_F32)
        s.reqs = fk.plan_requests(s.n, [0] * len(s.n), 0.0)
        s.ws = fk.alloc_workspace(s.desc, s.reqs)
    return s


def _prepare_pages(c, seed):
    s = State()
    s.c = c
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    _, Hkv, d, base = HEADS[c["heads"]]
    bs, NB = c["block_size"], c["blocks"]
    s.pool = torch.randn(c["layers"], 2, NB, bs, Hkv, d, generator=g, device=dev).to(TORCH[c["dtype"]])
    perm = torch.randperm(NB, generator=g, device=dev).int()
    if c["op"] == "copy":
        s.src, s.dst = perm[:c["moves"]], perm[NB - c["moves"]:]
        s.moves = torch.cat([torch.tensor([c["moves"], 0], device=dev).int(),
                             torch.stack([s.src, s.dst], 1).reshape(-1)])
    else:
        s.n = _lengths(c)
        s.blocks = [-(-n // bs) for n in s.n]
        total = sum(s.blocks)
        s.tab = perm[:total].clone()
        s.refs = torch.zeros(NB, dtype=torch.int32, device=dev)
        s.refs[s.tab.long()] = 1
        s.t0 = [sum(s.blocks[:i]) for i in range(len(s.blocks))]
        if c["op"] == "fork":
            at = torch.arange(total, device=dev)
            s.take = at.repeat(c["fan"])                      # dst entry -> src entry
            s.out = torch.empty(total * c["fan"], dtype=torch.int32, device=dev)
            part = [f * total + a + b - 1 for f in range(c["fan"])
                    for a, b, n in zip(s.t0, s.blocks, s.n) if n % bs]
            s.part = torch.tensor(part, dtype=torch.long, device=dev)
            whole = torch.ones(total * c["fan"], dtype=torch.bool, device=dev)
            whole[s.part] = False
            s.whole = whole.nonzero()[:, 0]
        else:                                                   # some sequences share their pages
            extra = list(range(0, len(s.n), 2)) if c["fan"] > 1 else []
            s.shared = extra
            idx = [torch.arange(s.t0[i], s.t0[i] + s.blocks[i], device=dev) for i in extra]
            s.tab = torch.cat([s.tab] + [s.tab[i] for i in idx])
            s.refs.zero_().index_add_(0, s.tab.long(), torch.ones_like(s.tab))
        s.tab0, s.refs0 = s.tab.clone(), s.refs.clone()
    if own:
        _handles_pages(s, Hkv, d, base, bs, NB)
    return s


def _handles_pages(s, Hkv, d, base, bs, NB):
    from rag_kv_cache_rerotate_gb300 import fusekv as fk
    c = s.c
    kind = fk.FUSE_BF16 if c["dtype"] == "bf16" else fk.FUSE_F32
    s.desc = fk.layer_desc(Hkv * d, Hkv, Hkv, d, base, kind)
    s.pools = fk.PagePools([p[0] for p in s.pool], [p[1] for p in s.pool], kind, bs)
    if c["op"] == "copy":
        s.ws = fk.alloc_pages_workspace(None)
        return

    def table(flat, starts, lens):
        entries = []
        for a, n in zip(starts, lens):
            e = fk.Chunk()
            e.k, e.v = s.pool[0, 0].data_ptr(), s.pool[0, 1].data_ptr()
            e.block_table, e.len = flat.data_ptr() + 4 * a, n
            entries.append(e)
        return fk.ChunkTable(entries, fk.FUSE_KV_PAGED, kind, block_size=bs, n_pool_blocks=NB,
                             keep=[flat])
    total = sum(s.blocks)
    if c["op"] == "fork":
        s.src = table(s.tab, s.t0 * c["fan"], s.n * c["fan"])
        s.dst = table(s.out, [f * total + a for f in range(c["fan"]) for a in s.t0], s.n * c["fan"])
        s.moves = fk.alloc_moves(len(s.n) * c["fan"])
        s.ws = fk.alloc_pages_workspace(s.src)
    else:
        more, at = [], total
        for i in s.shared:
            more.append(at)
            at += s.blocks[i]
        s.seqs = table(s.tab, s.t0 + more, s.n + [s.n[i] for i in s.shared])
        s.moves = fk.alloc_moves(NB // 2)
        s.ws = fk.alloc_pages_workspace(s.seqs)


def prepare(case, seed):
    if case["op"] == "attend":
        return _prepare_attend(case, seed)
    if case["op"] == "prompt":
        return _prepare_prompt(case, seed)
    return _prepare_pages(case, seed)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _values(codes, storage):
    """Stored elements as 32-bit numbers (codes of 4 bits unpacked)."""
    if storage == "u4":
        return torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()
    return codes.float()


def _plain_attend(s):
    c = s.c
    Hq, Hkv, d, _ = HEADS[c["heads"]]
    U, R, G = c["new"], c["requests"], Hq // Hkv
    at = s.slot[s.pad]                                          # [R, T] storage row of each token
    of = s.chunk_of[s.pad]
    k, v = _values(s.K[at], c["storage"]), _values(s.V[at], c["storage"])
    if s.ks is not None:
        k = s.kz.float()[of] + k * s.ks.float()[of]
        v = s.vz[at].float()[..., None] + v * s.vs[at].float()[..., None]
    ang = (s.off[of].double()[..., None] * s.theta)[:, :, None]
    cos, sin = ang.cos().float(), ang.sin().float()
    a, b = k[..., :d // 2], k[..., d // 2:]
    k = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    k, v = torch.cat([k, s.Ks[s.side].float()], 1), torch.cat([v, s.Vs[s.side].float()], 1)
    # context tokens that are there and not selected; side rows up to each new token
    T, S = s.pad.shape[1], s.side.shape[1]
    ctx = torch.arange(T, device=k.device)[None] < s.t_ctx[:, None]
    ctx[s.sel_req, s.idx.long()] = False
    u = torch.arange(U, device=k.device)
    side = torch.arange(S, device=k.device)[None, None] <= (s.t_side[:, None] + u[None])[..., None]
    seen = torch.cat([ctx[:, None].expand(R, U, T), side], -1)[:, None, :, None]   # [R,1,U,1,T+S]
    q = s.Q.float().view(R, U, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(R, Hkv, U * G, d)
    w = (q @ k.permute(0, 2, 3, 1) / math.sqrt(d)).view(R, Hkv, U, G, T + S)
    w = torch.where(seen, w, -math.inf)
    w = torch.exp(w - w.amax(-1, keepdim=True))
    w = (w / w.sum(-1, keepdim=True)).view(R, Hkv, U * G, T + S)
    o = (w @ v.permute(0, 2, 1, 3)).view(R, Hkv, U, G, d).permute(0, 2, 1, 3, 4)
    return o.reshape(R * U, Hq, d).to(s.Q.dtype)


def _plain_prompt(s):
    Hq, Hkv, d, _ = HEADS[s.c["heads"]]
    R, T = s.pad.shape
    G = Hq // Hkv
    q = s.Q[s.pad].float().view(R, T, Hkv, G, d).permute(0, 2, 3, 1, 4)      # [R, Hkv, G, T, d]
    k = s.K[s.pad].float().permute(0, 2, 3, 1)[:, :, None]                   # [R, Hkv, 1, d, T]
    v = s.V[s.pad].float().permute(0, 2, 1, 3)[:, :, None]
    rows = max(1, min(T, (1 << 30) // (R * Hq * T)))                          # scores of 4 GB at most
    o = torch.empty(R, Hkv, G, T, d, device=q.device)
    for t in range(0, T, rows):
        e = min(T, t + rows)
        w = q[..., t:e, :] @ k[..., :e] / math.sqrt(d)
        late = torch.arange(e, device=q.device)[None] > torch.arange(t, e, device=q.device)[:, None]
        w = w.masked_fill_(late, -math.inf)
        w = w.sub_(w.amax(-1, keepdim=True)).exp_()
        o[..., t:e, :] = (w @ v[..., :e, :]) / w.sum(-1, keepdim=True)
    o = o.permute(0, 3, 1, 2, 4).reshape(R * T, Hq, d)
    return o[s.back].to(s.Q.dtype)


def _plain_pages(s):
    c = s.c
    if c["op"] == "copy":
        s.pool[:, :, s.dst.long()] = s.pool[:, :, s.src.long()]
        return {"pool": s.pool}
    if c["op"] == "fork":
        new = (s.refs == 0).nonzero()[:s.part.numel(), 0]
        old = s.tab[s.take[s.part]].long()
        out = s.tab[s.take]
        out[s.part] = new.int()
        one = torch.ones_like(out)
        s.refs.index_add_(0, out[s.whole].long(), one[:s.whole.numel()])
        s.refs[new] = 1
        s.pool[:, :, new] = s.pool[:, :, old]
        forked = s.refs.clone()
        s.refs.index_add_(0, out.long(), -one)                  # the branches are dropped
        return {"tables": out, "forked": forked, "refs": s.refs, "pool": s.pool}
    refs, tab = s.refs.copy_(s.refs0), s.tab.copy_(s.tab0)
    live = refs > 0
    n = live.sum()
    ids = torch.arange(refs.numel(), device=refs.device)
    hole, tail = (~live & (ids < n)).nonzero()[:, 0], (live & (ids >= n)).nonzero()[:, 0]
    to = ids.clone()
    to[tail] = hole
    s.pool[:, :, hole] = s.pool[:, :, tail]
    refs[hole] = refs[tail]
    refs[tail] = 0
    tab.copy_(to[tab.long()])
    return {"tables": tab, "refs": refs, "live": n.int().view(1), "pool": s.pool}


def run(state):
    s = state
    op = s.c["op"]
    if not own:
        return {"attend": _plain_attend, "prompt": _plain_prompt}.get(op, _plain_pages)(s)
    from rag_kv_cache_rerotate_gb300 import fusekv as fk
    if op == "attend":
        fk.attend_chunks(s.desc, s.chunks, s.reqs, s.c["new"], s.Q, s.idx, s.Ks, s.Vs, s.O, s.ws)
        return s.O
    if op == "prompt":
        fk.attend_prompt(s.desc, s.reqs, s.Q, s.K, s.V, s.O, s.ws)
        return s.O
    if op == "copy":
        fk.pages_copy(s.desc, s.pools, s.moves, s.ws)
        return {"pool": s.pool}
    if op == "fork":
        fk.pages_fork(s.src, s.dst, s.refs, s.moves, s.ws)
        fk.pages_copy(s.desc, s.pools, s.moves, s.ws)
        forked = s.refs.clone()
        fk.pages_free(s.dst, s.refs, s.ws)
        return {"tables": s.out, "forked": forked, "refs": s.refs, "pool": s.pool}
    s.refs.copy_(s.refs0)
    s.tab.copy_(s.tab0)
    fk.pages_compact(s.seqs, s.refs, s.moves, s.ws)
    fk.pages_copy(s.desc, s.pools, s.moves, s.ws)
    return {"tables": s.tab, "refs": s.refs, "live": s.moves[1:2], "pool": s.pool}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _attention64(q, k, v, scale):
    """Rows of softmax(q k^T) v; q [u, h, d], k and v [t, h, d]."""
    z = torch.einsum("uhd,thd->hut", q, k) * scale
    p = torch.softmax(z, -1)
    return torch.einsum("hut,thd->uhd", p, v)


def _exact_attend(c, seed):
    s = _prepare_attend(c, seed)
    Hq, Hkv, d, base = HEADS[c["heads"]]
    f = torch.float64
    U = c["new"]
    out = torch.empty(c["requests"] * U, Hq, d, dtype=f, device="cuda")
    t = chunk = sel = row = 0
    for r, (lens, nq, k_r) in enumerate(_requests(c)):
        keys, vals = [], []
        for n, o in zip(lens, _starts(lens)):
            at = s.slot[t:t + n]
            parts = []
            for st in (s.K, s.V):
                x = st[at]
                if c["storage"] == "u4":
                    y = torch.empty(*x.shape[:-1], d, dtype=f, device=x.device)
                    y[..., 0::2], y[..., 1::2] = (x % 16).to(f), (x // 16).to(f)
                    x = y
                parts.append(x.to(f))
            kk, vv = parts
            if s.ks is not None:
                kk = kk * s.ks[chunk].to(f) + s.kz[chunk].to(f)
                vv = vv * s.vs[at].to(f).unsqueeze(-1) + s.vz[at].to(f).unsqueeze(-1)
            turn = torch.polar(torch.ones(d // 2, dtype=f, device=kk.device),
                               o * torch.pow(torch.tensor(base, dtype=f, device=kk.device),
                                             -torch.arange(0, d, 2, dtype=f, device=kk.device) / d))
            z = torch.complex(kk[..., :d // 2], kk[..., d // 2:]) * turn
            keys.append(torch.cat([z.real, z.imag], -1))
            vals.append(vv)
            t, chunk = t + n, chunk + 1
        keys, vals = torch.cat(keys), torch.cat(vals)
        keep = torch.ones(len(keys), dtype=torch.bool, device=keys.device)
        keep[s.idx[sel:sel + k_r].long()] = False
        keys, vals = keys[keep], vals[keep]
        for u in range(U):
            m = k_r + nq - U + u + 1
            kk = torch.cat([keys, s.Ks[row:row + m].to(f)]).repeat_interleave(Hq // Hkv, 1)
            vv = torch.cat([vals, s.Vs[row:row + m].to(f)]).repeat_interleave(Hq // Hkv, 1)
            i = r * U + u
            out[i:i + 1] = _attention64(s.Q[i:i + 1].to(f), kk, vv, d ** -0.5)
        sel, row = sel + k_r, row + k_r + nq
    return out


def _starts(lens):
    return [sum(lens[:i]) for i in range(len(lens))]


def _exact_prompt(c, seed):
    s = _prepare_prompt(c, seed)
    Hq, Hkv, d, _ = HEADS[c["heads"]]
    if work(c)["flops"] > 5e12:                                 # over 20 seconds in 64 bits
        return None
    f = torch.float64
    out = torch.empty(s.Q.shape, dtype=f, device="cuda")
    for a, n in zip(_starts(s.n), s.n):
        for h in range(Hq):
            q, k, v = (x[a:a + n, i].to(f) for x, i in ((s.Q, h), (s.K, h * Hkv // Hq), (s.V, h * Hkv // Hq)))
            for b in range(0, n, 4096):
                e = min(n, b + 4096)
                z = (q[b:e] @ k[:e].T) * d ** -0.5
                z.masked_fill_(torch.ones(e - b, e, dtype=torch.bool, device="cuda").triu_(1 + b), -math.inf)
                out[a + b:a + e, h] = torch.softmax(z, -1) @ v[:e]
    return out


def _exact_pages(c, seed):
    """Page by page on the host's lists, then the pool's pages moved as listed."""
    s = _prepare_pages(c, seed)
    if c["op"] == "copy":
        moves = list(zip(s.src.tolist(), s.dst.tolist()))
        return {"pool": _moved(s.pool, moves)}
    refs, tab, bs = s.refs.tolist(), s.tab.tolist(), c["block_size"]
    moves = []
    if c["op"] == "fork":
        free = iter([b for b, r in enumerate(refs) if r == 0])
        out, before = [], list(refs)
        for _ in range(c["fan"]):
            for a, n in zip(s.t0, s.n):
                for j in range(-(-n // bs)):
                    b = tab[a + j]
                    if (j + 1) * bs > n:
                        new = next(free)
                        moves.append((b, new))
                        b = new
                    refs[b] += 1
                    out.append(b)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        return {"tables": i32(out), "forked": i32(refs), "refs": i32(before), "pool": _moved(s.pool, moves)}
    live = [b for b, r in enumerate(refs) if r > 0]
    n = len(live)
    holes = [b for b in range(n) if refs[b] == 0]
    moves = list(zip([b for b in live if b >= n], holes))
    to = dict(moves)
    for a, b in moves:
        refs[b], refs[a] = refs[a], 0
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    return {"tables": i32([to.get(b, b) for b in tab]), "refs": i32(refs), "live": i32([n]),
            "pool": _moved(s.pool, moves)}


def _moved(pool, moves):
    p = pool.double()
    for a, b in moves:
        p[:, :, b] = pool[:, :, a]
    return p


def exact(case, seed):
    if case["op"] == "attend":
        return _exact_attend(case, seed)
    if case["op"] == "prompt":
        return _exact_prompt(case, seed)
    return _exact_pages(case, seed)
