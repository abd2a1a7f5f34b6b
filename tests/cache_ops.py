"""Plain statements, in fp64 numpy, of the cache operators (attention over
chunk caches, packed-prompt attention, page upkeep), with the bounds that the
GPU tests hold the kernels to, and the device buffers of a test case."""

from __future__ import annotations

import dataclasses
from typing import List, Optional, Sequence

import numpy as np
import torch

from oracle import fusion as orc
from rag_kv_cache_rerotate_gb300 import fusekv as fk

KIND = {"u4": fk.FUSE_U4_ASYM, "u8": fk.FUSE_U8_ASYM, "bf16": fk.FUSE_BF16, "f32": fk.FUSE_F32}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def attention(q, k, v, mag_k=None, mag_v=None):
    """One query [d] over keys and values [t, d]: the output, and for the error
    bound sum p |v| per channel and the largest sum |q k| / sqrt(d)."""
    d = q.shape[-1]
    s = k @ q / np.sqrt(d)
    p = np.exp(s - s.max())
    p /= p.sum()
    mk = np.abs(k) if mag_k is None else mag_k
    mv = np.abs(v) if mag_v is None else mag_v
    return p @ v, p @ mv, float(np.max(mk @ np.abs(q)) / np.sqrt(d))


# ---------------------------------------------------------------------------
# attention over chunk caches
# ---------------------------------------------------------------------------

@dataclasses.dataclass
class AttendCase:
    lens: List[List[int]]                 # chunk lengths per request
    n_query: List[int]
    k: List[int]                          # selected tokens per request
    heads: tuple = (8, 2, 128)            # query heads, KV heads, head dim
    dtype: str = "bf16"
    storage: str = "u4"
    paged: bool = False
    block_size: int = 16
    new: int = 1
    base: float = 1e6
    gap: int = 0                          # unused side rows behind each request
    pos_shift: int = 0                    # added to every chunk's angle offset
    spare_blocks: int = 0                 # pool pages before the used ones
    # stairs of a chunk's tokens: (tokens of a step, steps until they start over,
    # what a step adds to a score, to the logarithm (base 2) of the values)
    rise: Optional[tuple] = None
    seed: int = 0


class Attend:
    """Device buffers of a case and its reference."""

    def __init__(self, c: AttendCase):
        self.c = c
        Hq, Hkv, d = c.heads
        rng = np.random.default_rng(c.seed)
        n_ctx = [sum(x) for x in c.lens]
        self.n_ctx = n_ctx
        flat = [n for x in c.lens for n in x]
        T = sum(flat)
        f32 = lambda *s: rng.standard_normal(s).astype(np.float32).astype(np.float64)  # noqa: E731
        K = f32(T, Hkv, d) * np.exp(0.4 * f32(1, Hkv, d)) + 0.5 * f32(1, Hkv, d)
        V = f32(T, Hkv, d)
        if c.rise:
            # by the first channel of the slowest pair, which an offset hardly turns
            each, steps, score, value = c.rise
            at = (np.concatenate([np.arange(n) for n in flat]) // each % steps)[:, None]
            K[..., d // 2 - 1] = score * np.sqrt(d) / 4.0 * at
            V = (V * 2.0 ** (value * at)[..., None]).astype(np.float32).astype(np.float64)
        bits = {"u4": 4, "u8": 8}.get(c.storage)
        keys, vals, mk, mv = [], [], [], []
        codes = {"K": [], "V": [], "ks": [], "kz": [], "vs": [], "vz": []}
        t = 0
        for n in flat:
            k, v = K[t:t + n], V[t:t + n]
            t += n
            if bits and n:
                qk, sk, zk = orc.kivi_quantize_key(k, bits)
                qv, sv, zv = orc.kivi_quantize_value(v, bits)
                sk, zk, sv, zv = (x.astype(np.float16) for x in (sk, zk, sv, zv))
                w = lambda x: x.astype(np.float64)  # noqa: E731
                keys.append(w(zk) + qk * w(sk))
                vals.append(w(zv)[..., None] + qv * w(sv)[..., None])
                mk.append(np.abs(w(zk)) + np.abs(qk * w(sk)))
                mv.append(np.abs(w(zv))[..., None] + np.abs(qv * w(sv)[..., None]))
                pack = (lambda q: q[..., 0::2] | (q[..., 1::2] << 4)) if bits == 4 else (lambda q: q)
                for name, x in (("K", pack(qk.astype(np.uint8))), ("V", pack(qv.astype(np.uint8))),
                                ("ks", sk), ("kz", zk), ("vs", sv), ("vz", zv)):
                    codes[name].append(x)
            elif bits:
                for lst in (keys, vals, mk, mv):
                    lst.append(np.zeros((0, Hkv, d)))
                codes["ks"].append(np.zeros((Hkv, d), np.float16))
                codes["kz"].append(np.zeros((Hkv, d), np.float16))
            else:
                kt = torch.from_numpy(k).to(DT[c.storage])
                vt = torch.from_numpy(v).to(DT[c.storage])
                codes["K"].append(kt)
                codes["V"].append(vt)
                keys.append(f64(kt))
                vals.append(f64(vt))
                mk.append(np.abs(keys[-1]))
                mv.append(np.abs(vals[-1]))
        self.keys, self.vals, self.mk, self.mv = keys, vals, mk, mv
        to = lambda x: torch.from_numpy(np.ascontiguousarray(x))  # noqa: E731
        dk = d // 2 if bits == 4 else d
        if bits:
            one = lambda name, *s: to(np.concatenate(codes[name]) if codes[name] else np.zeros(s, np.uint8))  # noqa: E731
            Kst, Vst = one("K", 0, Hkv, dk), one("V", 0, Hkv, dk)
            self.ks = to(np.stack(codes["ks"])) if flat else torch.zeros(0, Hkv, d).half()
            self.kz = to(np.stack(codes["kz"])) if flat else torch.zeros(0, Hkv, d).half()
            vs = to(np.concatenate(codes["vs"])) if codes["vs"] else torch.zeros(0, Hkv).half()
            vz = to(np.concatenate(codes["vz"])) if codes["vz"] else torch.zeros(0, Hkv).half()
            self.ks, self.kz = self.ks.cuda(), self.kz.cuda()
        else:
            z = torch.zeros(0, Hkv, d, dtype=DT[c.storage])
            Kst, Vst = torch.cat(codes["K"] + [z]), torch.cat(codes["V"] + [z])
            self.ks = self.kz = vs = vz = None
        bs = c.block_size
        self.tables: List[torch.Tensor] = []
        if c.paged:
            blocks = [-(-n // bs) for n in flat]
            nb = sum(blocks) + c.spare_blocks
            perm = c.spare_blocks + rng.permutation(sum(blocks))
            fill = 0 if bits else float("nan")              # unused rows of a layer-type pool

            def pool(x):
                p = torch.empty(nb, bs, *x.shape[1:], dtype=x.dtype, device="cuda")
                if c.spare_blocks < 1000:
                    p.fill_(fill if x.dtype != torch.float16 else float("nan"))
                return p
            self.K, self.V = pool(Kst), pool(Vst)
            self.vs, self.vz = (pool(vs), pool(vz)) if bits else (None, None)
            t = b0 = 0
            for n, b in zip(flat, blocks):
                ids = perm[b0:b0 + b]
                for j, page in enumerate(ids):
                    m = min(bs, n - j * bs)
                    a = t + j * bs
                    for dst, src in ((self.K, Kst), (self.V, Vst)) + (((self.vs, vs), (self.vz, vz)) if bits else ()):
                        dst[page, :m] = src[a:a + m].cuda()
                self.tables.append(torch.from_numpy(ids.astype(np.int32)).cuda())
                t, b0 = t + n, b0 + b
            self.n_blocks = nb
        else:
            self.K, self.V = Kst.cuda(), Vst.cuda()
            self.vs, self.vz = (vs.cuda(), vz.cuda()) if bits else (None, None)
        # requests and their side rows
        self.desc = fk.layer_desc(64, Hq, Hkv, d, c.base, KIND[c.dtype])
        reqs, row, sel, out = [], 0, 0, 0
        for n, q, k in zip(n_ctx, c.n_query, c.k):
            reqs.append(fk.Request(row, 0, sel, out, n, q, k, 0))
            row, sel, out = row + n + q, sel + k, out + k + q + c.gap
        self.reqs = fk.RequestTable(reqs)
        self.Ks = torch.full((out, Hkv, d), float("nan"), dtype=DT[c.dtype], device="cuda")
        self.Vs = torch.full((out, Hkv, d), float("nan"), dtype=DT[c.dtype], device="cuda")
        for r in reqs:
            n = r.k + r.n_query
            for dst in (self.Ks, self.Vs):
                dst[r.out0:r.out0 + n] = torch.from_numpy(f32(n, Hkv, d)).to(DT[c.dtype]).cuda()
        self.idx_list = [np.sort(rng.permutation(n)[:k]) for n, k in zip(n_ctx, c.k)]
        self.idx = torch.from_numpy(np.concatenate(self.idx_list).astype(np.int32)).cuda()
        Q = 1.5 * f32(len(reqs) * c.new, Hq, d)
        if c.rise:
            Q[..., d // 2 - 1], Q[..., d - 1] = 4.0, 0.0
        self.Q = torch.from_numpy(Q).to(DT[c.dtype]).cuda()
        self.O = torch.full_like(self.Q, 7.0)
        self.chunks = self.table()
        self.ws = fk.alloc_attend_workspace(self.desc, self.chunks, self.reqs, c.new)

    def offsets(self):
        return [sum(x[:i]) + self.c.pos_shift for x in self.c.lens for i in range(len(x))]

    def table(self, tables: Optional[Sequence[torch.Tensor]] = None):
        c = self.c
        Hq, Hkv, d = c.heads
        tables = self.tables if tables is None else tables
        rb = self.K[0].numel() * self.K.element_size()
        entries, start, i = [], 0, 0
        offs = self.offsets()
        for r, lens in enumerate(c.lens):
            for n in lens:
                e = fk.Chunk()
                if n or not c.paged:
                    e.k = self.K.data_ptr() + (0 if c.paged else start * rb)
                    e.v = self.V.data_ptr() + (0 if c.paged else start * rb)
                if c.paged and n:
                    e.block_table = tables[i].data_ptr()
                if self.ks is not None and n:
                    at = 0 if c.paged else start * Hkv * 2
                    e.k_scale, e.k_zero = self.ks[i].data_ptr(), self.kz[i].data_ptr()
                    e.v_scale, e.v_zero = self.vs.data_ptr() + at, self.vz.data_ptr() + at
                e.dst_row = self.reqs[r].row0 + offs[i] - c.pos_shift
                e.pos, e.len = offs[i], n
                entries.append(e)
                start, i = start + n, i + 1
        return fk.ChunkTable(entries, fk.FUSE_KV_PAGED if c.paged else fk.FUSE_KV_CONTIGUOUS,
                             KIND[c.storage], block_size=c.block_size if c.paged else 0,
                             n_pool_blocks=self.n_blocks if c.paged else 0,
                             keep=[self.K, self.V, self.ks, self.kz, self.vs, self.vz, list(tables)])

    def run(self, stream=None):
        fk.attend_chunks(self.desc, self.chunks, self.reqs, self.c.new, self.Q, self.idx, self.Ks,
                         self.Vs, self.O, self.ws, stream)
        return self.O

    def segments(self, n_new=None):
        """Segments that the plan has cut the call's keys into."""
        Hq, Hkv, d = self.c.heads
        per = Hkv * -(-(Hq // Hkv) * (n_new or self.c.new) // 8)
        size = fk.attend_workspace_size(self.desc, self.chunks, self.reqs, n_new or self.c.new)
        return (size - 256) // (per * 8 * (8 + 4 * d))

    def reference(self, rows=None, unseen=()):
        """(O, tolerance) in fp64 for every output row, or for the (row, head)
        pairs of `rows`, the others NaN; `unseen`: side rows (request-local)
        that have no weight.

        With A = sum p |v| and S = max sum |q k| / sqrt(d) (magnitudes of a
        code's zero and scaled part added), a score is off by at most
        e = S * ((d + 16) 2^-23 + 2^-20): fp32 products and sums, q in two
        16-bit parts, and the angle (2^-25 of a turn); a weight's relative
        error is 2 e (numerator and sum), plus its rounding where it meets the
        values: 2^-11 in fp16 beside codes of a bf16 layer; 2^-15 where it is
        kept in two bf16 parts; in a fp32 layer 2^-21.  Sums of n terms in
        fp32 add n 2^-24 A at most.  The output is rounded once."""
        c = self.c
        Hq, Hkv, d = c.heads
        offs = self.offsets()
        O = np.full((len(c.lens) * c.new, Hq, d), np.nan if rows is not None else 0.0)
        tol = np.zeros_like(O)
        Ks, Vs, Q = f64(self.Ks), f64(self.Vs), f64(self.Q)
        i = 0
        for r, lens in enumerate(c.lens):
            R = self.reqs[r]
            keep = np.ones(R.n_ctx, bool)
            keep[self.idx_list[r]] = False
            ch = range(i, i + len(lens))
            i += len(lens)
            z = np.zeros((0, Hkv, d))
            # R^pos q'k: the magnitudes of a rotated pair are at most their sum
            rot = [orc.rope_rotate(self.keys[j], offs[j], c.base) for j in ch]
            mag = [np.concatenate([m[..., :d // 2] + m[..., d // 2:]] * 2, -1) for m in (self.mk[j] for j in ch)]
            k = np.concatenate([z] + rot)[keep]
            mk = np.concatenate([z] + mag)[keep]
            v = np.concatenate([z] + [self.vals[j] for j in ch])[keep]
            mv = np.concatenate([z] + [self.mv[j] for j in ch])[keep]
            for u in range(c.new):
                m = R.k + R.n_query - c.new + u + 1
                seen = R.out0 + np.setdiff1d(np.arange(m), np.asarray(unseen, int))
                sk, sv = Ks[seen], Vs[seen]
                kk, vv = np.concatenate([k, sk]), np.concatenate([v, sv])
                ma, mb = np.concatenate([mk, np.abs(sk)]), np.concatenate([mv, np.abs(sv)])
                for h in range(Hq):
                    if rows is not None and (r * c.new + u, h) not in rows:
                        continue
                    g = h * Hkv // Hq
                    o, A, S = attention(Q[r * c.new + u, h], kk[:, g], vv[:, g], ma[:, g], mb[:, g])
                    n = len(kk)
                    e = S * ((d + 16) * 2.0 ** -23 + 2.0 ** -20)
                    if c.dtype == "bf16":
                        t = 2.0 ** -8 * np.abs(o) + (2.0 ** -11 + 2 * e + n * 2.0 ** -24) * A
                    else:
                        t = 2.0 ** -24 * np.abs(o) + (2.0 ** -21 + 2 * e + n * 2.0 ** -24) * A
                    O[r * c.new + u, h], tol[r * c.new + u, h] = o, t
        return O, tol


# ---------------------------------------------------------------------------
# packed prompts
# ---------------------------------------------------------------------------

def prompt_reference(Q, K, V, spans, dtype):
    """(O, tolerance) of causal attention inside the row ranges `spans`; rows
    outside are NaN.  Bounds as for the chunk caches, with the weights of a
    bf16 layer rounded to bf16 (2^-8) where they meet the values."""
    Q, K, V = f64(Q), f64(K), f64(V)
    Hq, Hkv, d = Q.shape[1], K.shape[1], Q.shape[2]
    O, tol = np.full(Q.shape, np.nan), np.full(Q.shape, np.nan)
    for a, n in [x for x in spans if x[1] > 0]:
        for h in range(Hq):
            g = h * Hkv // Hq
            k, v = K[a:a + n, g], V[a:a + n, g]
            s = Q[a:a + n, h] @ k.T / np.sqrt(d)
            s[np.triu_indices(n, 1)] = -np.inf
            p = np.exp(s - s.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            o, A = p @ v, p @ np.abs(v)
            S = np.max(np.tril(np.abs(Q[a:a + n, h]) @ np.abs(k).T), axis=1, keepdims=True) / np.sqrt(d)
            e = S * ((d + 16) * 2.0 ** -23 + 2.0 ** -21)
            w, r = (2.0 ** -8, 2.0 ** -8) if dtype == "bf16" else (2.0 ** -21, 2.0 ** -24)
            O[a:a + n, h] = o
            tol[a:a + n, h] = r * np.abs(o) + (w + 2 * e + n * 2.0 ** -24) * A
    return O, tol


# ---------------------------------------------------------------------------
# pages
# ---------------------------------------------------------------------------

def fork_reference(tables, lens, refs, bs):
    """(dst tables, refs, moves) or None when the free pages do not suffice."""
    refs = list(refs)
    free = [b for b, r in enumerate(refs) if r == 0]
    need = sum(1 for n in lens if n % bs)
    if need > len(free):
        return None
    out, moves = [], []
    for t, n in zip(tables, lens):
        d = []
        for j in range(-(-n // bs)):
            b = int(t[j])
            if (j + 1) * bs > n:
                new = free.pop(0)
                moves.append((b, new))
                b = new
            refs[b] += 1
            d.append(b)
        out.append(d)
    return out, refs, moves


def compact_reference(tables, refs):
    """(tables, refs, moves, live)."""
    refs = list(refs)
    live = [b for b, r in enumerate(refs) if r > 0]
    n = len(live)
    moves = list(zip([b for b in live if b >= n], [b for b in range(n) if refs[b] == 0]))
    to = dict(moves)
    for a, b in moves:
        refs[b], refs[a] = refs[a], 0
    return [[to.get(int(b), int(b)) for b in t] for t in tables], refs, moves, n


def page_table(tables, lens, bs, n_blocks, k=4096, v=4096):
    """A paged chunk table over int32 device tensors."""
    entries = []
    for t, n in zip(tables, lens):
        e = fk.Chunk()
        e.k, e.v, e.len = k, v, n
        if n:
            e.block_table = t.data_ptr()
        entries.append(e)
    return fk.ChunkTable(entries, fk.FUSE_KV_PAGED, fk.FUSE_BF16, block_size=bs,
                         n_pool_blocks=n_blocks, keep=list(tables))
