"""Plain statements, in fp64 numpy, of the operators of a speculative step over
a paged cache (rotate and append, attention of a tree, verification, keeping the
accepted rows), with the bounds that the GPU tests hold the kernels to, and the
device buffers of a test case."""

from __future__ import annotations

import dataclasses
import math
from typing import Optional, Sequence

import numpy as np
import torch

from rag_kv_cache_rerotate_gb300 import fusekv as fk

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
KIND = {"bf16": fk.FUSE_BF16, "f32": fk.FUSE_F32}
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def i32(x):
    return torch.tensor(np.asarray(x, dtype=np.int32), device="cuda")


def random_tree(n, width, rng):
    """Parents: each node follows one of the `width` nodes before it."""
    return [-1] + [max(0, i - 1 - int(rng.integers(width))) for i in range(1, n)] if n else []


def depths(parents):
    d = []
    for p in parents:
        d.append(0 if p < 0 else d[p] + 1)
    return d


def ancestors(parents):
    """seen[i, j]: j is i or one of its ancestors."""
    n = len(parents)
    seen = np.zeros((n, n), bool)
    for i, p in enumerate(parents):
        if p >= 0:
            seen[i] |= seen[p]
        seen[i, i] = True
    return seen


@dataclasses.dataclass
class StepCase:
    lens: Sequence[int]                    # held tokens
    new: Sequence[int]                     # new rows
    heads: tuple = (8, 2, 128)             # query heads, KV heads, head dim
    dtype: str = "bf16"
    block_size: int = 16
    width: int = 3                         # 0: parents are not given
    front: int = 0                         # rows in front of the first sequence's
    behind: int = 0                        # rows behind the last one's
    pages: int = 3                         # pages that no sequence has
    scale: float = 1.0                     # of the queries
    base: float = 1e4
    seed: int = 0


class Step:
    """Device buffers of a case."""

    def __init__(self, c: StepCase):
        self.c = c
        self.Hq, self.Hkv, self.d = Hq, Hkv, d = c.heads
        rng = np.random.default_rng(c.seed)
        bs = c.block_size
        need = [-(-(a + n) // bs) for a, n in zip(c.lens, c.new)]
        self.n_pages = sum(need) + c.pages
        perm = rng.permutation(self.n_pages)
        tab = np.full((len(need), max([1] + need)), -7, np.int32)
        at = 0
        for s, k in enumerate(need):
            tab[s, :k] = perm[at:at + k]
            at += k
        self.tab = tab
        self.starts = [c.front + sum(c.new[:i]) for i in range(len(need) + 1)]
        self.n_rows = self.starts[-1] + c.behind
        self.trees = [random_tree(n, c.width, rng) if c.width else list(range(-1, n - 1)) for n in c.new]
        par = [-1] * c.front + [p for t in self.trees for p in t] + [-1] * c.behind
        self.parents = i32(par) if c.width else None
        self.tables, self.lens, self.rows = i32(tab), i32(c.lens), i32(self.starts)
        dt = DT[c.dtype]
        make = lambda *z: torch.from_numpy(rng.standard_normal(z).astype(np.float32)).to(dt).cuda()  # noqa: E731
        self.kp, self.vp = make(self.n_pages, bs, Hkv, d), make(self.n_pages, bs, Hkv, d)
        self.qkv = make(self.n_rows, Hq + 2 * Hkv, d)
        self.Q, self.K, self.V = self.qkv[:, :Hq], self.qkv[:, Hq:Hq + Hkv], self.qkv[:, Hq + Hkv:]
        self.Qr = (make(self.n_rows, Hq, d) * c.scale).contiguous()
        self.O = make(self.n_rows, Hq, d)
        self.desc = fk.layer_desc(64, Hq, Hkv, d, c.base, KIND[c.dtype])
        self.seqs = fk.Sequences(self.tables, self.lens, self.rows, bs, self.n_pages,
                                 max([1] + list(c.new)))
        self.ws = fk.alloc_tree_workspace(self.desc, self.seqs)

    def slots(self, s, tokens):
        """(page, row of the page) of tokens of sequence s."""
        t = np.asarray(tokens, dtype=np.int64)
        return self.tab[s, t // self.c.block_size].astype(np.int64), t % self.c.block_size

    def attend(self, stream=None):
        fk.attend_tree(self.desc, self.seqs, self.parents, self.Qr, self.kp, self.vp, self.O, self.ws, stream)
        return self.O

    def tree_reference(self, rows=None, lens: Optional[Sequence[int]] = None):
        """(O, tolerance) of attend_tree in fp64, NaN outside the sequences' rows.

        With A = sum p |v| and S = max sum |q k| / sqrt(d), a score is off by at
        most e = S (d + 16) 2^-23 + S 2^-21 (fp32 products and sums); a weight by
        2 e relative (numerator and sum) plus its rounding where it meets the
        values: 2^-8 in bf16 layers, 2^-21 in fp32 ones (exp2 and the joins'
        factors).  Sums of n terms in fp32 add n 2^-24 A.  One rounding at the end."""
        c = self.c
        O, tol = np.full(self.O.shape, np.nan), np.full(self.O.shape, np.nan)
        K, V, Q = f64(self.kp), f64(self.vp), f64(self.Qr)
        for s, (held, n) in enumerate(zip(c.lens if lens is None else lens, c.new)):
            if n == 0:
                continue
            page, at = self.slots(s, range(held + n))
            seen = np.concatenate([np.ones((n, held), bool), ancestors(self.trees[s])], 1)
            for i in range(n):
                r = self.starts[s] + i
                if rows is not None and r not in rows:
                    continue
                pg, a = page[seen[i]], at[seen[i]]
                for h in range(self.Hq):
                    g = h * self.Hkv // self.Hq
                    k, v = K[pg, a, g], V[pg, a, g]
                    x = k @ Q[r, h] / math.sqrt(self.d)
                    p = np.exp(x - x.max())
                    p /= p.sum()
                    o, A = p @ v, p @ np.abs(v)
                    S = np.max(np.abs(k) @ np.abs(Q[r, h])) / math.sqrt(self.d)
                    e = S * ((self.d + 16) * 2.0 ** -23 + 2.0 ** -21)
                    w = 2.0 ** -8 if c.dtype == "bf16" else 2.0 ** -21
                    O[r, h] = o
                    tol[r, h] = HALF_STEP[c.dtype] * np.abs(o) + (w + 2 * e + len(k) * 2.0 ** -24) * A
        return O, tol


def check_close(got, want, tol, what=""):
    """Every element of `want` that is a number, within its tolerance."""
    have = ~np.isnan(want)
    err = np.abs(got - want)
    bad = have & ~(err <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {have.sum()} elements off; worst "
                           f"{np.nanmax(np.where(bad, err / tol, 0)):.3g} of the tolerance")


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------

def thetas(base, rot, scaling=fk.FUSE_ROPE_PLAIN, factor=1.0, original_len=0, low=0.0, high=0.0):
    out = []
    for m in range(rot // 2):
        th = base ** (-2.0 * m / rot)
        if scaling == fk.FUSE_ROPE_LINEAR:
            th = th / factor
        elif scaling == fk.FUSE_ROPE_LLAMA3:
            wave = 2 * math.pi / th
            if wave > original_len / low:
                th = th / factor
            elif wave >= original_len / high:
                c = (original_len / wave - low) / (high - low)
                th = (1 - c) * th / factor + c * th
        elif scaling == fk.FUSE_ROPE_YARN:
            t = lambda x: rot * math.log(original_len / (x * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
            a, b = max(0, math.floor(t(high))), min(rot - 1, math.ceil(t(low)))
            r = min(1.0, max(0.0, (m - a) / max(b - a, 0.001)))
            th = th * (1 - r) + th / factor * r
        out.append(th)
    return np.array(out)


def rotate(x, pos, theta, layout, mscale, dtype):
    """(rotated, tolerance) of rows x [n, heads, d] at positions pos [n].

    Cosine and sine are off by at most 2^-21: the argument's rounding (pi 2^-25),
    sincospi's (2^-23), mscale's two (2^-23); products and their difference add
    2^-23 of |x0| + |x1|, the result's rounding half a step."""
    rot = 2 * len(theta)
    y, tol = x.copy(), np.zeros_like(x)
    ang = np.outer(pos, theta)
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    lo, hi = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == fk.FUSE_ROPE_HALF else \
        (slice(0, rot, 2), slice(1, rot, 2))
    a, b = x[..., lo], x[..., hi]
    y[..., lo], y[..., hi] = mscale * (a * c - b * s), mscale * (b * c + a * s)
    both = mscale * (np.abs(a) + np.abs(b)) * (2.0 ** -21 + 2.0 ** -23)
    tol[..., lo] = both + HALF_STEP[dtype] * np.abs(y[..., lo])
    tol[..., hi] = both + HALF_STEP[dtype] * np.abs(y[..., hi])
    return y, tol


# ---------------------------------------------------------------------------
# verification
# ---------------------------------------------------------------------------

def verify(parents, tokens, P, Q, u, u_next):
    """One sequence: (path, next token), the remainders taken in turn."""
    path, r, S = [0], P[0], 1.0
    for i in range(1, len(parents)):
        if parents[i] != path[-1]:
            continue
        x = tokens[i]
        q = Q[path[-1]] if Q is not None else np.eye(1, len(r), x)[0]
        if r[x] > 0 and u[i] * S * q[x] < r[x]:
            path.append(i)
            r, S = P[i], 1.0
        elif Q is not None:
            r = np.maximum(r - S * q, 0)
            S = r.sum()
        else:
            S -= r[x]
            r = np.where(np.arange(len(r)) == x, 0, r)
    if r.sum() <= 0:
        r = P[path[-1]]
    cum = np.cumsum(r)
    return path, int(np.argmax(cum > u_next * cum[-1]))
