"""Verification of drafted tokens next to its borders, on the GPU against exact
rational arithmetic: drafts and next tokens that a sum of 24 bits would decide
the other way, and remainders that are nearly nothing."""

from fractions import Fraction

import numpy as np
import pytest
import torch

from rag_kv_cache_rerotate_gb300 import fusekv as fk

from step_ops import i32

pytestmark = pytest.mark.gpu


def exact(parents, tokens, P, Q, u, u_next):
    """One sequence: (path, next token), without a rounding."""
    f = lambda row: {x: Fraction(float(v)) for x, v in enumerate(row) if v}  # noqa: E731
    path, r, S = [0], f(P[0]), Fraction(1)
    for i in range(1, len(parents)):
        if parents[i] != path[-1]:
            continue
        x, q = tokens[i], f(Q[path[-1]])
        rx = r.get(x, 0)
        if rx > 0 and Fraction(float(u[i])) * S * q.get(x, 0) < rx:
            path.append(i)
            r, S = f(P[i]), Fraction(1)
        else:
            r = {y: v - S * q.get(y, 0) for y, v in r.items() if v > S * q.get(y, 0)}
            S = sum(r.values(), Fraction(0))
    if not r:
        r = f(P[path[-1]])
    t, cum = Fraction(float(u_next)) * sum(r.values()), Fraction(0)
    for x in sorted(r):
        cum += r[x]
        if cum > t:
            return path, x


def run(parents, tokens, P, Q, u, u_next):
    """Sequences of equal trees: P, Q [n, nodes, vocab], tokens, u [n, nodes]."""
    n, k, vocab = P.shape
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()  # noqa: E731
    path, count, nxt = (torch.full(z, -9, dtype=torch.int32, device="cuda") for z in ((n, k), (n,), (n,)))
    ws = fk.alloc_cache_workspace()
    fk.verify_tree(i32(np.arange(n + 1) * k), i32(np.tile(parents, n)), i32(np.reshape(tokens, -1)),
                   t(P).view(n * k, vocab), t(Q).view(n * k, vocab) if Q is not None else None, t(u).view(-1), t(u_next),
                   path, count, nxt, ws)
    fk.check_errors(ws)
    return [p[:c] for p, c in zip(path.tolist(), count.tolist())], nxt.tolist()


@pytest.mark.parametrize("vocab", [4, 3001])
@pytest.mark.parametrize("children", [1, 24, 25, 26, 40, 63])
def test_star_of_refused_tokens(children, vocab):
    # each refusal halves what is left of the other tokens, whose probabilities stay in proportion
    n = 8
    P, Q = np.zeros((n, children + 1, vocab)), np.zeros((n, children + 1, vocab))
    at = [0, 1, vocab // 2, vocab - 1]
    P[..., at], Q[..., at] = [0, .25, .25, .5], [.5, .125, .125, .25]
    tokens = np.zeros((n, children + 1), np.int32)
    u, un = np.full((n, children + 1), 0.5), np.array([0, .2, .25, .26, .49, .5, .6, .99999994], np.float32)
    parents = [-1] + [0] * children
    got = run(parents, tokens, P, Q, u, un)
    assert got[0] == [[0]] * n
    assert got[1] == [exact(parents, tokens[s], P[s], Q[s], u[s], un[s])[1] for s in range(n)]
    # a last child with a token of the others: what is left of it against its share
    tokens[:, -1], u[:, -1] = at[3], np.linspace(0.05, 0.95, n)
    if children > 1:
        want = [exact(parents, tokens[s], P[s], Q[s], u[s], un[s]) for s in range(n)]
        assert run(parents, tokens, P, Q, u, un) == ([w[0] for w in want], [w[1] for w in want])
