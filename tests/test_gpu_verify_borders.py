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


def close(a, b, lo=2.0 ** -42, hi=2.0 ** -28):
    """Whether a and b differ by that much, relative to b.  The kernel's pairs have 48 bits: a sum or a product
    of them is off by some 2^-46, so that from 2^-42 on both sides agree on the order; 24 bits do not tell."""
    return b != 0 and lo <= abs(a / b - 1) <= hi


def draw(rng, *shape):
    # (numbers of 24 bits, between a quarter and a half)
    return (rng.integers(1 << 23, 1 << 24, shape) * 2.0 ** -25).astype(np.float32)


def test_drafts_next_to_their_border():
    # u q against p, and u S q against p - q behind a refusal
    rng = np.random.default_rng(0)
    F = lambda x: Fraction(float(x))  # noqa: E731
    cases = []
    while len(cases) < 600:
        p, q, u = draw(rng, 3), draw(rng, 3), np.float32(rng.random())
        p[1] = u * q[1]                                    # rounded
        if close(F(u) * F(q[1]), F(p[1])):
            cases.append((p, q, [0, 0, u], [0, 1, 1]))     # the first child's token, or the second one's
        p, q = draw(rng, 3), draw(rng, 3)
        p[0] = 0                                           # the first child is refused
        left = [max(F(a) - F(b), Fraction(0)) for a, b in zip(p, q)]
        if left[1] > 0:
            u = np.float32(float(left[1] / (sum(left) * F(q[1]))))
            if u < 1 and close(F(u) * sum(left) * F(q[1]), left[1]):
                cases.append((p, q, [0, 0, u], [0, 0, 1]))
    P, Q = (np.stack([np.stack([c[i]] * 3) for c in cases]) for i in range(2))
    u, tokens = np.array([c[2] for c in cases], np.float32), np.array([c[3] for c in cases])
    for c, row in zip(cases, u):
        if c[3][1] == 1:
            row[1] = c[2][2]                               # the first child itself is next to its border
    un = rng.random(len(cases)).astype(np.float32)
    parents = [-1, 0, 0]
    want = [exact(parents, tokens[s], P[s], Q[s], u[s], un[s])[0] for s in range(len(cases))]
    assert 100 < sum(len(w) > 1 for w in want) < 500       # both sides of the border
    assert run(parents, tokens, P, Q, u, un)[0] == want


@pytest.mark.parametrize("refused", [0, 1, 2])
@pytest.mark.parametrize("vocab", [4, 5003])
def test_next_tokens_next_to_their_border(refused, vocab):
    # u' sum r against r(0) + .. + r(x), where r is what refusals leave
    rng = np.random.default_rng(refused)
    F = lambda x: Fraction(float(x))  # noqa: E731
    at = [0, 1, vocab // 2 + 1, vocab - 1]
    cases = []
    while len(cases) < 300:
        p, q = draw(rng, 4), draw(rng, 4) / 2
        p[0] = 0                                           # the children's token
        r, S = [F(x) for x in p], Fraction(1)
        for _ in range(refused):
            r = [max(a - S * F(b), Fraction(0)) for a, b in zip(r, q)]
            S = sum(r)
        part = r[0] + r[1] + (r[2] if len(cases) % 2 else 0)
        un = np.float32(float(part / sum(r)))
        # (p, q and sums are about 1: 2^-42 of that, however small the part is)
        if un < 1 and abs(F(un) * sum(r) - part) >= 2.0 ** -42 and close(F(un) * sum(r), part):
            cases.append((p, q, un))
    n, k = len(cases), refused + 1
    P, Q = np.zeros((n, k, vocab), np.float32), np.zeros((n, k, vocab), np.float32)
    P[..., at], Q[..., at] = (np.stack([c[i] for c in cases])[:, None] for i in range(2))
    un = np.array([c[2] for c in cases], np.float32)
    parents, tokens, u = [-1] + [0] * refused, np.zeros((n, k), np.int32), np.full((n, k), 0.5, np.float32)
    want = [exact(parents, tokens[s], P[s], Q[s], u[s], un[s])[1] for s in range(n)]
    got = run(parents, tokens, P, Q if refused else None, u, un)[1]
    assert [(s, a, b) for s, (a, b) in enumerate(zip(got, want)) if a != b] == []


@pytest.mark.parametrize("drawn", [True, False])
def test_random_numbers_out_of_range(drawn):
    # below 0 as 0, from 1 on as the last float before 1, NaN accepts nothing
    values = [-1.0, -np.inf, -0.0, 1.0, 1.5, np.inf, 3e38, np.nan]
    as_if = [0.0, 0.0, 0.0] + [0.99999994] * 4
    n = len(values)
    P = np.zeros((n, 2, 5), np.float32)
    P[..., 1:4] = [0.25, 0.25, 0.5]
    P[:, 0, 2] = 0.25 if drawn else 1.0                    # accepted whatever its number is, 1 and more aside
    if not drawn:
        P[:, 0, [1, 3]] = 0.0
    Q = P.copy() if drawn else None
    tokens, un = np.full((n, 2), 2), np.full(n, 0.5, np.float32)
    u = np.array([[0.0, x] for x in values], np.float32)
    got = run([-1, 0], tokens, P, Q, u, un)[0]
    assert got == [[0, 1]] * len(as_if) + [[0]]
    if drawn:                                              # a draft that its distribution does not have
        Q[:, 0, 2] = 0.0
        assert run([-1, 0], tokens, P, Q, u, un)[0] == got
        P[:, 0, 2] = 0.0                                   # one that the target does not have
        assert run([-1, 0], tokens, P, Q, u, un)[0] == [[0]] * n
