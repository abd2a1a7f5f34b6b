"""Verification of drafted tokens on the GPU against an fp64 statement, and a
run of the operators of a speculative step together."""

import numpy as np
import pytest
import torch

from rag_kv_cache_rerotate_gb300 import fusekv as fk

import step_ops
from step_ops import Step, StepCase, f64, i32, random_tree

pytestmark = pytest.mark.gpu


class Verify:
    def __init__(self, new, vocab, width=3, drawn=True, seed=0, blur=0.7, stride=None, front=0, sharp=3.0):
        rng = np.random.default_rng(seed)
        self.new, self.vocab = new, vocab
        self.starts = [front + sum(new[:i]) for i in range(len(new) + 1)]
        n = self.starts[-1]
        self.trees = [random_tree(k, width, rng) for k in new]
        z = sharp * rng.standard_normal((n, vocab))
        soft = lambda x: (np.exp(x - x.max(1, keepdims=True)) /  # noqa: E731
                          np.exp(x - x.max(1, keepdims=True)).sum(1, keepdims=True)).astype(np.float32)
        self.P, self.Q = soft(z), soft(z + blur * rng.standard_normal((n, vocab)))
        self.parents = np.array([-1] * front + [p for t in self.trees for p in t], dtype=np.int32)
        self.tokens = np.zeros(n, np.int32)
        for s, a in enumerate(self.starts[:-1]):
            for i, p in enumerate(self.trees[s]):
                w = self.Q[a + max(p, 0)].astype(np.float64)
                self.tokens[a + i] = rng.choice(vocab, p=w / w.sum())
        self.u, self.u_next = rng.random(n).astype(np.float32), rng.random(len(new)).astype(np.float32)
        if not drawn:
            self.Q = None
        self.stride = stride or vocab

    def dev(self, x):
        if x is None:
            return None
        t = torch.zeros(x.shape[0], self.stride, device="cuda")
        t[:, :self.vocab] = torch.from_numpy(x).cuda()
        return t[:, :self.vocab]

    def run(self, stream=None, ws=None, check=True):
        n, m = len(self.new), max([1] + list(self.new))
        self.path, self.count, self.next = (torch.full(z, -9, dtype=torch.int32, device="cuda") for z in ((n, m), (n,), (n,)))
        ws = fk.alloc_cache_workspace() if ws is None else ws
        fk.verify_tree(i32(self.starts), i32(self.parents), i32(self.tokens), self.dev(self.P), self.dev(self.Q),
                       torch.from_numpy(self.u).cuda(), torch.from_numpy(self.u_next).cuda(), self.path, self.count,
                       self.next, ws, stream)
        if check:
            fk.check_errors(ws)
        return [p[:k] for p, k in zip(self.path.tolist(), self.count.tolist())], self.next.tolist()

    def expected(self):
        paths, tokens = [], []
        for s, a in enumerate(self.starts[:-1]):
            b = self.starts[s + 1]
            if a == b:
                paths.append([])
                tokens.append(-1)
                continue
            P = self.P[a:b].astype(np.float64)
            Q = self.Q[a:b].astype(np.float64) if self.Q is not None else None
            p, t = step_ops.verify(self.trees[s], self.tokens[a:b], P, Q, self.u[a:b].astype(np.float64),
                                   float(self.u_next[s]))
            paths.append(p)
            tokens.append(t)
        return paths, tokens

    def check(self):
        assert self.run() == self.expected()
        for p, k in zip(self.path.tolist(), self.count.tolist()):
            assert all(x == -1 for x in p[k:])


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("vocab", [1, 2, 7, 127, 1000, 4099, 32000])
@pytest.mark.parametrize("width", [1, 4])
def test_vocabularies(vocab, width, drawn):
    Verify([8, 1, 16, 0, 5], vocab, width, drawn, seed=vocab + width).check()


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("n", [1, 40, 100, 700])
def test_batches(n, drawn):
    # one, several and a single CTA a sequence
    rng = np.random.default_rng(n)
    Verify(rng.integers(0, 12, n).tolist(), 501, 3, drawn, seed=n).check()


def test_all_nodes_and_a_large_vocabulary():
    Verify([64, 64], 128256, 8, True, seed=3).check()
    Verify([64, 33], 150001, 64, True, seed=4, blur=2.0).check()            # a star: many refusals in a row
    Verify([64, 33], 150001, 64, False, seed=5).check()


@pytest.mark.parametrize("stride", [0, 1, 2, 3, 5])
def test_strides_and_alignment(stride):
    Verify([5, 9, 3], 1001, 2, True, seed=9, stride=1001 + stride, front=3).check()
    Verify([5, 9, 3], 1000, 2, False, seed=9, stride=1000 + stride).check()


def test_probabilities_and_targets_of_different_alignment():
    v = Verify([6, 6], 999, 2, seed=2)
    want = v.expected()
    buf = torch.zeros(12 * 1000 + 2, device="cuda")
    Q = buf[1:1 + 12 * 1000].view(12, 1000)[:, :999]
    Q.copy_(torch.from_numpy(v.Q))
    v.dev = (lambda d: lambda x: Q if x is v.Q else d(x))(v.dev)
    assert v.run() == want


def test_extreme_random_numbers():
    v = Verify([6] * 4, 333, 2, seed=6)
    v.u[:] = 0.0                                           # every first child of positive probability
    v.u_next[:] = [0.0, 0.5, 0.99999994, 0.25]
    v.check()
    v.u[:] = 0.99999994
    v.check()
    v.u_next[:] = [1.0, 1.5, float("nan"), -1.0]           # as the last float before 1, and 0
    got = v.run()
    v.u_next[:] = [0.99999994, 0.99999994, 0.0, 0.0]
    assert got == v.expected()
    v.u[:] = float("nan")                                  # nothing is accepted
    assert [len(p) for p in v.run()[0]] == [1] * 4


def test_certain_targets():
    # one-hot targets: a draft stands exactly when it is the target's token
    v = Verify([5] * 30, 50, 1, seed=8)
    v.P[:] = 0.0
    rng = np.random.default_rng(1)
    hot = np.where(rng.random(len(v.tokens)) < 0.6, np.roll(v.tokens, -1), rng.integers(0, 50, len(v.tokens)))
    v.P[np.arange(len(hot)), hot] = 1.0
    v.check()
    w = Verify([5] * 30, 50, 1, drawn=False, seed=8)
    w.P = v.P
    w.check()


def test_same_token_twice():
    for drawn in (True, False):
        v = Verify([8] * 40, 20, 64, drawn, seed=12)
        v.tokens[:] = np.random.default_rng(0).integers(0, 3, len(v.tokens))
        v.check()


def test_draft_equal_to_target():
    # nothing is refused; where nothing is left of the target, its own row decides
    v = Verify([8] * 10, 300, 2, seed=13, blur=0.0)
    v.Q = v.P.copy()
    assert all(len(p) > 1 for p in v.run()[0])
    v.check()
    v.Q = np.minimum(1.0, v.P * 2).astype(np.float32)      # above the target everywhere
    v.u[:] = 0.99
    v.check()


def test_last_token_of_a_part():
    # all weight at the ends of the vocabulary and of its parts
    for at in (0, 1, 3, 4, 127, 128, 4095, 4096, 4998, 4999):
        v = Verify([1, 3], 5000, 1, seed=at)
        v.P[:] = 0.0
        v.P[:, at] = 1.0
        v.check()
        assert v.next.tolist()[0] == at


@pytest.mark.parametrize("what", ["token", "parent", "probability", "rows"])
def test_device_bounds(what):
    v = Verify([6, 6, 6], 100, 1, seed=15)
    v.u[:] = 0.0                                           # all drafts stand
    full, _ = v.run()
    assert [len(p) for p in full] == [6, 6, 6]
    if what == "token":
        v.tokens[8] = 100                                  # sequence 1, node 2
    elif what == "parent":
        v.parents[8] = 2
    elif what == "probability":
        v.P[7, v.tokens[8]] = float("nan")
    else:
        v.starts = [0, 6, 13, 18]                          # more than max_path
    got = v.run(check=False)[0]
    assert got[0] == full[0]
    assert len(got[1]) == (0 if what == "rows" else 2)
    ws = fk.alloc_cache_workspace()
    v.run(ws=ws, check=False)
    with pytest.raises(fk.FuseError) as e:
        fk.check_errors(ws)
    assert e.value.status == fk.FUSE_ERR_DEVICE_BOUNDS


def test_tokens_are_distributed_as_the_target():
    # 40000 sequences of one draft, the same two rows: the token that stands first
    n, vocab = 40000, 6
    rng = np.random.default_rng(21)
    P = np.array([[0.4, 0.05, 0.25, 0.2, 0.1, 0.0]] * 2, np.float32)
    Q = np.array([[0.1, 0.3, 0.1, 0.1, 0.2, 0.2]] * 2, np.float32)
    x = rng.choice(vocab, n, p=Q[0].astype(np.float64) / Q[0].astype(np.float64).sum())
    tok = np.zeros(2 * n, np.int32)
    tok[1::2] = x
    path, count, nxt = (torch.zeros(z, dtype=torch.int32, device="cuda") for z in ((n, 2), (n,), (n,)))
    ws = fk.alloc_cache_workspace()
    dev = lambda a: torch.from_numpy(np.tile(a, (n, 1))).cuda()  # noqa: E731
    fk.verify_tree(i32(np.arange(n + 1) * 2), i32([-1, 0] * n), i32(tok), dev(P), dev(Q),
                   torch.from_numpy(rng.random(2 * n).astype(np.float32)).cuda(),
                   torch.from_numpy(rng.random(n).astype(np.float32)).cuda(), path, count, nxt, ws)
    fk.check_errors(ws)
    first = np.where(count.cpu().numpy() == 2, x, nxt.cpu().numpy())
    share = np.bincount(first, minlength=vocab) / n
    assert np.all(np.abs(share - P[0]) <= 5 * np.sqrt(P[0] * (1 - P[0]) / n) + 1e-9)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_step_after_step(dtype):
    """Append a tree, attend it, verify, keep, twice over two layers, captured
    once: the kept tokens' attention is that of a cache that never held the
    other drafts."""
    c = StepCase(lens=[40, 0, 130], new=[9, 6, 12], heads=(4, 2, 64), dtype=dtype, block_size=8, width=3, pages=2)
    s = Step(c)
    room = 8                                               # table entries for the tokens that are kept
    extra = s.n_pages + np.arange(3 * room).reshape(3, room)
    need = [-(-(a + n) // 8) for a, n in zip(c.lens, c.new)]
    tab = np.full((3, max(need) + room), -1, np.int32)
    for q in range(3):
        tab[q, :need[q]] = s.tab[q, :need[q]]
        tab[q, need[q]:need[q] + room] = extra[q]
    s.tab = tab
    s.tables = i32(tab)
    pages = s.n_pages + 3 * room
    rng = np.random.default_rng(3)
    dt = step_ops.DT[dtype]
    make = lambda *z: torch.from_numpy(rng.standard_normal(z).astype(np.float32)).to(dt).cuda()  # noqa: E731
    kp, vp = [make(pages, 8, 2, 64) for _ in range(2)], [make(pages, 8, 2, 64) for _ in range(2)]
    s.n_pages = pages
    s.seqs = fk.Sequences(s.tables, s.lens, s.rows, 8, pages, 12)
    pools = fk.PagePools(kp, vp, step_ops.KIND[dtype], 8)
    rope = fk.rope_desc()
    vocab = 200
    v = Verify(c.new, vocab, seed=1)
    v.trees = s.trees
    tokens, P, Qd, u, un = i32(v.tokens), v.dev(v.P), v.dev(v.Q), torch.from_numpy(v.u).cuda(), torch.from_numpy(v.u_next).cuda()
    path, count, nxt = (torch.zeros(z, dtype=torch.int32, device="cuda") for z in ((3, 12), (3,), (3,)))
    O = [torch.zeros_like(s.Qr) for _ in range(2)]

    def step():
        for layer in range(2):
            fk.cache_append(s.desc, rope, s.seqs, s.parents, s.Q, s.K, s.V, s.Qr, None, kp[layer], vp[layer], s.ws)
            fk.attend_tree(s.desc, s.seqs, s.parents, s.Qr, kp[layer], vp[layer], O[layer], s.ws)
        fk.verify_tree(s.rows, s.parents, tokens, P, Qd, u, un, path, count, nxt, s.ws)
        fk.cache_keep(s.desc, pools, s.seqs, path, count, s.ws)

    k0, v0, l0 = [t.clone() for t in kp], [t.clone() for t in vp], s.lens.clone()
    step()
    for a, b in zip(kp + vp, k0 + v0):
        a.copy_(b)
    s.lens.copy_(l0)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    held = list(c.lens)
    for _ in range(2):
        s.c = StepCase(**{**c.__dict__, "lens": list(held)})
        before = [t.clone() for t in kp + vp]
        g.replay()
        fk.check_errors(s.ws)
        want = []
        for q in range(3):
            a = s.starts[q]
            b = s.starts[q + 1]
            want.append(step_ops.verify(s.trees[q], v.tokens[a:b], v.P[a:b].astype(np.float64),
                                        v.Q[a:b].astype(np.float64), v.u[a:b].astype(np.float64), float(v.u_next[q])))
        assert nxt.tolist() == [t for _, t in want]
        assert [p[:k] for p, k in zip(path.tolist(), count.tolist())] == [p for p, _ in want]
        assert s.lens.tolist() == [h + len(p) for h, (p, _) in zip(held, want)]
        theta = step_ops.thetas(c.base, 64)
        for q, (p, _) in enumerate(want):
            # the kept rows lie rotated at their positions; what was held is untouched
            a = s.starts[q]
            x = f64(s.K)[a + np.array(p)]
            y, tol = step_ops.rotate(x, held[q] + np.arange(len(p)), theta, fk.FUSE_ROPE_HALF, 1.0, dtype)
            pg, at = s.slots(q, held[q] + np.arange(len(p)))
            old = s.slots(q, np.arange(held[q]))
            for layer in range(2):
                step_ops.check_close(f64(kp[layer])[pg, at], y, tol, "kept keys")
                assert np.array_equal(f64(vp[layer])[pg, at], f64(s.V)[a + np.array(p)])
                assert torch.equal(kp[layer][old], before[layer][old])
            # a kept node's attention: of the kept cache, itself last
            for layer in range(2):
                K, V, Q = f64(kp[layer]), f64(vp[layer]), f64(s.Qr)
                for i, node in enumerate(p):
                    pg, at = s.slots(q, np.arange(held[q] + i + 1))
                    for h in range(4):
                        k, w = K[pg, at, h // 2], V[pg, at, h // 2]
                        z = k @ Q[a + node, h] / 8
                        e = np.exp(z - z.max())
                        e /= e.sum()
                        bound = (2.0 ** -7 if dtype == "bf16" else 2.0 ** -18) * (e @ np.abs(w))
                        assert np.all(np.abs(f64(O[layer])[a + node, h] - e @ w) <= bound)
            held[q] += len(p)
