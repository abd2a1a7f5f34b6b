"""Attention of trees of new tokens over a paged cache, on the GPU against an
fp64 statement."""

import numpy as np
import pytest
import torch

from rag_kv_cache_rerotate_gb300 import fusekv as fk

from step_ops import Step, StepCase, check_close, f64, i32

pytestmark = pytest.mark.gpu


def check(s, rows=None, lens=None):
    before = f64(s.O)
    O, tol = s.tree_reference(rows, lens)
    got = f64(s.attend())
    fk.check_errors(s.ws)
    out = np.ones(s.n_rows, bool)
    out[s.starts[0]:s.starts[-1]] = False
    assert np.array_equal(got[out], before[out]), "rows outside the sequences"
    check_close(got, O, tol, "O")
    return got


HEADS = [("bf16", (8, 2, 128)), ("bf16", (8, 8, 128)), ("bf16", (16, 2, 64)), ("bf16", (4, 2, 64)),
         ("f32", (4, 2, 64)), ("f32", (8, 1, 128))]


@pytest.mark.parametrize("dtype,heads", HEADS)
@pytest.mark.parametrize("lens,new", [
    ([0], [1]), ([1], [1]), ([300], [1]), ([0, 0, 5], [1, 17, 2]), ([127, 128, 129, 0], [1, 1, 1, 128 - 64]),
    ([255, 64, 700], [3, 0, 33])])
def test_shapes(dtype, heads, lens, new):
    check(Step(StepCase(lens=lens, new=new, heads=heads, dtype=dtype, front=1, behind=2)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bs", [1, 5, 24, 64, 128, 1000])
def test_pages(bs, dtype):
    check(Step(StepCase(lens=[131, 40, 513], new=[13, 64, 5], block_size=bs, dtype=dtype, heads=(8, 4, 64), seed=bs)))


@pytest.mark.parametrize("width", [0, 1, 2, 8, 64])
@pytest.mark.parametrize("heads", [(8, 1, 128), (8, 2, 128), (4, 2, 64)])
def test_trees(width, heads):
    # 0: parents are not given; 64: nearly a star
    check(Step(StepCase(lens=[250, 3], new=[64, 40], width=width, heads=heads, seed=width)))


@pytest.mark.parametrize("dtype,heads", [("bf16", (8, 1, 128)), ("bf16", (16, 4, 64)), ("f32", (4, 2, 64))])
def test_long_contexts(dtype, heads):
    # many workers share a unit
    s = Step(StepCase(lens=[9000, 20011, 1], new=[2, 64, 5], heads=heads, dtype=dtype, block_size=32))
    check(s, rows=[0, 1, 2, 33, 65, 66, 70])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("slope", [0.05, 0.28, 4.0, -0.28])
def test_scores_that_rise_or_fall(dtype, slope):
    # from key to key by 1.44 * slope (log2): a worker's tiles outweigh the ones before them by a little or by far
    s = Step(StepCase(lens=[20000], new=[64], heads=(16, 4, 64), dtype=dtype, block_size=32, width=3, scale=0.1))
    s.Qr[..., 0] = 8.0
    page, at = s.slots(0, range(20064))
    s.kp[torch.as_tensor(page).cuda(), torch.as_tensor(at).cuda(), :, 0] = (
        slope * torch.arange(20064, device="cuda")[:, None]).to(s.kp.dtype)
    check(s, rows=[0, 1, 31, 63])


def test_calls_without_rows_of_a_sequence():
    # every row lies outside the sequences; what follows finds the lengths as the call did
    s = Step(StepCase(lens=[40, 7], new=[0, 0], front=5, behind=3))             # tables of 48 and 16 slots
    for _ in range(8):
        check(s)
        s.lens.add_(1)


def test_many_sequences():
    # workers take several units; sequences without rows between them
    n = 300
    rng = np.random.default_rng(4)
    check(Step(StepCase(lens=rng.integers(0, 90, n).tolist(), new=rng.integers(0, 4, n).tolist(), heads=(4, 2, 64))))


@pytest.mark.parametrize("bs", [16, 5])
@pytest.mark.parametrize("d", [128, 64])
def test_many_short_parts(d, bs):
    # a worker takes a dozen units of one to six tiles, whose tiles take turns in its ring
    n = 120
    rng = np.random.default_rng(d + bs)
    check(Step(StepCase(lens=rng.integers(0, 700, n).tolist(), new=rng.integers(1, 9, n).tolist(), width=2,
                        heads=(16, 16, d), block_size=bs, seed=bs)))


@pytest.mark.parametrize("d", [128, 64])
def test_many_full_trees(d):
    # both accumulators of a worker in use, units of one to four tiles, several a worker
    n = 60
    rng = np.random.default_rng(d)
    new = rng.integers(40, 65, n).tolist()
    s = Step(StepCase(lens=rng.integers(0, 400, n).tolist(), new=new, width=5, heads=(64, 16, d), seed=d))
    check(s, rows=[r for a, b in zip(s.starts, s.starts[1:]) for r in (a, a + 31, b - 1)])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_and_lowest_scores(dtype):
    # one key takes all of a row's weight; scores near the type's range
    s = Step(StepCase(lens=[200, 300], new=[5, 20], dtype=dtype, scale=60.0))
    check(s)
    s = Step(StepCase(lens=[200], new=[9], dtype=dtype))
    s.kp[..., 0] = -1.0
    s.Qr[..., 0] = 3.0e38                                  # every score at the bottom of the range: equal weights
    s.Qr[..., 1:] = 0.0
    O = f64(s.attend())
    page, at = s.slots(0, range(209))
    v = f64(s.vp)[page, at]
    want = np.stack([np.repeat(v[np.concatenate([np.ones(200, bool), m])].mean(0), 4, 0)
                     for m in __import__("step_ops").ancestors(s.trees[0])])
    assert np.max(np.abs(O - want)) <= 2.0 ** -7 * np.abs(v).max()


BAD = [float("nan"), float("inf"), float("-inf")]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads", [(8, 2, 128), (16, 2, 64)])
@pytest.mark.parametrize("held", [0, 100, 128, 1000])
def test_what_a_row_does_not_see(dtype, heads, held):
    s = Step(StepCase(lens=[held, 50], new=[20, 3], dtype=dtype, heads=heads, block_size=24, width=4, pages=4))
    used = np.zeros((s.n_pages, 24), bool)
    for q in range(2):
        page, at = s.slots(q, range(s.c.lens[q] + s.c.new[q]))
        used[page, at] = True
    free = torch.from_numpy(~used).cuda()
    clean = s.attend().clone()
    fk.check_errors(s.ws)
    for x in BAD:                                          # behind the last slots, and in pages of nobody
        s.kp[free], s.vp[free] = x, x
        assert torch.equal(s.attend(), clean)
    # a node's key and value: its row and its descendants' get it, no other does
    from step_ops import ancestors
    seen = ancestors(s.trees[0])
    for node, x in ((7, BAD[0]), (19, BAD[1]), (0, BAD[0])):
        page, at = s.slots(0, [held + node])
        k, v = s.kp[page, at].clone(), s.vp[page, at].clone()
        s.kp[page, at], s.vp[page, at] = x, x
        got = s.attend()
        hit = torch.from_numpy(seen[:, node]).cuda()
        assert torch.equal(got[:20][~hit], clean[:20][~hit]) and torch.equal(got[20:], clean[20:])
        assert not torch.isfinite(got[:20][hit]).any()
        s.kp[page, at] = k                                 # the value alone
        got = s.attend()
        assert torch.equal(got[:20][~hit], clean[:20][~hit])
        assert not torch.isfinite(got[:20][hit]).any()
        s.vp[page, at, :, 3:] = v[..., 3:]                 # three of its channels
        got = s.attend()
        assert torch.equal(got[:20][~hit], clean[:20][~hit])
        assert not torch.isfinite(got[:20][hit][..., :3]).any() and torch.equal(got[:20][hit][..., 3:], clean[:20][hit][..., 3:])
        s.vp[page, at] = v
    assert torch.equal(s.attend(), clean)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_keys_of_score_minus_infinity(dtype):
    # they have no weight; the other keys keep theirs
    s = Step(StepCase(lens=[300], new=[4], dtype=dtype, heads=(4, 2, 64)))
    s.Qr[..., 0] = 1.0
    page, at = s.slots(0, range(0, 200))
    s.kp[page, at, :, 0] = float("-inf")
    t = Step(StepCase(lens=[300], new=[4], dtype=dtype, heads=(4, 2, 64)))
    t.Qr[..., 0] = 1.0
    tab = s.tab.copy()
    O = f64(s.attend())
    # the same attention without those keys, in fp64
    K, V, Q = f64(t.kp), f64(t.vp), f64(t.Qr)
    pg, a = t.slots(0, range(200, 304))
    from step_ops import ancestors
    seen = np.concatenate([np.ones((4, 100), bool), ancestors(t.trees[0])], 1)
    for i in range(4):
        for h in range(4):
            k, v = K[pg, a, h // 2][seen[i]], V[pg, a, h // 2][seen[i]]
            x = k @ Q[i, h] / 8
            p = np.exp(x - x.max())
            p /= p.sum()
            assert np.all(np.abs(O[i, h] - p @ v) <= 2.0 ** -7 * (p @ np.abs(v)))
    assert np.array_equal(tab, s.tab)


def test_bad_pages_and_rows():
    s = Step(StepCase(lens=[100, 200, 50], new=[3, 3, 3]))
    clean = s.attend().clone()
    fk.check_errors(s.ws)
    bad = s.tables.clone()
    s.tables[1, 2], s.tables[1, 5] = s.n_pages, -1
    got = s.attend().clone()
    with pytest.raises(fk.FuseError) as e:
        fk.check_errors(s.ws)
    assert e.value.status == fk.FUSE_ERR_DEVICE_BOUNDS
    assert torch.equal(got[:3], clean[:3]) and torch.equal(got[6:], clean[6:])
    # their 32 tokens are not there
    gone = np.r_[32:48, 80:96]
    K, V, Q = f64(s.kp), f64(s.vp), f64(s.Qr)
    from step_ops import ancestors
    pg, a = s.slots(1, range(203))
    for i in range(3):
        seen = np.concatenate([np.ones(200, bool), ancestors(s.trees[1])[i]])
        seen[gone] = False
        for h in range(8):
            k, v = K[pg, a, h // 4][seen], V[pg, a, h // 4][seen]
            x = k @ Q[3 + i, h] / np.sqrt(128)
            p = np.exp(x - x.max())
            p /= p.sum()
            assert np.all(np.abs(f64(got)[3 + i, h] - p @ v) <= 2.0 ** -7 * (p @ np.abs(v)))
    s.tables.copy_(bad)
    s.lens[1] = -5                                         # the sequence is left out
    s.O.fill_(7.0)
    got = s.attend().clone()
    with pytest.raises(fk.FuseError):
        fk.check_errors(s.ws)
    assert torch.equal(got[:3], clean[:3]) and torch.equal(got[6:], clean[6:]) and (got[3:6] == 7.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_replays_take_new_lengths(dtype):
    # captured once, replayed with other lengths, rows and trees; another stream runs between
    s = Step(StepCase(lens=[500, 90, 0], new=[6, 1, 20], dtype=dtype, heads=(8, 2, 64)))
    t = Step(StepCase(lens=[800, 3], new=[9, 9], dtype=dtype, heads=(8, 2, 64), seed=5))
    alone, other = s.attend().clone(), t.attend().clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        s.attend()
    s.O.zero_()
    with torch.cuda.stream(side):
        for _ in range(3):
            g.replay()
            t.attend(side)
    side.synchronize()
    assert torch.equal(s.O, alone) and torch.equal(t.O, other)
    s.lens.copy_(i32([17, 90, 0]))
    O, tol = s.tree_reference(lens=[17, 90, 0])
    g.replay()
    torch.cuda.synchronize()
    check_close(f64(s.O), O, tol, "replayed")


def test_calls_with_workspaces_of_their_own_overlap():
    a = Step(StepCase(lens=[20000], new=[30], heads=(8, 2, 128)))
    b = Step(StepCase(lens=[20000], new=[30], heads=(8, 2, 128), seed=3))
    wa, wb = a.attend().clone(), b.attend().clone()
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(one):
            a.attend(one)
        with torch.cuda.stream(two):
            b.attend(two)
    torch.cuda.synchronize()
    assert torch.equal(a.O, wa) and torch.equal(b.O, wb)


def test_pool_past_32_bits():
    # elements of a pool beyond 2^31: a page at its end
    d, bs, pages = 128, 64, (1 << 31) // (64 * 8 * 128) + 40
    s = Step(StepCase(lens=[100], new=[5], heads=(8, 8, d), block_size=bs))
    kp = torch.empty(pages, bs, 8, d, dtype=torch.bfloat16, device="cuda")
    vp = torch.empty_like(kp)
    clean = s.attend().clone()
    for i in range(s.tab.shape[1]):
        kp[pages - 1 - i], vp[pages - 1 - i] = s.kp[s.tab[0, i]], s.vp[s.tab[0, i]]
    s.tables.copy_(i32([[pages - 1 - i for i in range(s.tab.shape[1])]]))
    s.kp, s.vp = kp, vp
    s.seqs = fk.Sequences(s.tables, s.lens, s.rows, bs, pages, 5)
    assert torch.equal(s.attend(), clean)
    fk.check_errors(s.ws)
