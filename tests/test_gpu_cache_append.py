"""Rotating and appending rows, and keeping the accepted ones, on the GPU
against fp64 statements."""

import numpy as np
import pytest
import torch

from rag_kv_cache_rerotate_gb300 import fusekv as fk

import step_ops
from step_ops import KIND, Step, StepCase, check_close, f64, i32, rotate, thetas

pytestmark = pytest.mark.gpu

ROPES = {
    "half": dict(),
    "interleaved": dict(layout=fk.FUSE_ROPE_INTERLEAVED),
    "part": dict(rot_dim=32),
    "part interleaved": dict(layout=fk.FUSE_ROPE_INTERLEAVED, rot_dim=16),
    "linear": dict(scaling=fk.FUSE_ROPE_LINEAR, factor=4.0),
    "llama3": dict(scaling=fk.FUSE_ROPE_LLAMA3, factor=8.0, original_len=8192, low=1.0, high=4.0),
    "yarn": dict(scaling=fk.FUSE_ROPE_YARN, factor=4.0, original_len=4096, low=1.0, high=32.0, mscale=1.1386),
}


def expected(s, kw, lens):
    """(Qr, Kr, k pool, v pool) with tolerances, in fp64."""
    c = s.c
    r = fk.rope_desc(**kw)
    rot = r.rot_dim or s.d
    th = thetas(c.base, rot, r.scaling, r.factor, r.original_len, r.low, r.high)
    x = f64(s.qkv)
    pos = np.zeros(s.n_rows)
    kp, vp = f64(s.kp), f64(s.vp)
    tk, tv = np.zeros_like(kp), np.zeros_like(vp)
    for q, (held, n) in enumerate(zip(lens, c.new)):
        a = s.starts[q]
        pos[a:a + n] = held + np.array(step_ops.depths(s.trees[q]))
    y, tol = rotate(x[:, :s.Hq + s.Hkv], pos, th, r.layout, r.mscale, c.dtype)
    for q, (held, n) in enumerate(zip(lens, c.new)):
        a = s.starts[q]
        page, at = s.slots(q, range(held, held + n))
        kp[page, at], vp[page, at] = y[a:a + n, s.Hq:], x[a:a + n, s.Hq + s.Hkv:]
        tk[page, at] = tol[a:a + n, s.Hq:]
    Q, tq = y[:, :s.Hq], tol[:, :s.Hq]
    out = np.ones(s.n_rows, bool)
    out[s.starts[0]:s.starts[-1]] = False
    return (Q, tq, out), (y[:, s.Hq:], tol[:, s.Hq:]), (kp, tk), (vp, tv)


def run(s, kw, **over):
    a = dict(parents=s.parents, Q=s.Q, K=s.K, V=s.V, Qr=s.Qr, Kr=None, k_pool=s.kp, v_pool=s.vp, ws=s.ws)
    a.update(over)
    fk.cache_append(s.desc, fk.rope_desc(**kw), s.seqs, **a)


def check(s, kw, lens=None, Kr=None):
    lens = s.c.lens if lens is None else lens
    before = f64(s.Qr)
    (Q, tq, out), (K, tk), (kp, tkp), (vp, tvp) = expected(s, kw, lens)
    run(s, kw, Kr=Kr)
    fk.check_errors(s.ws)
    got = f64(s.Qr)
    assert np.array_equal(got[out], before[out]), "rows outside the sequences"
    check_close(got[~out], Q[~out], tq[~out], "Qr")
    if Kr is not None:
        check_close(f64(Kr)[~out], K[~out], tk[~out], "Kr")
    check_close(f64(s.kp), kp, tkp, "k pool")
    assert np.array_equal(f64(s.vp), vp), "v pool"


@pytest.mark.parametrize("kind", sorted(ROPES))
@pytest.mark.parametrize("dtype,heads", [("bf16", (8, 2, 128)), ("f32", (4, 4, 64)), ("bf16", (16, 2, 64))])
def test_ropes(kind, dtype, heads):
    s = Step(StepCase(lens=[37, 0, 1000], new=[9, 3, 1], heads=heads, dtype=dtype, front=2, behind=1))
    check(s, ROPES[kind], Kr=torch.zeros(s.n_rows, heads[1], heads[2], dtype=step_ops.DT[dtype], device="cuda"))


@pytest.mark.parametrize("bs", [1, 5, 16, 64, 4096])
@pytest.mark.parametrize("lens,new,width", [
    ([0], [1], 2), ([15, 16, 17, 0, 4], [1, 0, 64, 1, 2], 4), ([3] * 70, [1, 2, 0, 3, 1, 1, 4] * 10, 1),
    ([0, 7], [700, 333], 0)])
def test_sequences_and_pages(lens, new, width, bs):
    check(Step(StepCase(lens=lens, new=new, width=width, block_size=bs, heads=(2, 1, 64), behind=5, seed=bs)),
          ROPES["half"])


@pytest.mark.parametrize("pos", [10 ** 5, 2 ** 24 + 1, 2 ** 30 + 12345])
def test_far_positions(pos):
    # one page holds the far slots: table entries in front of it are not read
    s = Step(StepCase(lens=[0], new=[40], width=0, heads=(2, 1, 128), dtype="f32", block_size=64, base=1e6))
    tab = torch.zeros(1, pos // 64 + 3, dtype=torch.int32, device="cuda")
    tab[:, -4:] = torch.tensor([0, 1, 2, 3], device="cuda") % s.n_pages
    s.tab = tab.cpu().numpy()
    lens = i32([pos])
    s.seqs = fk.Sequences(tab, lens, s.rows, 64, s.n_pages, 40)
    check(s, dict(), lens=[pos])


def test_many_rows_each_once():
    # more rows than a launch has CTAs: several of each
    s = Step(StepCase(lens=[5, 0, 31], new=[9000, 1, 2500], width=0, heads=(2, 2, 64), block_size=32))
    check(s, ROPES["interleaved"])


def test_in_place_and_without_queries():
    s = Step(StepCase(lens=[20, 3], new=[7, 12]))
    (Q, tq, _), (K, tk), (kp, tkp), (vp, _) = expected(s, dict(), s.c.lens)
    q, k = s.Q.contiguous(), s.K.contiguous()
    run(s, dict(), Q=q, Qr=q, K=k, Kr=k)
    check_close(f64(q), Q, tq, "Q in place")
    check_close(f64(k), K, tk, "K in place")
    check_close(f64(s.kp), kp, tkp, "k pool")
    t = Step(StepCase(lens=[20, 3], new=[7, 12]))
    run(t, dict(), Q=None, Qr=None)
    fk.check_errors(t.ws)
    assert torch.equal(t.kp, s.kp) and torch.equal(t.vp, s.vp)


def test_values_that_are_no_numbers_stay():
    s = Step(StepCase(lens=[20], new=[7]))
    s.qkv[2, :, 5] = float("nan")
    s.qkv[3, :, 70] = float("-inf")
    run(s, dict(rot_dim=32))
    _, at = s.slots(0, range(20, 27))
    page, _ = s.slots(0, range(20, 27))
    k, v = f64(s.kp)[page, at], f64(s.vp)[page, at]
    bad = np.zeros_like(k, dtype=bool)
    bad[2, :, [5, 21]] = True                              # the pair
    bad[3, :, 70] = True                                   # not rotated
    assert np.array_equal(~np.isfinite(k), bad)
    assert np.isnan(v[2, :, 5]).all() and np.isneginf(v[3, :, 70]).all()


@pytest.mark.parametrize("what", ["descending rows", "too many rows", "past n_rows", "negative length", "past the table",
                                  "bad page", "bad parent"])
def test_device_bounds(what):
    s = Step(StepCase(lens=[20, 30, 5], new=[3, 4, 3], heads=(2, 1, 64)))
    left = Step(StepCase(lens=[20, 30, 5], new=[3, 4, 3], heads=(2, 1, 64)))
    skipped = [1]
    if what == "descending rows":
        s.rows.copy_(i32([0, 7, 3, 10]))
        skipped = [0, 1, 2]                                # 0 and 2 share rows, whose owner is not defined
    elif what == "too many rows":
        s.seqs = fk.Sequences(s.tables, s.lens, s.rows, 16, s.n_pages, 3)
    elif what == "past n_rows":
        s.rows.copy_(i32([0, 3, 7, 11]))
        skipped = [2]
    elif what == "negative length":
        s.lens[1] = -1
    elif what == "past the table":
        s.lens[1] = s.tab.shape[1] * 16 - 3
    elif what == "bad page":
        s.tables[1, 1:3] = torch.tensor([s.n_pages, -1], device="cuda")
    else:
        s.parents[6] = 3
        skipped = []
    run(s, dict())
    with pytest.raises(fk.FuseError) as e:
        fk.check_errors(s.ws)
    assert e.value.status == fk.FUSE_ERR_DEVICE_BOUNDS
    run(left, dict())
    for q in range(3):
        page, at = left.slots(q, range(left.c.lens[q] + left.c.new[q]))
        same = torch.equal(s.vp[page, at], left.vp[page, at])
        if q not in skipped:
            assert same, q
        elif what != "descending rows":
            assert not same, q


# ---------------------------------------------------------------------------
# keep
# ---------------------------------------------------------------------------

def pools_of(s, layers):
    rng = np.random.default_rng(7)
    make = lambda: torch.from_numpy(rng.standard_normal(tuple(s.kp.shape)).astype(np.float32)).to(s.kp.dtype).cuda()  # noqa: E731
    k, v = [make() for _ in range(layers)], [make() for _ in range(layers)]
    return k, v, fk.PagePools(k, v, KIND[s.c.dtype], s.c.block_size)


def random_path(n, rng):
    if n == 0:
        return []
    return [0] + [i for i in range(1, n) if rng.random() < 0.4]


@pytest.mark.parametrize("layers", [1, 3, 70])
@pytest.mark.parametrize("dtype,heads,bs", [("bf16", (8, 2, 128), 16), ("f32", (4, 4, 64), 5), ("bf16", (16, 16, 128), 1)])
def test_keep(layers, dtype, heads, bs):
    s = Step(StepCase(lens=[37, 0, 100, 8], new=[9, 64, 1, 0], heads=heads, dtype=dtype, block_size=bs))
    k, v, pools = pools_of(s, layers)
    rng = np.random.default_rng(bs)
    paths = [random_path(n, rng) for n in s.c.new]
    path = np.full((4, 64), -1, np.int32)
    for q, p in enumerate(paths):
        path[q, :len(p)] = p
    want = []
    for t in k + v:
        x = t.clone()
        for q, p in enumerate(paths):
            if p:
                a, b = s.slots(q, s.c.lens[q] + np.array(p)), s.slots(q, s.c.lens[q] + np.arange(len(p)))
                x[b[0], b[1]] = t[a[0], a[1]]
        want.append(x)
    fk.cache_keep(s.desc, pools, s.seqs, i32(path), i32([len(p) for p in paths]), s.ws)
    fk.check_errors(s.ws)
    assert all(torch.equal(a, b) for a, b in zip(k + v, want))
    assert s.lens.tolist() == [n + len(p) for n, p in zip(s.c.lens, paths)]


def test_keep_without_pools_raises_lengths():
    s = Step(StepCase(lens=[5, 9], new=[4, 4]))
    _, _, pools = pools_of(s, 1)
    pools.c.n_pools = 0
    fk.cache_keep(s.desc, pools, s.seqs, i32([[0, 2], [0, -1]]), i32([2, 1]), s.ws)
    fk.check_errors(s.ws)
    assert s.lens.tolist() == [7, 10]


@pytest.mark.parametrize("path,count", [([0, 0, 3], 3), ([0, 2, 1], 3), ([0, 2, 9], 3), ([-1, 2, 3], 3), ([0, 1, 2], 4),
                                        ([0, 1, 2], -1)])
def test_keep_leaves_a_bad_path(path, count):
    s = Step(StepCase(lens=[5, 9], new=[9, 4]))
    k, v, pools = pools_of(s, 2)
    k0 = [t.clone() for t in k]
    fk.cache_keep(s.desc, pools, s.seqs, i32([path, [0, 2, -1]]), i32([count, 2]), s.ws)
    with pytest.raises(fk.FuseError) as e:
        fk.check_errors(s.ws)
    assert e.value.status == fk.FUSE_ERR_DEVICE_BOUNDS
    assert s.lens.tolist() == [5, 11]
    page, at = s.slots(0, range(14))
    assert all(torch.equal(a[page, at], b[page, at]) for a, b in zip(k, k0))


@pytest.mark.parametrize("n", [3, 128, 129, 5000])
@pytest.mark.parametrize("what", ["negative length", "past the table", "rows behind n_rows", "descending rows"])
def test_bad_sequences_without_rows_are_recorded(what, n):
    # no row leads to them; what the others bring is appended
    lens, new = [9] * n, [0] * n
    new[0], new[n // 2] = 3, 5
    s = Step(StepCase(lens=lens, new=new, heads=(2, 1, 64), width=0))
    bad = n - 1
    if what == "negative length":
        s.lens[bad] = -1
    elif what == "past the table":
        s.lens[bad] = s.tab.shape[1] * 16 + 1
    elif what == "rows behind n_rows":
        s.rows[n] = s.n_rows + 2
    else:
        s.rows[n] = s.n_rows - 1
    t = Step(StepCase(lens=lens, new=new, heads=(2, 1, 64), width=0))
    run(s, dict())
    run(t, dict())
    fk.check_errors(t.ws)
    with pytest.raises(fk.FuseError) as e:
        fk.check_errors(s.ws)
    assert e.value.status == fk.FUSE_ERR_DEVICE_BOUNDS
    last = 8 if what != "descending rows" else 7           # (a start that descends may cost rows next to it)
    assert torch.equal(s.Qr[:last], t.Qr[:last])
    for q in (0, n // 2):
        page, at = s.slots(q, range(9, 9 + new[q] - (what == "descending rows")))
        assert torch.equal(s.kp[page, at], t.kp[page, at]) and torch.equal(s.vp[page, at], t.vp[page, at])
