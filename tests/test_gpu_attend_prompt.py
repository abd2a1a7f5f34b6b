"""fuse_attend_prompt on the GPU against its fp64 statement: types, head
layouts, lengths around the tiles' edges, rows between and behind requests,
values that a row must not see, many requests, streams and graphs."""

import numpy as np
import pytest
import torch

from rag_kv_cache_rerotate_gb300 import fusekv as fk

from cache_ops import DT, KIND, f64, prompt_reference

pytestmark = pytest.mark.gpu


class Prompt:
    def __init__(self, spans, heads, dtype, seed=0, rows=None, split=0):
        Hq, Hkv, d = heads
        g = torch.Generator().manual_seed(seed)
        self.spans, self.dtype = spans, dtype
        T = rows or max(a + n for a, n in spans)
        nan = float("nan")
        mk = lambda h, s: (s * torch.randn(T, h, d, generator=g)).to(DT[dtype])  # noqa: E731
        self.Q, self.K, self.V = mk(Hq, 1.5), mk(Hkv, 1.0), mk(Hkv, 1.0)
        inside = torch.zeros(T, dtype=torch.bool)
        for a, n in spans:
            inside[a:a + n] = True
        for x in (self.Q, self.K, self.V):                 # rows of no request
            x[~inside] = nan
        self.inside = inside
        self.Q, self.K, self.V = self.Q.cuda(), self.K.cuda(), self.V.cuda()
        self.O = torch.full_like(self.Q, 7.0)
        self.desc = fk.layer_desc(64, Hq, Hkv, d, 1e6, KIND[dtype])
        self.reqs = fk.RequestTable([fk.Request(a, 0, 0, 0, n - min(split, n), min(split, n), 0, 0)
                                     for a, n in spans])
        self.ws = fk.alloc_workspace(self.desc, self.reqs)

    def run(self, stream=None):
        fk.attend_prompt(self.desc, self.reqs, self.Q, self.K, self.V, self.O, self.ws, stream)
        return self.O

    def check(self):
        got = f64(self.run())
        fk.check_errors(self.ws)
        want, tol = prompt_reference(self.Q, self.K, self.V, self.spans, self.dtype)
        m = self.inside.numpy()
        err = np.abs(got[m] - want[m])
        bad = ~(err <= tol[m])
        assert not bad.any(), (int(bad.sum()), float(np.nanmax(err / tol[m])), np.argwhere(bad)[:3].tolist())
        assert (got[~m] == 7.0).all()                       # rows of no request are left alone


def packed(lens, gap=0):
    out, a = [], 0
    for n in lens:
        out.append((a, n))
        a += n + gap
    return out


HEADS = [(8, 1, 128), (8, 2, 128), (4, 2, 128), (3, 3, 128), (8, 1, 64), (8, 2, 64), (4, 2, 64), (2, 2, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads", HEADS)
def test_packed_prompts(dtype, heads):
    Prompt(packed([1, 17, 128, 300, 0, 129, 64]), heads, dtype, split=5).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 33, 63, 65, 127, 128, 129, 255, 257, 511, 640])
def test_lengths_around_the_tiles(dtype, n):
    Prompt([(0, n)], (8, 2, 128) if n % 2 else (4, 1, 64), dtype, seed=n).check()


@pytest.mark.parametrize("heads", [(8, 1, 128), (2, 1, 128), (4, 4, 64)])
def test_longer_prompts(heads):
    Prompt(packed([1500, 2049]), heads, "bf16").check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_between_and_behind_requests(dtype):
    Prompt(packed([40, 130, 5], gap=9), (4, 2, 128), dtype, rows=300).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads", [(8, 1, 128), (2, 2, 128), (4, 2, 64)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_later_rows_do_not_reach_earlier_ones(dtype, heads, value):
    p = Prompt(packed([150, 77]), heads, dtype)
    want, tol = prompt_reference(p.Q, p.K, p.V, p.spans, dtype)
    for row in (3, 10, 131, 149, 150 + 40):
        p2 = Prompt(packed([150, 77]), heads, dtype)
        p2.V[row, 0, 5] = value
        p2.K[row, -1, 2] = value
        got = f64(p2.run())
        fk.check_errors(p2.ws)
        end = 150 if row < 150 else 227
        unseen = np.ones(227, bool)
        unseen[row:end] = False
        assert (np.abs(got[unseen] - want[unseen]) <= tol[unseen]).all(), row
        g = heads[0] // heads[1]
        assert not np.isfinite(got[row:end, :g, 5]).any(), row       # and it does reach those that see it


def test_masked_scores_may_be_infinite():
    # keys whose scores overflow sit only where they are masked
    p = Prompt([(0, 200)], (2, 1, 128), "bf16")
    want, tol = prompt_reference(p.Q, p.K, p.V, p.spans, "bf16")
    p.K[199] = 3e38
    got = f64(p.run())
    assert (np.abs(got[:199] - want[:199]) <= tol[:199]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scores_near_the_lowest_number(dtype):
    # equal scores of -2^127 (before the scale): every row is the mean of the
    # values it sees.  Weights are 1 exactly; n additions in fp32, the quotient
    # and the output's rounding are left.
    p = Prompt([(0, 300)], (2, 1, 128), dtype)
    p.Q.fill_(2.0 ** 60)
    p.K.fill_(-2.0 ** 60)
    got = f64(p.run())
    fk.check_errors(p.ws)
    V = f64(p.V)
    n = np.arange(1, 301)[:, None, None]
    want, span = np.cumsum(V, 0) / n, np.cumsum(np.abs(V), 0) / n
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    assert (np.abs(got - want) <= half * np.abs(want) + (n + 4) * 2.0 ** -23 * span).all()


def test_large_scores():
    # one key takes all of the weight
    p = Prompt([(0, 260)], (2, 1, 64), "bf16")
    p.Q.mul_(30)
    p.check()


def test_more_requests_than_one_launch_takes():
    rng = np.random.default_rng(3)
    Prompt(packed([int(x) for x in rng.integers(0, 40, size=600)]), (2, 1, 64), "bf16").check()


@pytest.mark.parametrize("lens", [[50, 3], [300, 257], [260, 33, 64] * 9 + [1, 31]])
@pytest.mark.parametrize("heads", [(4, 2, 64), (8, 1, 128), (2, 2, 128)])
def test_fp32_tiles_of_few_and_many_rows(lens, heads):
    # 16, 32 and 64 rows a tile, by the number of tiles
    Prompt(packed(lens, gap=1), heads, "f32").check()


def test_equal_lengths_and_a_single_row_each():
    Prompt(packed([1] * 70), (8, 2, 128), "bf16").check()


def test_repeated_runs_other_stream_and_graph():
    p = Prompt(packed([333, 128, 77]), (8, 2, 128), "bf16")
    want = p.run().clone()
    assert torch.equal(p.run(), want)
    s = torch.cuda.Stream()
    p.O.zero_()
    torch.cuda.synchronize()
    p.run(stream=s)
    s.synchronize()
    assert torch.equal(p.O, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        p.run(stream=s)
    p.Q.mul_(0.5)
    g.replay()
    got = p.O.clone()
    assert torch.equal(p.run(), got) and not torch.equal(got, want)


@pytest.mark.parametrize("dtype,heads", [("bf16", (8, 2, 128)), ("bf16", (4, 1, 64)), ("f32", (4, 2, 64))])
@pytest.mark.parametrize("n", [1, 128, 140, 300])
def test_keys_of_score_minus_infinity_have_no_weight(dtype, heads, n):
    # the first n keys score -infinity: rows behind them are as without them, to
    # the same bound (weights of 0 add nothing); rows that see no other key are
    # NaN, 0 / 0
    p = Prompt([(0, 400)], heads, dtype)
    p.Q[..., 0] = 1.0
    want, tol = prompt_reference(p.Q, p.K, p.V, [(n, 400 - n)], dtype)
    p.K[:n, :, 0] = -float("inf")
    got = f64(p.run())
    fk.check_errors(p.ws)
    assert (np.abs(got[n:] - want[n:]) <= tol[n:]).all()
    assert np.isnan(got[:n]).all()
