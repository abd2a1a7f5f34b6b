"""Attention of trees at the edges of its definition, on the GPU: rows that nothing
is left for, and, against an fp64 statement, scores that are exact, so that the bound
is that of the weights and sums alone."""

import numpy as np
import pytest
import torch

from rag_kv_cache_rerotate_gb300 import fusekv as fk

from step_ops import HALF_STEP, Step, StepCase, ancestors, f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads", [(8, 2, 128), (16, 2, 64)])
@pytest.mark.parametrize("held,new", [(0, 1), (0, 9), (60, 64), (5000, 3), (20000, 40)])
@pytest.mark.parametrize("how", ["no page is in the pool", "every score is -infinity"])
def test_rows_that_nothing_is_left_for(how, held, new, heads, dtype):
    # zeros, whether one worker takes the unit or many do; the sequence beside it keeps its outputs
    s = Step(StepCase(lens=[held, 50], new=[new, 3], heads=heads, dtype=dtype, block_size=24))
    s.Qr[..., 0] = 1.0
    clean = s.attend().clone()
    fk.check_errors(s.ws)
    assert torch.isfinite(clean).all() and clean[:new].any(-1).all()
    if how == "no page is in the pool":
        s.tables[0] = torch.where(torch.arange(s.tables.shape[1], device="cuda") % 2 == 0, -1, s.n_pages)
        s.attend()
        with pytest.raises(fk.FuseError) as e:
            fk.check_errors(s.ws)
        assert e.value.status == fk.FUSE_ERR_DEVICE_BOUNDS
    else:
        page, at = s.slots(0, range(held + new))
        s.kp[page, at, :, 0] = float("-inf")
        s.attend()
        fk.check_errors(s.ws)
    assert (s.O[:new] == 0).all()
    assert torch.equal(s.O[new:], clean[new:])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads,block_size", [((16, 4, 64), 32), ((8, 1, 128), 5), ((4, 2, 128), 128)])
@pytest.mark.parametrize("step", [0.25, 0.5, 2.0, 32.0, -0.5, -32.0])
def test_exact_scores_that_rise_or_fall(step, heads, block_size, dtype):
    """Key j has the score step * j (and a constant): rising by 0.03 to 5.8 (log2) a
    key, so that a tile outweighs the one before it by 2^4 to 2^700, or falling.  Its two
    digits of base 256 and the queries' powers of two have few bits, so scores are exact.

    With A = sum p |v|: the scale takes three roundings, the reference's product one, their
    difference one and the join two, each at most 2^-24 of a number below X = |reference| + 64
    (log2; what lies further below has no weight), so a weight is off by X 2^-21 relative; its
    own rounding is 2^-8 in bf16 layers, 2^-21 in fp32 ones (exp2, factors).  Sums of the n keys
    that have weight add n 2^-24 each, numerator and weights."""
    n, new = 20000, 64
    Hq, Hkv, d = heads
    s = Step(StepCase(lens=[n], new=[new], heads=heads, dtype=dtype, block_size=block_size, width=3))
    total = n + new
    at0 = (total if step > 0 else 0)
    j = np.arange(total)
    back = np.abs(j - at0)                                 # 0 .. total: score -|step| back
    page, at = (torch.as_tensor(x).cuda() for x in s.slots(0, range(total)))
    hi, lo = (torch.from_numpy(x.astype(np.float32)).to(s.kp.dtype).cuda() for x in (back // 256, back % 256))
    s.kp[page, at, :, 0], s.kp[page, at, :, 1] = hi[:, None], lo[:, None]
    s.Qr[:] = 0
    s.Qr[..., 0], s.Qr[..., 1] = -256 * abs(step), -abs(step)
    O = f64(s.attend())
    fk.check_errors(s.ws)
    x = -abs(step) * back / np.sqrt(d)                     # exact up to here, the same for every head
    seen = np.concatenate([np.ones((new, n), bool), ancestors(s.trees[0])], 1)
    z = np.where(seen, x, -np.inf)
    p = np.exp(z - z.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    pg, a = s.slots(0, range(total))
    V = f64(s.vp)[pg, a]                                   # [keys, Hkv, d]
    V = np.repeat(V, Hq // Hkv, 1)
    want, A = np.einsum("nk,khd->nhd", p, V), np.einsum("nk,khd->nhd", p, np.abs(V))
    X = np.abs(z.max(1)) / np.log(2) + 64
    heavy = (p > 2.0 ** -40).sum(1)
    w = HALF_STEP["bf16"] if dtype == "bf16" else 2.0 ** -21
    tol = HALF_STEP[dtype] * np.abs(want) + (w + X * 2.0 ** -21 + 2 * heavy * 2.0 ** -24)[:, None, None] * A
    assert (tol <= (2.0 ** -6 if dtype == "bf16" else 2.0 ** -11) * A).all()
    err = np.abs(O - want)
    assert (err <= tol).all(), f"{(err > tol).sum()} of {err.size} off; worst {np.max(err / tol):.3g} of the tolerance"
