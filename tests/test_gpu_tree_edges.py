"""Attention of trees at the edges of its definition, on the GPU: rows that nothing
is left for."""

import pytest
import torch

from rag_kv_cache_rerotate_gb300 import fusekv as fk

from step_ops import Step, StepCase

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
