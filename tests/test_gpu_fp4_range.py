"""Queries beyond f16 over a 4-bit cache: they are flagged, and such a row never looks like one without keys."""
import numpy as np
import pytest

import fp4_rows as f4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,sq", [(16, 1), (32, 1), (64, 1), (128, 1), (100, 2)])
@pytest.mark.parametrize("num_sms", [0, 2])  # several splits, one
@pytest.mark.parametrize("value", [-70000.0, 70000.0, float("-inf")])
def test_a_query_whose_scores_are_all_infinite_is_no_empty_row(heads, sq, num_sms, value):
    """+-70000 times keys that are positive there: f16 makes every score infinite, and the row NaN."""
    import torch
    import paged_mla_decode_latent_gb300 as mla
    p = f4.Fp4Problem(3, sq, heads, [1300, 0, 77], 16, sq > 1, seed=17)
    p.cache[:, :, 2] = 0x22  # dims 4 and 5: 1 times the block's scale
    p.cache[:, :, 256] = np.where(p.cache[:, :, 256] == 0x7F, 0x7F, 0x38)
    t = p.to_device()
    good, good_l, _, status = p.run(num_sms, t)
    assert status == 0
    t["q"][0, 0, 3, 5] = value
    out, lse, _, status = p.run(num_sms, t)
    assert status == mla.DEVFLAG_Q_RANGE
    assert np.isnan(out[0, 0, 3]).all() and np.isnan(lse[0, 0, 3])
    out[0, 0, 3], lse[0, 0, 3] = good[0, 0, 3], good_l[0, 0, 3]
    assert np.array_equal(out, good) and np.array_equal(lse, good_l)  # the other rows, and those without a key
    assert np.all(out[1] == 0) and np.all(np.isneginf(lse[1]))


@pytest.mark.parametrize("heads", [16, 128])
def test_rows_that_the_mask_leaves_nothing_stay_empty_beside_it(heads):
    """More tokens than keys: the first ones see none, also where a later one is beyond f16."""
    import paged_mla_decode_latent_gb300 as mla
    p = f4.Fp4Problem(1, 4, heads, [2], 16, True, seed=18)
    p.cache[:, :, 2] = 0x22
    t = p.to_device()
    t["q"][0, :, 3, 5] = -70000.0
    out, lse, _, status = p.run(0, t)
    assert status == mla.DEVFLAG_Q_RANGE
    assert np.all(out[0, :2] == 0) and np.all(np.isneginf(lse[0, :2]))
    assert np.isnan(out[0, 2:, 3]).all() and np.isnan(lse[0, 2:, 3]).all()


@pytest.mark.parametrize("heads", [16, 128])
def test_a_planned_on_the_device_call_says_so_too(heads):
    import torch
    import paged_mla_decode_latent_gb300 as mla
    p = f4.Fp4Problem(2, 1, heads, [2100, 300], 16, seed=19)
    p.cache[:, :, 2] = 0x22
    t = p.to_device()
    t["q"][1, 0, 0, 4] = -70000.0
    d = mla.dplan_info(2, heads, 1, 16, mla.KV_FP4_E2M1, False, int(p.table.shape[1]) * 16)
    ws = mla.workspace_for(d)
    out, lse = torch.empty(2, 1, heads, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 1, heads, device="cuda")
    mla.plan_device(d, t["lens"], ws)
    mla.fwd_dplan(d, t["q"], t["cache"], t["scale"], t["bt"], p.scale, out, lse, ws)
    mla.combine_dplan(d, out, lse, ws)
    assert mla.dplan_check(d, ws) == mla.DEVFLAG_Q_RANGE
    assert out[1, 0, 0].isnan().all() and lse[1, 0, 0].isnan()
    assert out[1, 0, 1:].isfinite().all() and out[0].isfinite().all()
