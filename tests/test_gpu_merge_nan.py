"""The merge on partials set by hand, in a plan of every cache: a NaN split makes its row NaN, also where no other split
has keys; rows without keys stay empty."""
import numpy as np
import pytest

import paged_mla_decode_latent_gb300 as mla

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv_dtype", [mla.KV_BF16, mla.KV_FP8_E4M3, mla.KV_FP4_E2M1])
@pytest.mark.parametrize("heads", [16, 128])
def test_nan_partials(kv_dtype, heads):
    import torch
    plan = mla.plan([4000, 3000], heads, 1, 16, kv_dtype)
    B, S = 2, plan.num_splits
    assert S > 2
    rng = np.random.default_rng(heads)
    part = rng.standard_normal((B, S, heads, 512)).astype(np.float32)
    lse = rng.uniform(-3, 3, (B, S, heads)).astype(np.float32)
    nan, none = np.float32("nan"), np.float32("-inf")
    lse[0, :, 1] = nan            # every split
    lse[0, :, 2], lse[0, S - 1, 2] = none, nan  # the one that has keys
    lse[1, 1, 3] = nan            # one of several
    lse[1, :, 4] = none           # no keys at all
    lse[1, 1:, 5] = none          # one split has keys
    part[lse == none] = nan       # what is never read
    w = np.exp(lse.astype(np.float64))
    total = w.sum(1, keepdims=True)
    with np.errstate(all="ignore"):
        want_l = np.log(total[:, 0])
        share = np.where(total > 0, w / total, np.where(np.isnan(total), np.nan, 0.0))
    want = (share[..., None] * np.where(w[..., None] == 0, 0.0, part.astype(np.float64))).sum(1)
    ws = mla.workspace_for(plan)
    for x, at in ((part, plan.ws_partial_o_offset), (lse, plan.ws_partial_lse_offset)):
        ws[at:at + x.nbytes] = torch.from_numpy(x.reshape(-1).view(np.uint8)).cuda()
    out, got_l = torch.zeros(B, 1, heads, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(B, 1, heads, device="cuda")
    mla.combine(plan, torch.tensor([4000, 3000], dtype=torch.int32, device="cuda"), out, got_l, ws)
    out, got_l = out.double().cpu().numpy()[:, 0], got_l.double().cpu().numpy()[:, 0]
    bad = np.isnan(want_l)
    assert bad.sum() == 3 and np.array_equal(np.isnan(got_l), bad)
    assert np.array_equal(np.isnan(out).all(2), bad) and np.array_equal(np.isnan(out).any(2), bad)
    assert np.array_equal(np.isneginf(got_l), np.isneginf(want_l)) and (out[1, 4] == 0).all()
    ok = np.isfinite(want_l)
    # lse: S terms and the logarithm in fp32, of values below 16 in size: an absolute (S + 4) 2^-24 of the sum, 2^-20 of
    # the result.  out: bf16 rounding (2^-8 of the value), S + 4 fp32 roundings of the sum of |w o|, at most max |o|.
    assert np.abs(got_l[ok] - want_l[ok]).max() <= (S + 4) * 2.0 ** -24 + 2.0 ** -19
    most = np.nanmax(np.abs(part))
    assert (np.abs(out[ok] - want[ok]) <= np.abs(want[ok]) * 2.0 ** -8 + (S + 8) * 2.0 ** -23 * most).all()
