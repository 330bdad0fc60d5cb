"""The append and the shared-prefix decode as a generation loop runs them: one plan with room for the
steps to come, contexts that grow into it, and past it."""
import numpy as np
import pytest

import mla_synth as syn
from parity import assert_close
from prefix_problems import PrefixProblem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("prefix,start", [(300, [303, 300, 301, 340]), (250, [250] * 4)])
def test_steps_up_to_the_plan_and_past_it(fp8, prefix, start):
    import torch
    import paged_mla_decode_latent_gb300 as mla
    B, H, ps, room = 4, 16, 16, 7
    p = PrefixProblem(B, 1, H, [n + room for n in start], prefix, ps, syn.KV_FP8_E4M3 if fp8 else syn.KV_BF16, seed=5)
    t, scale = p.to_device(), None
    if fp8:
        scale = t["scale"]
    plan = mla.prefix_plan([n + room for n in start], prefix, H, 1, ps, p.kv_dtype)
    ws = mla.workspace_for(plan)
    g = torch.Generator(device="cuda").manual_seed(6)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    cs = torch.randn(1000, 64, generator=g, device="cuda")
    q = torch.empty(B, H, 576, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(B, 1, H, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(B, 1, H, device="cuda")
    for k in range(1, room + 1):
        lens = np.asarray([n + k for n in start], np.int32)
        pos = torch.from_numpy(lens.astype(np.int64) - 1).cuda()
        slots = torch.tensor([int(p.slots[b, n - 1]) for b, n in enumerate(lens)], device="cuda")
        t["lens"].copy_(torch.from_numpy(lens))
        mla.rope_epilogue(rnd(B, H, 512), rnd(B, H, 64), rnd(B, 512), rnd(B, 64), pos, cs, slots, q, t["cache"], scale)
        mla.prefix_fwd(plan, q.view(B, 1, H, 576), t["cache"], scale, t["pt"], t["bt"], t["lens"], p.scale, out, lse, ws)
        assert mla.prefix_check(plan, ws) == 0
        p.lens = lens
        p.q_bits = q.view(torch.int16).cpu().numpy().view(np.uint16).reshape(B, 1, H, 576)
        c = t["cache"].cpu()
        p.cache = c.numpy() if fp8 else c.view(torch.int16).numpy().view(np.uint16)
        ref = p.reference()
        assert_close(out.double().cpu().numpy(), lse.double().cpu().numpy(), *ref, f"step {k}")
    # One more: the longest context is cut off at the plan's, and reported.
    t["lens"][start.index(max(start))] += 1
    mla.prefix_fwd(plan, q.view(B, 1, H, 576), t["cache"], scale, t["pt"], t["bt"], t["lens"], p.scale, out, lse, ws)
    assert mla.prefix_check(plan, ws) == mla.DEVFLAG_CTX_RANGE
    assert_close(out.double().cpu().numpy(), lse.double().cpu().numpy(), *ref, "past the plan")
