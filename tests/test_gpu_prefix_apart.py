"""Own keys that the plan keeps apart (decode kernels of their own from the prefix's end on, merged
with the shared part): both cache types, 128-row and few-row blocks, one split and many, at the bar
of parity.py.  Every case asserts that its plan is the form it is here for."""
import numpy as np
import pytest

import mla_synth as syn
from parity import assert_close
from prefix_problems import PrefixProblem

pytestmark = pytest.mark.gpu

BF16, FP8 = syn.KV_BF16, syn.KV_FP8_E4M3
SHORT = [3, 0, 101, 100, 102]  # sequences that end in the prefix, at it, with fewer own keys than tokens

CASES = {
    # name: ((batch, sq, heads, lens, prefix, page_size, kv_dtype, causal), key tile, splits)
    "fp8_128_rows": ((3, 1, 128, [9100, 90100, 90], 100, 16, FP8, False), 64, "many"),
    "fp8_few_rows": ((2, 2, 8, [140100, 500], 100, 64, FP8, True), 128, "many"),
    "fp8_128_rows_one_split": ((92, 1, 100, [1857 - i for i in range(90)] + [257, 0], 257, 7, FP8, False), 64, "one"),
    "fp8_few_rows_one_split": ((165, 2, 8, [1757 - i for i in range(160)] + SHORT, 101, 7, FP8, True), 128, "one"),
    "fp8_row_blocks_one_split": ((82, 2, 65, [2757 + i for i in range(80)] + [3, 258], 257, 7, FP8, True), 64, "one"),
    "bf16_128_rows_one_split": ((102, 1, 128, [1857 - i for i in range(100)] + [257, 0], 257, 16, BF16, False), 64, "one"),
    "bf16_few_rows_one_split": ((135, 1, 16, [1000 + i for i in range(130)] + SHORT, 100, 16, BF16, False), 128, "one"),
    "bf16_wide_rows_causal": ((95, 4, 12, [3070 + i for i in range(90)] + SHORT, 100, 7, BF16, True), 128, "one"),
}


def apart(p, key_tile, splits):
    plan = p.plan()
    assert plan.own_folded == 0 and plan.prefix_tiles > 0 and plan.key_tile == key_tile
    assert plan.own_splits == 1 if splits == "one" else plan.own_splits > 1
    return plan


@pytest.mark.parametrize("name", list(CASES))
def test_against_oracle(name):
    args, key_tile, splits = CASES[name]
    p = PrefixProblem(*args, seed=len(name))
    out, lse, _, status = p.run(plan=apart(p, key_tile, splits))
    assert status == 0
    assert_close(out, lse, *p.reference(), name)


@pytest.mark.parametrize("dtype", [BF16, FP8])
def test_replayed_with_shorter_contexts(dtype):
    """One split, captured; then contexts down to the prefix's end and below: out and lse are the
    shared part's alone where no own key is left."""
    import torch
    import paged_mla_decode_latent_gb300 as mla
    lens = np.asarray([1757 - i for i in range(160)], np.int32)
    p = PrefixProblem(160, 1, 8, lens, 257, 16, dtype, seed=4)
    plan = apart(p, 128, "one")
    t, ws = p.to_device(), mla.workspace_for(plan)
    out = torch.empty(160, 1, 8, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(160, 1, 8, device="cuda")
    call = lambda: mla.prefix_fwd(plan, t["q"], t["cache"], t["scale"], t["pt"], t["bt"], t["lens"],  # noqa: E731
                                  p.scale, out, lse, ws)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for new in (lens, np.maximum(257, lens - 1400), np.full(160, 257), np.arange(160) * 2):
        p.lens = new.astype(np.int32)
        t["lens"].copy_(torch.from_numpy(p.lens))
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert mla.prefix_check(plan, ws) == 0
        assert_close(out.double().cpu().numpy(), lse.double().cpu().numpy(), *p.reference(), f"{new[:3]}")


def test_contexts_beyond_the_plan_are_clamped_and_flagged():
    import paged_mla_decode_latent_gb300 as mla
    p = PrefixProblem(160, 1, 8, [1757 - i for i in range(160)], 257, 16, FP8, seed=5)
    plan, t, ref = apart(p, 128, "one"), p.to_device(), p.reference()
    t["lens"][0] = 5000  # clamped to the plan's 1757, which it holds
    out, lse, _, status = p.run(t=t, plan=plan)
    assert status == mla.DEVFLAG_CTX_RANGE
    assert_close(out, lse, *ref, "clamped")


@pytest.mark.parametrize("value", [70000.0, 2.0 ** 100])
def test_apart_large_keys_are_values(value):
    """The range rule of the decode kernels holds for own keys apart: a bf16 value beyond 65504 is one."""
    lens = [300, 290, 100, 80000]
    p = PrefixProblem(4, 1, 16, lens, 256, 16, seed=13)
    plan = apart(p, 128, "many")
    p.cache[p.block_table[1, 270 // 16], 270 % 16, 9] = syn.f32_to_bf16_bits(np.float32(value))[0]
    p.q_bits[1, 0, :, 9] = syn.f32_to_bf16_bits(np.float32(1.0 / value))[0]
    out, lse, _, status = p.run(plan=plan)
    assert status == 0
    ref, ref_lse = p.reference()
    assert np.abs(lse - ref_lse).max() <= 1e-3
    err = np.linalg.norm(out - ref, axis=-1) / np.linalg.norm(ref, axis=-1)
    assert err.max() <= 4e-3


def test_bad_pages_of_own_keys_are_flagged():
    import paged_mla_decode_latent_gb300 as mla
    p = PrefixProblem(160, 1, 8, [1757 - i for i in range(160)], 257, 16, FP8, seed=6)
    plan, t, ref = apart(p, 128, "one"), p.to_device(), p.reference()
    t["bt"][7, 40] = 1 << 29
    t["bt"][8, 3] = -7  # before the prefix's end: not read
    out, lse, _, status = p.run(t=t, plan=plan)
    assert status == mla.DEVFLAG_BAD_PAGE
    keep = [b for b in range(160) if b != 7]
    assert_close(out[keep], lse[keep], ref[0][keep], ref[1][keep], "the other sequences")
