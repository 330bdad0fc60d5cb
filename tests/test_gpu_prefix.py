"""The shared-prefix decode against the fp64 oracle on the same bits, at the
bar of parity.py: the pass over the shared keys, the merge with each sequence's
own keys, the masks and the walk of the CTA pairs over row blocks."""
import numpy as np
import pytest

import mla_synth as syn
from parity import assert_close
from prefix_problems import PrefixProblem

pytestmark = pytest.mark.gpu

BF16, FP8 = syn.KV_BF16, syn.KV_FP8_E4M3

CASES = {
    # name: (batch, sq, heads, lens, prefix, page_size, kv_dtype, causal)
    "one_key": (1, 1, 1, [1], 1, 1, BF16, False),
    "one_row_one_own_key": (1, 1, 1, [2], 1, 1, BF16, False),
    "tile_minus_one": (2, 1, 16, [255, 300], 255, 16, BF16, False),
    "tile": (2, 1, 16, [256, 257], 256, 16, BF16, False),
    "tile_plus_one": (2, 1, 16, [257, 258], 257, 16, BF16, False),
    "h128": (3, 1, 128, [700, 701, 900], 700, 1, BF16, False),
    "h128_one_block_short": (1, 1, 100, [1300], 1200, 16, BF16, False),
    "h16_b20_fp8": (20, 1, 16, [1000 + 7 * i for i in range(20)], 1000, 64, FP8, False),
    "h128_fp8": (2, 1, 128, [640, 530], 512, 64, FP8, False),
    "odd_pages": (13, 3, 12, [4999 + 1 + 25 * i for i in range(13)], 4999, 7, FP8, True),
    "causal_mtp": (5, 4, 16, [520, 604, 513, 530, 777], 512, 16, BF16, True),
    # Sequences shorter than the prefix, shorter than the tokens, empty, just at it.
    "short_sequences": (8, 4, 16, [0, 2, 5, 255, 300, 511, 512, 516], 512, 16, BF16, True),
    "short_sequences_unmasked": (4, 1, 40, [0, 1, 300, 700], 640, 16, BF16, False),
    "all_empty": (3, 1, 16, [0, 0, 0], 64, 16, BF16, False),
    "no_prefix": (3, 1, 16, [40, 0, 129], 0, 16, BF16, False),
    "no_own_keys": (4, 1, 64, [600] * 4, 600, 1, BF16, False),
    "long_own": (2, 1, 128, [3300, 400], 300, 16, BF16, False),
    "rows_two_blocks_a_sequence": (2, 2, 128, [900, 850], 800, 16, BF16, True),
    "blocks_across_sequences": (9, 3, 20, [700 + 9 * i for i in range(9)], 700, 16, BF16, True),
    "one_row_sequences": (150, 1, 1, [300 + i % 7 * 30 for i in range(150)], 300, 16, FP8, False),
    "own_apart": (3, 1, 128, [100 + 9000, 100 + 90000, 90], 100, 16, BF16, False),
    "own_apart_few_rows": (2, 2, 8, [100 + 140000, 100 + 400], 100, 64, BF16, True),
    "rows_200_a_sequence": (5, 2, 100, [420 + 60 * i for i in range(5)], 400, 16, BF16, True),
    "own_exact_tiles": (2, 1, 128, [512 + 256, 512 + 512], 512, 16, BF16, False),
}


@pytest.mark.parametrize("name", list(CASES))
def test_against_oracle(name):
    p = PrefixProblem(*CASES[name], seed=len(name))
    out, lse, plan, status = p.run()
    assert status == 0
    assert_close(out, lse, *p.reference(), name)


@pytest.mark.parametrize("num_sms", [2, 4, 6, 10, 38, 152])
def test_pairs_and_segments(num_sms):
    """One pair walks every row block; more cut row blocks at odd tiles."""
    p = PrefixProblem(5, 1, 128, [1500 + i for i in range(5)], 1450, 1, seed=3)
    ref = p.reference()
    out, lse, plan, status = p.run(num_sms=num_sms)
    assert status == 0 and plan.pairs <= num_sms // 2
    assert_close(out, lse, *ref, f"{plan.pairs} pairs")


def test_plan_of_every_pair_count():
    """Any pair count gives the same rows, within the bar: the merge of cut row blocks."""
    p = PrefixProblem(3, 1, 100, [2100, 2090, 2400], 2080, 16, seed=5)
    ref, t = p.reference(), p.to_device()
    for sms in range(2, 56, 6):
        out, lse, plan, status = p.run(t=t, num_sms=sms)
        assert status == 0
        assert_close(out, lse, *ref, f"sms {sms}, {plan.pairs} pairs")


@pytest.mark.parametrize("heads,sq,dtype", [(16, 4, BF16), (128, 1, BF16), (16, 1, FP8)])
def test_outlier_keys(heads, sq, dtype):
    p = PrefixProblem(6, sq, heads, [2300 + 30 * i for i in range(6)], 2222, 16, dtype, sq > 1,
                      seed=11, outlier_frac=0.01)
    out, lse, plan, status = p.run()
    assert status == 0
    assert_close(out, lse, *p.reference(), "outliers")


def test_running_maximum_is_rescaled():
    """Scores that climb by far more than the lag from tile to tile."""
    p = PrefixProblem(2, 1, 128, [1300, 1290], 1280, 1, seed=2)
    ramp = np.linspace(0.02, 3.0, 1280, dtype=np.float32)
    f = syn.bf16_bits_to_f32(p.cache)
    q0 = syn.bf16_bits_to_f32(p.q_bits)[0, 0, 0]
    for j in range(1280):  # key j leans on the first row's query more and more
        f[p.prefix_table[j], 0] += ramp[j] * q0
    p.cache = syn.f32_to_bf16_bits(f)
    out, lse, plan, status = p.run()
    assert status == 0
    ref = p.reference()
    assert ref[1].max() > 100  # the climb is there
    assert_close(out, lse, *ref, "ramp")


@pytest.mark.parametrize("scale", [0.0, 2.0 ** -10, 0.5])
def test_scales(scale):
    p = PrefixProblem(3, 1, 32, [300, 100, 270], 260, 16, seed=4, scale=scale, q_mult=0.25)
    out, lse, _, status = p.run()
    assert status == 0
    assert_close(out, lse, *p.reference(), f"scale {scale}")


def test_same_as_the_decode_without_sharing():
    """The documented equality: the plain decode on tables that hold the prefix."""
    import torch
    import paged_mla_decode_latent_gb300 as mla
    p = PrefixProblem(4, 2, 16, [700, 650, 649, 800], 640, 16, causal=True, seed=8)
    t = p.to_device()
    out, lse, _, _ = p.run(t=t)
    full = t["bt"].clone()
    full[:, :40] = t["pt"]
    o2, l2 = mla.decode(t["q"], t["cache"], full, t["lens"], softmax_scale=p.scale, causal=True)
    assert_close(out, lse, o2.double().cpu().numpy(), l2.double().cpu().numpy(), "decode")
    o3, l3 = mla.decode_prefix(t["q"], t["cache"], full[0], full, t["lens"], 640,
                               softmax_scale=p.scale, causal=True)
    torch.cuda.synchronize()
    assert np.array_equal(o3.double().cpu().numpy(), out) and np.array_equal(l3.double().cpu().numpy(), lse)


def test_deterministic_and_workspace_reuse():
    import torch
    import paged_mla_decode_latent_gb300 as mla
    p = PrefixProblem(9, 1, 64, [3000 + i for i in range(9)], 2950, 16, seed=6)
    t, plan = p.to_device(), p.plan()
    ws = torch.full((int(plan.workspace_bytes),), 255, dtype=torch.uint8, device="cuda")
    a = p.run(t=t, plan=plan, workspace=ws)
    b = p.run(t=t, plan=plan, workspace=ws)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
    assert_close(a[0], a[1], *p.reference(), "reuse")
    assert mla.prefix_check(plan, ws) == 0


def test_graph_replay_with_new_lengths():
    """Captured once; the lengths, the queries and the cache change under it."""
    import torch
    import paged_mla_decode_latent_gb300 as mla
    big = PrefixProblem(6, 1, 128, [1400, 1280, 1100, 1350, 1281, 1290], 1280, 16, seed=9)
    t, plan = big.to_device(), big.plan()
    ws = mla.workspace_for(plan)
    out = torch.empty(6, 1, 128, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(6, 1, 128, device="cuda")
    call = lambda: mla.prefix_fwd(plan, t["q"], t["cache"], None, t["pt"], t["bt"], t["lens"],  # noqa: E731
                                  big.scale, out, lse, ws)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for lens in ([1400, 1280, 1100, 1350, 1281, 1290], [1290, 0, 1100, 1281, 1281, 700],
                 [1, 1280, 1000, 1300, 1281, 1285]):
        big.lens = np.asarray(lens, np.int32)
        t["lens"].copy_(torch.from_numpy(big.lens))
        t["q"].mul_(-1.0)
        big.q_bits = big.q_bits ^ np.uint16(0x8000)
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert mla.prefix_check(plan, ws) == 0
        assert_close(out.double().cpu().numpy(), lse.double().cpu().numpy(), *big.reference(), f"{lens}")


def test_side_stream():
    import torch
    import paged_mla_decode_latent_gb300 as mla
    p = PrefixProblem(3, 1, 64, [600, 610, 590], 580, 16, seed=10)
    t, plan = p.to_device(), p.plan()
    ws = mla.workspace_for(plan)
    out = torch.empty(3, 1, 64, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(3, 1, 64, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    mla.prefix_fwd(plan, t["q"], t["cache"], None, t["pt"], t["bt"], t["lens"], p.scale, out, lse,
                   ws, stream=s)
    assert mla.prefix_check(plan, ws, stream=s) == 0
    assert_close(out.double().cpu().numpy(), lse.double().cpu().numpy(), *p.reference(), "stream")


def test_bad_pages_and_contexts_are_flagged():
    import paged_mla_decode_latent_gb300 as mla
    p = PrefixProblem(4, 1, 16, [600, 610, 590, 640], 580, 16, seed=12)
    t, plan = p.to_device(), p.plan()
    t["pt"][3] = 1 << 28
    assert p.run(t=t, plan=plan)[3] & mla.DEVFLAG_BAD_PAGE
    t = p.to_device()
    t["bt"][2, 36] = -5
    out, lse, _, status = p.run(t=t, plan=plan)
    assert status & mla.DEVFLAG_BAD_PAGE
    ref = p.reference()
    keep = [0, 1, 3]
    assert_close(out[keep], lse[keep], ref[0][keep], ref[1][keep], "the other sequences")
    t = p.to_device()
    t["lens"][1] = 100000  # clamped to the plan's 640: the table has no page there for it
    t["bt"][1, 38:] = t["bt"][1, 37]
    t["lens"][0] = -3
    out, lse, _, status = p.run(t=t, plan=plan)
    assert status & mla.DEVFLAG_CTX_RANGE
    assert np.all(out[0] == 0) and np.all(np.isneginf(lse[0]))
    assert_close(out[2:], lse[2:], ref[0][2:], ref[1][2:], "the other sequences")


@pytest.mark.parametrize("value", [70000.0, float("nan"), float("-inf")])
@pytest.mark.parametrize("fold", [True, False])
def test_keys_beyond_f16_spoil_the_rows_that_see_them(value, fold):
    """A shared key: every row that sees it; an own key: its sequence's rows.  The others stay."""
    import paged_mla_decode_latent_gb300 as mla
    lens = [300, 290, 100, 280] if fold else [300, 290, 100, 80000]
    p = PrefixProblem(4, 1, 16, lens, 256, 16, seed=13)
    ref, t, plan = p.reference(), p.to_device(), p.plan()
    assert plan.own_folded == fold
    keep = t["cache"].clone()
    t["cache"][int(p.prefix_table[200 // 16]), 200 % 16, 9] = value  # the third sequence has 100 keys
    out, lse, _, status = p.run(t=t, plan=plan)
    assert status == mla.DEVFLAG_KV_RANGE
    for b in (0, 1, 3):
        assert np.isnan(out[b]).all() and np.isnan(lse[b]).all()
    assert_close(out[2], lse[2], ref[0][2], ref[1][2], "too short to see it")
    if fold:
        t["cache"].copy_(keep)
        t["cache"][int(p.block_table[1, 270 // 16]), 270 % 16, 575] = value
        out, lse, _, status = p.run(t=t, plan=plan)
        assert status == mla.DEVFLAG_KV_RANGE
        assert np.isnan(out[1]).all() and np.isnan(lse[1]).all()
        for b in (0, 2, 3):
            assert_close(out[b], lse[b], ref[0][b], ref[1][b], "another sequence")


def test_a_causal_token_before_a_bad_key_stays():
    import paged_mla_decode_latent_gb300 as mla
    p = PrefixProblem(3, 3, 16, [300, 290, 280], 256, 16, causal=True, seed=16)
    ref, t = p.reference(), p.to_device()
    t["cache"][int(p.block_table[1, 289 // 16]), 289 % 16, 0] = float("inf")  # the last token's key
    out, lse, _, status = p.run(t=t)
    assert status == mla.DEVFLAG_KV_RANGE
    assert np.isnan(out[1, 2]).all()
    for b, i in ((0, 0), (0, 2), (1, 0), (1, 1), (2, 2)):
        assert_close(out[b, i], lse[b, i], ref[0][b, i], ref[1][b, i], f"{b} {i}")


@pytest.mark.parametrize("value", [70000.0, float("nan"), float("inf")])
@pytest.mark.parametrize("prefix,sms", [(256, 0), (256, 2), (3000, 0)])
def test_queries_beyond_f16_spoil_their_row(value, prefix, sms):
    """NaN, not an empty row's zeros; in a whole row block and in a cut one."""
    import paged_mla_decode_latent_gb300 as mla
    p = PrefixProblem(2, 1, 16, [prefix + 44, prefix + 34], prefix, 16, seed=13)
    ref, t = p.reference(), p.to_device()
    t["q"][1, 0, 3, 5] = value
    out, lse, _, status = p.run(t=t, num_sms=sms)
    assert status == mla.DEVFLAG_Q_RANGE
    assert np.isnan(out[1, 0, 3]).all() and np.isnan(lse[1, 0, 3])
    rest = [h for h in range(16) if h != 3]
    assert_close(out[1, 0, rest], lse[1, 0, rest], ref[0][1, 0, rest], ref[1][1, 0, rest], "the other heads")
    assert_close(out[0], lse[0], ref[0][0], ref[1][0], "the other sequence")


@pytest.mark.parametrize("prefix,sms,own", [(256, 0, 44), (256, 2, 44), (3000, 0, 44), (3000, 0, 0), (1, 0, 0)])
def test_a_query_whose_scores_are_all_minus_infinity_is_no_empty_row(prefix, sms, own):
    """-70000 times keys that are positive there: f16 makes every score -inf, and the row NaN."""
    import paged_mla_decode_latent_gb300 as mla
    p = PrefixProblem(2, 1, 16, [prefix + own, 0], prefix, 16, seed=17)
    t = p.to_device()
    t["cache"][:, :, 5] = 1.0
    t["q"][0, 0, 3, 5] = -70000.0
    out, lse, _, status = p.run(t=t, num_sms=sms)
    assert status == mla.DEVFLAG_Q_RANGE
    assert np.isnan(out[0, 0, 3]).all() and np.isnan(lse[0, 0, 3])
    rest = [h for h in range(16) if h != 3]
    assert np.isfinite(out[0, 0, rest]).all() and np.isfinite(lse[0, 0, rest]).all()
    assert np.all(out[1] == 0) and np.all(np.isneginf(lse[1]))  # no key: still empty


def test_small_values():
    """Below 2^-14 the staged values keep an absolute 2^-25: q and cache scaled down."""
    p = PrefixProblem(2, 1, 64, [400, 380], 300, 1, seed=14, q_mult=2.0 ** -9)
    out, lse, _, status = p.run()
    assert status == 0
    assert_close(out, lse, *p.reference(), "small q")


def test_a_wait_that_runs_out():
    """A 1 us limit ends every long wait; the call reports it and the next one is whole."""
    import paged_mla_decode_latent_gb300 as mla
    p = PrefixProblem(16, 1, 128, [4096 + 64] * 16, 4096, 16, seed=15)
    t, plan = p.to_device(), p.plan()
    ws = mla.workspace_for(plan)
    plan.wait_limit_us = 1
    assert p.run(t=t, plan=plan, workspace=ws)[3] & mla.DEVFLAG_TIMEOUT
    plan.wait_limit_us = 0
    out, lse, _, status = p.run(t=t, plan=plan, workspace=ws)
    assert status == 0
    assert_close(out, lse, *p.reference(), "after the timeout")


@pytest.mark.parametrize("seed", range(16))
def test_random_shapes(seed):
    """Heads, tokens, pages, types, prefixes and ragged, short and empty contexts drawn at random."""
    rng = np.random.default_rng(1000 + seed)
    heads = int(rng.choice([1, 3, 8, 16, 20, 33, 64, 100, 128]))
    sq = int(rng.integers(1, 5)) if heads <= 100 else int(rng.integers(1, 3))
    batch = int(rng.integers(1, 9))
    prefix = int(np.exp(rng.uniform(0, np.log(1500))))
    own = int(np.exp(rng.uniform(0, np.log(700))))
    lens = prefix + rng.integers(0, own + 1, batch)
    if seed % 3 == 0:
        lens[int(rng.integers(batch))] = int(rng.integers(0, prefix + 1))
    p = PrefixProblem(batch, sq, heads, lens, prefix, int(rng.choice([1, 5, 16, 64])),
                      FP8 if rng.random() < 0.4 else BF16, bool(rng.random() < 0.6), seed=seed,
                      outlier_frac=0.01 if rng.random() < 0.3 else 0.0)
    ref, t = p.reference(), p.to_device()
    for sms in (0, int(rng.integers(2, 40))):
        out, lse, plan, status = p.run(t=t, num_sms=sms)
        assert status == 0
        assert_close(out, lse, *ref, f"seed {seed} {plan.as_dict()}")


def test_many_row_blocks():
    """40960 query rows: 320 row blocks, more than the partition keeps in registers."""
    p = PrefixProblem(320, 1, 128, [64 + i % 5 for i in range(320)], 64, 16, seed=17)
    out, lse, plan, status = p.run()
    assert status == 0 and plan.row_blocks == 320
    assert_close(out, lse, *p.reference(), "320 row blocks")


def test_long_prefix():
    """70001 shared keys, against the formula in 64 bits on the GPU."""
    import torch
    p = PrefixProblem(3, 1, 16, [70001, 70040, 69000], 70001, 64, FP8, seed=18)
    out, lse, _, status = p.run()
    assert status == 0
    flat = torch.from_numpy(p.cache).view(torch.float8_e4m3fn).cuda().reshape(-1, 576)
    q = torch.from_numpy(p.q_bits.view(np.int16)).view(torch.bfloat16).cuda().double()
    for b in range(3):
        k = flat[torch.from_numpy(p.slots[b, :p.lens[b]].astype(np.int64)).cuda()].double() * p.kv_scale
        z = q[b, 0] @ k.t() * p.scale
        ref_l = torch.logsumexp(z, 1)
        ref_o = torch.exp(z - ref_l[:, None]) @ k[:, :512]
        assert_close(out[b, 0], lse[b, 0], ref_o.cpu().numpy(), ref_l.cpu().numpy(), f"sequence {b}")


def test_cache_beyond_4_gb():
    """Pages whose byte offsets pass 32 bits, shared and own."""
    import torch
    import paged_mla_decode_latent_gb300 as mla
    p = PrefixProblem(2, 1, 16, [300, 333], 290, 16, seed=19)
    t, plan = p.to_device(), p.plan()
    n, shift = t["cache"].shape[0], 240_000
    big = torch.zeros(shift + n, 16, 576, dtype=torch.bfloat16, device="cuda")
    big[shift:] = t["cache"]
    t["cache"] = big
    t["pt"] += shift
    t["bt"][t["bt"] >= 0] += shift
    out, lse, _, status = p.run(t=t, plan=plan)
    assert status == 0
    assert_close(out, lse, *p.reference(), "far pages")


def test_two_streams_at_once():
    """Two calls in flight, each with its workspace."""
    import torch
    import paged_mla_decode_latent_gb300 as mla
    ps = [PrefixProblem(6, 1, 128, [2000 + 7 * i for i in range(6)], 1990, 16, seed=20 + k) for k in range(2)]
    ts, plans = [p.to_device() for p in ps], [p.plan() for p in ps]
    wss = [mla.workspace_for(x) for x in plans]
    outs = [torch.empty(6, 1, 128, 512, dtype=torch.bfloat16, device="cuda") for _ in ps]
    lses = [torch.empty(6, 1, 128, device="cuda") for _ in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    for _ in range(5):
        for k, p in enumerate(ps):
            mla.prefix_fwd(plans[k], ts[k]["q"], ts[k]["cache"], None, ts[k]["pt"], ts[k]["bt"],
                           ts[k]["lens"], p.scale, outs[k], lses[k], wss[k], stream=streams[k])
    for k, p in enumerate(ps):
        assert mla.prefix_check(plans[k], wss[k], stream=streams[k]) == 0
        assert_close(outs[k].double().cpu().numpy(), lses[k].double().cpu().numpy(), *p.reference(), f"stream {k}")


def test_contexts_are_flagged_without_a_prefix_too():
    import paged_mla_decode_latent_gb300 as mla
    for lens in ([40, 60], [0, 0]):
        p = PrefixProblem(2, 1, 16, lens, 0, 16, seed=23)
        t, plan = p.to_device(), p.plan()
        t["lens"][1] = 61
        assert p.run(t=t, plan=plan)[3] == mla.DEVFLAG_CTX_RANGE
        t["lens"][1] = -1
        out, lse, _, status = p.run(t=t, plan=plan)
        assert status == mla.DEVFLAG_CTX_RANGE
        assert np.all(out[1] == 0) and np.all(np.isneginf(lse[1]))


def test_refusals_of_the_binding():
    import torch
    import paged_mla_decode_latent_gb300 as mla
    p = PrefixProblem(2, 1, 16, [300, 290], 256, 16, seed=24)
    plan = p.plan()
    good = p.to_device()
    out = torch.empty(2, 1, 16, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(2, 1, 16, device="cuda")
    ws = mla.workspace_for(plan)

    def call(**kw):
        a = dict(good, out=out, lse=lse, ws=ws)
        a.update(kw)
        mla.prefix_fwd(plan, a["q"], a["cache"], None, a["pt"], a["bt"], a["lens"], p.scale, a["out"],
                       a["lse"], a["ws"])

    call()
    bad = [dict(q=good["q"].float()), dict(q=good["q"][:1]), dict(q=good["q"].cpu()),
           dict(q=good["q"].expand(2, 1, 16, 576).transpose(0, 2).contiguous().transpose(0, 2)),
           dict(cache=good["cache"][:, :8]), dict(cache=good["cache"].to(torch.float16)),
           dict(pt=good["pt"][:15]), dict(pt=good["pt"].long()), dict(pt=None), dict(bt=None),
           dict(bt=good["bt"][:, :18]), dict(bt=good["bt"][:1]), dict(lens=good["lens"].long()),
           dict(lens=good["lens"][:1]), dict(out=out.float()), dict(lse=lse.half()), dict(out=out[..., :511])]
    for kw in bad:
        with pytest.raises(mla.MLADecodeError) as e:
            call(**kw)
        assert e.value.status == mla.ERR_INVALID_ARG, kw
    with pytest.raises(mla.MLADecodeError) as e:
        call(ws=ws[:1000])
    assert e.value.status == mla.ERR_WORKSPACE


@pytest.mark.parametrize("before", ["nothing", "copy", "kernel", "fill", "join of two kernels",
                                    "join of a kernel and a copy", "event of a kernel"])
def test_captured_behind(before):
    """The call as the first work after other nodes of a graph, which write its inputs."""
    import torch
    import paged_mla_decode_latent_gb300 as mla
    p = PrefixProblem(5, 1, 16, [1024 + 3 * b for b in range(5)], 1024, 16, seed=29)
    t, plan = p.to_device(), p.plan()
    ws = mla.workspace_for(plan)
    out = torch.full((5, 1, 16, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((5, 1, 16), float("nan"), device="cuda")
    q, lens = t["q"].clone(), t["lens"].clone()
    main, side = torch.cuda.Stream(), torch.cuda.Stream()

    def work():
        if before.startswith("join"):
            side.wait_stream(main)
            with torch.cuda.stream(side):
                t["lens"].copy_(lens) if before.endswith("copy") else torch.add(lens, 0, out=t["lens"])
            torch.mul(q, 1.0, out=t["q"])
            main.wait_stream(side)
        elif before == "event of a kernel":
            side.wait_stream(main)
            with torch.cuda.stream(side):
                torch.mul(q, 1.0, out=t["q"])
                torch.add(lens, 0, out=t["lens"])
            main.wait_stream(side)
        else:
            if before in ("kernel", "fill"):
                torch.mul(q, 1.0, out=t["q"])
            if before == "fill":
                out.zero_()
            if before == "copy":
                t["q"].copy_(q)
                t["lens"].copy_(lens)
        mla.prefix_fwd(plan, t["q"], t["cache"], None, t["pt"], t["bt"], t["lens"], p.scale, out, lse, ws)

    main.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(main):
        work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        work()
    if before not in ("nothing", "kernel", "fill"):
        t["lens"].fill_(7)
    if before != "nothing":
        t["q"].zero_()
    out.fill_(float("nan"))
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert mla.prefix_check(plan, ws) == 0
    assert_close(out.double().cpu().numpy(), lse.double().cpu().numpy(), *p.reference(), before)


@pytest.mark.parametrize("heads,planned", [(16, [3000]), (16, [900, 40, 2000, 700, 10, 0, 1500, 300, 299]), (128, [2500, 1])])
def test_contexts_shorter_than_the_plan_leave_pairs_without_work(heads, planned):
    """Planned with long own keys and hardly any shared ones, called with short contexts, down to empty."""
    import paged_mla_decode_latent_gb300 as mla
    batch = len(planned)
    plan = mla.prefix_plan([1 + n for n in planned], 1, heads, 1, 16, BF16, False, 0)
    assert plan.own_folded and plan.pairs > plan.row_blocks * 3  # the units of the shared keys alone
    width = -(-(1 + max(planned)) // 16)
    for lens in ([1] * batch, [0] * batch, [1 + b % 2 for b in range(batch)], [1 + min(n, 40) for n in planned],
                 [1 + n for n in planned]):
        p = PrefixProblem(batch, 1, heads, lens, 1, 16, seed=31)
        t = p.to_device()
        if t["bt"].shape[1] < width:  # entries past a sequence's last page are not read
            t["bt"] = torch_pad(t["bt"], width)
        out, lse, _, status = p.run(t=t, plan=plan)
        assert status == 0
        assert_close(out, lse, *p.reference(), f"{lens}")


def torch_pad(bt, width):
    import torch
    return torch.nn.functional.pad(bt, (0, width - bt.shape[1]), value=-1).contiguous()
