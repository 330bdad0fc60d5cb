"""The 4-bit cache on the GPU: the decode in all its forms and the inserts, against 64 bits.

The decode's bounds are those of parity.py: its arithmetic is the fp8 cache's (f16 operands that hold every code times
its scale exactly, f16 weights, fp32 sums), on rows of the same size."""
import numpy as np
import pytest

import fp4_rows as f4
import mla_synth as syn
from parity import assert_close

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch,sq,heads,lens,page,causal", [
    (1, 1, 1, [1], 1, False), (1, 1, 16, [64], 64, False), (2, 1, 16, [129, 128], 7, False),
    (3, 1, 16, [300, 0, 77], 16, False), (2, 2, 8, [31, 33], 16, True), (1, 16, 1, [5], 3, True),
    (2, 1, 17, [65, 64], 1, False), (2, 1, 128, [63, 1], 16, False), (1, 3, 12, [500], 7, True),
    (2, 4, 16, [2, 4], 64, True), (1, 2, 128, [190], 16, True), (1, 16, 64, [97], 4096, True),
    (4, 1, 20, [1, 2, 3, 4], 1, False), (1, 1, 16, [4097], 64, False), (1, 1, 128, [2049], 1, False),
    (2, 1, 32, [1000, 127], 16, False), (2, 2, 16, [385, 2], 16, True), (2, 1, 33, [200, 64], 16, False),
    (3, 8, 4, [7, 9, 257], 1, True), (1, 4, 8, [3], 16, True), (1, 1, 25, [129], 5, False)])
@pytest.mark.parametrize("num_sms", [0, 8])
def test_decode(batch, sq, heads, lens, page, causal, num_sms):
    p = f4.Fp4Problem(batch, sq, heads, lens, page, causal, seed=len(lens) + heads)
    out, lse, plan, status = p.run(num_sms)
    assert status == 0
    assert_close(out, lse, *p.reference(), f"{plan.num_splits} splits")


@pytest.mark.parametrize("heads", [16, 128])
def test_every_code_and_scale(heads):
    p = f4.Fp4Problem(2, 1, heads, [260, 131], 16, seed=5, raw=True)
    p.scale = 0.02  # scores near 1
    out, lse, _, status = p.run()
    assert status == 0
    ref, ref_l = p.reference()
    assert np.isfinite(ref).all()
    # Each weight is rounded to f16 (2^-11) and each output to bf16 (2^-8); the fp32 sums of weights and
    # scores are far below.  With w the rounded weights the output moves by 2^-11 sum w |v| at most; 2^-10 for
    # the two roundings of a weight and its share of the sum.
    for b in range(2):
        keys = np.abs(p.keys(b)[:, :512]).max()
        tol = np.abs(ref[b]) * 2.0 ** -8 + keys * 2.0 ** -10
        assert (np.abs(out[b] - ref[b]) <= tol).all()
    assert np.abs(lse - ref_l).max() <= 1e-3


@pytest.mark.parametrize("heads,sq", [(16, 1), (32, 2)])
def test_outliers_many_splits(heads, sq):
    p = f4.Fp4Problem(3, sq, heads, [3000, 1, 2222], 16, sq > 1, seed=9, outliers=0.02)
    out, lse, plan, status = p.run()
    assert status == 0 and plan.num_splits > 1
    assert_close(out, lse, *p.reference(), "outliers")


@pytest.mark.parametrize("heads,sq", [(16, 1), (40, 3)])
@pytest.mark.parametrize("csr", [False, True])
def test_planned_on_the_device(heads, sq, csr):
    import torch
    import paged_mla_decode_latent_gb300 as mla
    p = f4.Fp4Problem(4, sq, heads, [700, 0, 15, 2100], 16, sq > 1, seed=11)
    t = p.to_device()
    d = mla.dplan_info(4, heads, sq, 16, mla.KV_FP4_E2M1, p.causal, int(p.table.shape[1]) * 16)
    ws = mla.workspace_for(d)
    out = torch.empty(4, sq, heads, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(4, sq, heads, device="cuda")
    table, indptr = t["bt"], None
    if csr:
        counts = -(-p.lens // 16)
        indptr = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
        table = torch.from_numpy(np.concatenate([p.table[b, :n] for b, n in enumerate(counts)])).cuda()
    mla.plan_device(d, t["lens"], ws, indptr)
    mla.fwd_dplan(d, t["q"], t["cache"], t["scale"], table, p.scale, out, lse, ws, indptr)
    mla.combine_dplan(d, out, lse, ws)
    assert mla.dplan_check(d, ws) == 0
    assert_close(out.double().cpu().numpy(), lse.double().cpu().numpy(), *p.reference(), "device plan")


def test_decode_and_noalloc_are_the_three_calls():
    import ctypes
    import torch
    import paged_mla_decode_latent_gb300 as mla
    p = f4.Fp4Problem(2, 1, 16, [900, 333], 64, seed=2)
    t = p.to_device()
    out, lse, plan, _ = p.run(t=t)
    o, l = mla.decode(t["q"], t["cache"], t["bt"], t["lens"], kv_scale=t["scale"], softmax_scale=p.scale)
    assert np.array_equal(o.double().cpu().numpy(), out) and np.array_equal(l.double().cpu().numpy(), lse)
    o.zero_()
    ptr = lambda x: ctypes.c_void_p(x.data_ptr())  # noqa: E731
    st = mla.lib().mla_decode_fwd_noalloc(ctypes.byref(plan), ptr(t["q"]), ptr(t["cache"]), t["cache"].shape[0], ptr(t["scale"]),
                                          ptr(t["bt"]), t["bt"].stride(0), ptr(t["lens"]), p.scale, ptr(o), ptr(l), None)
    torch.cuda.synchronize()
    assert st == 0 and np.array_equal(o.double().cpu().numpy(), out)


def test_bad_pages_and_lengths_are_flagged():
    import torch
    import paged_mla_decode_latent_gb300 as mla
    p = f4.Fp4Problem(2, 1, 16, [300, 200], 16, seed=3)
    t = p.to_device()
    good, _, _, _ = p.run(t=t)
    t["bt"][0, 2] = p.cache.shape[0] + 5
    out, _, _, status = p.run(t=t)
    assert status == mla.DEVFLAG_BAD_PAGE and np.array_equal(out[1], good[1]) and np.isfinite(out).all()
    t = p.to_device()
    t["lens"][1] = 301
    plan = mla.plan(p.lens, 16, 1, 16, mla.KV_FP4_E2M1)
    ws = mla.workspace_for(plan)
    o = torch.empty(2, 1, 16, 512, dtype=torch.bfloat16, device="cuda")
    t["bt"][1] = t["bt"][0]
    mla.fwd(plan, t["q"], t["cache"], t["scale"], t["bt"], t["lens"], p.scale, o, torch.empty(2, 1, 16, device="cuda"), ws)
    assert mla.check(plan, ws) == mla.DEVFLAG_CTX_RANGE


@pytest.mark.parametrize("heads", [16, 128])
@pytest.mark.parametrize("at", [7, 30])  # a block of either CTA's half
@pytest.mark.parametrize("n", [100, 700])  # one split, several
def test_a_nan_scale_spoils_the_sequence_that_holds_it(heads, at, n):
    p = f4.Fp4Problem(2, 1, heads, [n, n - 10], 16, seed=4)
    good, _, _, _ = p.run()
    p.cache[p.table[1, 2], 3, 256 + at] = 0x7F
    out, lse, _, status = p.run()
    assert status == 0 and np.isnan(out[1]).all() and np.isnan(lse[1]).all() and np.array_equal(out[0], good[0])


# What a key's rope adds to every score, by its place in the sequence: the running maximum rises with most tiles, with
# the keys of one CTA's half of a 256-key tile only, once by much, never after the first key.
RAMPS = {"up": lambda j: j / 20.0, "up in the first half": lambda j: np.where(j % 256 < 128, j / 20.0, 0.0),
         "up in the second half": lambda j: np.where(j % 256 >= 128, j / 20.0, 0.0),
         "a jump": lambda j: np.where(j == 700, 100.0, 0.0), "down": lambda j: np.where(j == 0, 80.0, 0.0)}


@pytest.mark.parametrize("heads,sq", [(16, 1), (32, 1), (64, 1), (128, 1), (100, 2)])
@pytest.mark.parametrize("ramp", RAMPS)
def test_running_maximum(heads, sq, ramp):
    p = f4.Fp4Problem(2, sq, heads, [1300, 801], 16, sq > 1, seed=8)
    p.q_bits[..., 512:] = 0
    p.q_bits[..., 512] = 0x4280  # 64
    unit = 64.0 * p.scale * p.kv_scale
    for b in range(2):
        j = np.arange(p.lens[b])
        rope = np.zeros((p.lens[b], 64), np.float16)
        rope[:, 0] = RAMPS[ramp](j) / unit
        p.cache[p.table[b, j // 16], j % 16, 288:] = rope.view(np.uint8)
    for num_sms in (0, 2):  # several splits, one
        out, lse, plan, status = p.run(num_sms)
        assert status == 0
        assert_close(out, lse, *p.reference(), f"{ramp}, {plan.num_splits} splits")


@pytest.mark.parametrize("heads,sq,lens", [(33, 1, [255, 256, 257]), (64, 1, [1, 128, 129]), (65, 1, [512, 3, 400]),
                                           (128, 8, [700, 20, 16]), (43, 3, [130, 0, 5])])
def test_row_blocks(heads, sq, lens):
    p = f4.Fp4Problem(3, sq, heads, lens, 16, sq > 1, seed=10)
    for num_sms in (0, 2):
        out, lse, plan, status = p.run(num_sms)
        assert status == 0
        assert_close(out, lse, *p.reference(), f"{plan.num_splits} splits")


@pytest.mark.parametrize("heads", [40, 128])
def test_waits_of_a_pair_run_out_without_a_fault(heads):
    """With a bound of 1 us the waits of both CTAs of a pair give up, and the next call is right."""
    test_waits_run_out_without_a_fault(heads)


@pytest.mark.parametrize("heads", [16, 32])
def test_waits_run_out_without_a_fault(heads):
    """With a bound of 1 us the pipeline's waits give up, the call says so, and the next one is right."""
    import ctypes
    import torch
    import paged_mla_decode_latent_gb300 as mla
    p = f4.Fp4Problem(4, 1, heads, [4096] * 4, 16, seed=12)
    t = p.to_device()
    plan = mla.plan(p.lens, heads, 1, 16, mla.KV_FP4_E2M1)
    ws = mla.workspace_for(plan)
    short = mla.Plan.from_buffer_copy(plan)
    short.wait_limit_us = 1
    out, lse = torch.zeros(4, 1, heads, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(4, 1, heads, device="cuda")
    for pl in (short, plan):
        mla.fwd(pl, t["q"], t["cache"], t["scale"], t["bt"], t["lens"], p.scale, out, lse, ws)
        mla.combine(pl, t["lens"], out, lse, ws)
        v = ctypes.c_int32(0)
        st = mla.lib().mla_decode_check(ctypes.byref(pl), ctypes.c_void_p(ws.data_ptr()), mla._stream(None), ctypes.byref(v))
        if pl is short:
            assert st == mla.ERR_TIMEOUT and v.value & mla.DEVFLAG_TIMEOUT
        else:
            assert st == 0
    assert_close(out.double().cpu().numpy(), lse.double().cpu().numpy(), *p.reference(), "after a call that gave up")


def inputs(tokens, heads, seed, values=None):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    t = {"ql": rnd(tokens, heads, 512), "qp": rnd(tokens, heads, 64), "kc": rnd(tokens, 512), "kp": rnd(tokens, 64)}
    if values is not None:
        t["kc"].copy_(values)
    return t


def latent_values(tokens):
    """Blocks of 16 where the definition has its edges: zeros, a lone value, borders of codes and scales, tiny and huge
    values, infinities, NaN."""
    import torch
    rng = np.random.default_rng(1)
    x = rng.standard_normal((tokens, 32, 16))
    x[:, 0] = 0.0
    x[:, 1] = 0.0
    x[:, 1, 3] = -1.0
    x[:, 2] = np.array([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, -6])
    x[:, 3] = np.linspace(-6, 6, 16)
    x[:, 4] *= 1e-30
    x[:, 5] *= 1e30
    x[:, 6] = 2.0 ** -9 * 6 * np.linspace(0.25, 0.5, 16)  # scales around the least one's half
    x[:, 7, 5] = np.inf
    x[:, 8, 9] = -np.inf
    x[:, 9, 15] = np.nan
    x[:, 10, 0] = np.nan
    return torch.from_numpy(x.reshape(tokens, 512)).to(torch.bfloat16)


@pytest.mark.parametrize("tokens,heads,page", [(1, 8, 64), (77, 12, 7), (300, 1, 16), (5, 128, 1)])
@pytest.mark.parametrize("kv_scale", [1.0, 0.0017, 3.0, 1e-38, 1e38])
@pytest.mark.parametrize("rotated", [False, True])
def test_insert(tokens, heads, page, kv_scale, rotated):
    import torch
    import paged_mla_decode_latent_gb300 as mla
    t = inputs(tokens, heads, 3, latent_values(tokens))
    pages = -(-2 * tokens // page)
    cache = torch.randint(0, 256, (pages, page, 416), dtype=torch.uint8, device="cuda")
    before = cache.cpu().numpy().reshape(-1, 416).copy()
    slots = torch.randperm(pages * page, device="cuda")[:tokens]
    slots[tokens // 2] = -1
    q = torch.empty(tokens, heads, 576, dtype=torch.bfloat16, device="cuda")
    scale = torch.tensor([kv_scale], device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    if rotated:  # by quarters of a turn, so that the rotated values are whole inputs again
        cs = torch.zeros(4, 64, device="cuda")
        cs[torch.arange(4), :32] = torch.tensor([1., 0., -1., 0.], device="cuda")[:, None]
        cs[torch.arange(4), 32:] = torch.tensor([0., 1., 0., -1.], device="cuda")[:, None]
        pos = torch.randint(0, 4, (tokens,), device="cuda")
        mla.rope_epilogue(t["ql"], t["qp"], t["kc"], t["kp"], pos, cs, slots, q, cache, scale, interleaved=False, status=status)
        c, s = cs[pos, :32].double(), cs[pos, 32:].double()
        k = t["kp"].double()
        rope = torch.cat([k[:, :32] * c - k[:, 32:] * s, k[:, 32:] * c + k[:, :32] * s], 1).cpu().numpy()
    else:
        mla.epilogue(t["ql"], t["qp"], t["kc"], t["kp"], slots, q, cache, scale, status=status)
        rope = t["kp"].double().cpu().numpy()
        assert torch.equal(q, torch.cat([t["ql"], t["qp"]], 2))
    assert int(status) == 0
    at = slots.cpu().numpy()
    rows = f4.encode(t["kc"].double().cpu().numpy(), rope, kv_scale)
    before[at[at >= 0]] = rows[at >= 0]
    got = cache.cpu().numpy().reshape(-1, 416)
    # -0 and +0 are one value: their codes may differ in the sign.
    assert np.array_equal(got[:, 256:288], before[:, 256:288])
    assert np.array_equal(got[:, :256], before[:, :256])
    a, b = (np.ascontiguousarray(x[:, 288:]).view(np.float16) for x in (got, before))
    assert np.array_equal(a, b, equal_nan=True)


def test_insert_skips_slots_out_of_range():
    import torch
    import paged_mla_decode_latent_gb300 as mla
    t = inputs(3, 4, 1)
    cache = torch.zeros(2, 16, 416, dtype=torch.uint8, device="cuda")
    q, status = torch.empty(3, 4, 576, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    scale = torch.ones(1, device="cuda")
    mla.epilogue(t["ql"], t["qp"], t["kc"], t["kp"], torch.tensor([32, -1, 5], device="cuda"), q, cache, scale, status=status)
    assert int(status) == mla.DEVFLAG_BAD_PAGE
    assert (cache.view(32, 416).any(1).nonzero().flatten().cpu() == torch.tensor([5])).all()


@pytest.mark.parametrize("heads,sq", [(16, 1), (64, 2)])
def test_step_is_insert_then_decode(heads, sq):
    import torch
    import paged_mla_decode_latent_gb300 as mla
    p = f4.Fp4Problem(3, sq, heads, [500, 40, 129], 16, sq > 1, seed=6, poison=False)
    t = p.to_device()
    T = 3 * sq
    x = inputs(T, heads, 8)
    slots = np.array([int(p.table[b, (n - sq + i) // 16]) * 16 + (n - sq + i) % 16 for b, n in enumerate(map(int, p.lens))
                      for i in range(sq)])
    plan = mla.plan(p.lens, heads, sq, 16, mla.KV_FP4_E2M1, p.causal)
    ws = mla.workspace_for(plan)
    q = torch.empty(3, sq, heads, 576, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.empty(3, sq, heads, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(3, sq, heads, device="cuda")
    args = (x["ql"], x["qp"], x["kc"], x["kp"], torch.from_numpy(slots).cuda())
    mla.step(plan, *args, q, t["cache"], t["scale"], t["bt"], t["lens"], p.scale, out, lse, ws)
    assert mla.check(plan, ws) == 0
    p.cache.reshape(-1, 416)[slots] = f4.encode(x["kc"].double().cpu().numpy(), x["kp"].double().cpu().numpy(), p.kv_scale)
    p.q_bits = torch.cat([x["ql"], x["qp"]], 2).view(torch.int16).cpu().numpy().view(np.uint16).reshape(3, sq, heads, 576)
    assert_close(out.double().cpu().numpy(), lse.double().cpu().numpy(), *p.reference(), "step")


def test_captured_and_replayed_on_another_stream():
    import torch
    import paged_mla_decode_latent_gb300 as mla
    p = f4.Fp4Problem(2, 1, 16, [700, 90], 64, seed=7)
    t = p.to_device()
    want, want_l, plan, _ = p.run(t=t)
    ws, s = mla.workspace_for(plan), torch.cuda.Stream()
    out, lse = torch.zeros(2, 1, 16, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 1, 16, device="cuda")
    g = torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        mla.fwd(plan, t["q"], t["cache"], t["scale"], t["bt"], t["lens"], p.scale, out, lse, ws)
        mla.combine(plan, t["lens"], out, lse, ws)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(out.double().cpu().numpy(), want) and np.array_equal(lse.double().cpu().numpy(), want_l)


def test_calls_that_do_not_take_4_bit_rows():
    import torch
    import paged_mla_decode_latent_gb300 as mla
    p = f4.Fp4Problem(2, 1, 16, [40, 30], 16, seed=1)
    t = p.to_device()
    bf = dict(dtype=torch.bfloat16, device="cuda")
    k, v, status = torch.zeros(70, 2, 192, **bf), torch.zeros(70, 2, 128, **bf), torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 40, 70], dtype=torch.int32, device="cuda")
    with pytest.raises(mla.MLADecodeError) as e:
        mla.gather_kv_b_proj(t["cache"], t["scale"], t["bt"], t["lens"], cu, 40, torch.zeros(2, 256, 512, **bf), k, v, status)
    assert e.value.status == mla.ERR_UNSUPPORTED
    with pytest.raises(mla.MLADecodeError):
        mla.decode_prefix(t["q"], t["cache"], t["bt"][0, :1].contiguous(), t["bt"], t["lens"], 16, kv_scale=t["scale"])
    ql, qp, kc, kp = (torch.zeros(s, **bf) for s in ((2, 16, 512), (2, 16, 64), (2, 512), (2, 64)))
    slots = torch.arange(2, device="cuda")
    for cache in (t["cache"][:, ::2], t["cache"][None]):  # strided, one layer too many
        with pytest.raises(mla.MLADecodeError):
            mla.epilogue(ql, qp, kc, kp, slots, torch.zeros(2, 16, 576, **bf), cache, t["scale"])


@pytest.mark.parametrize("heads", [16, 64, 128])
def test_steps_one_after_another_on_a_cache_16_bytes_off(heads):
    """Each step inserts a token and decodes right behind the insert, over a cache that begins between two sectors; the
    row before the new one was read by the step before."""
    import torch
    import paged_mla_decode_latent_gb300 as mla
    B, page, first, n = 3, 16, [30, 300, 511], 6
    p = f4.Fp4Problem(B, 1, heads, [m + n for m in first], page, False, seed=13, poison=False)
    t = p.to_device()
    flat = torch.zeros(t["cache"].numel() + 16, dtype=torch.uint8, device="cuda")
    cache = flat[16:].view(t["cache"].shape)
    cache.copy_(t["cache"])
    for b, m in enumerate(first):  # what the steps write is not there yet
        for j in range(m, m + n):
            cache[int(p.table[b, j // page]), j % page] = 0x7F
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    plan = mla.plan(p.lens, heads, 1, page, mla.KV_FP4_E2M1)
    ws, out = mla.workspace_for(plan), torch.empty(B, 1, heads, 512, dtype=torch.bfloat16, device="cuda")
    lse, q, got = torch.empty(B, 1, heads, device="cuda"), torch.empty(B, heads, 576, dtype=torch.bfloat16, device="cuda"), []
    for k in range(n):
        ql, qp, kc, kp = rnd(B, heads, 512), rnd(B, heads, 64), rnd(B, 512), rnd(B, 64)
        lens = torch.tensor([m + k + 1 for m in first], dtype=torch.int32, device="cuda")
        slots = torch.tensor([int(p.table[b, (m + k) // page]) * page + (m + k) % page for b, m in enumerate(first)], device="cuda")
        mla.step(plan, ql, qp, kc, kp, slots, q, cache, t["scale"], t["bt"], lens, p.scale, out, lse, ws)
        got.append((q.clone(), out.double().cpu().numpy(), lse.double().cpu().numpy()))
    assert mla.check(plan, ws) == 0
    p.cache = cache.cpu().numpy()
    for k, (qk, o, l) in enumerate(got):
        p.q_bits, p.lens = qk.view(torch.int16).cpu().numpy().view(np.uint16).reshape(B, 1, heads, 576), np.array([m + k + 1 for m in first], np.int32)
        assert_close(o, l, *p.reference(), f"step {k}")
