"""The rotating epilogue against its formula in 64 bits.

Bounds: copied dims and unrotated bf16 rows are exact.  A rotated value is
fp32 arithmetic on exact inputs (two products and a sum: at most 3 * 2^-24 of
|x c| + |y s|) rounded once: half a bf16 step (2^-8 relative, eps / 2), or for
the fp8 cache the fp32 quotient (2^-24 more) and half an e4m3 step."""
import numpy as np
import pytest

import mla_synth as syn
from prefix_problems import PrefixProblem
from parity import assert_close

pytestmark = pytest.mark.gpu


def inputs(T, H, ps, fp8, seed=0, padded=0, max_pos=5000, layout="views"):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    if layout == "views":  # as the projections leave them
        q = rnd(T, H, 192)
        kv = rnd(T, 576)
        ql, qp, kc, kp = rnd(H, T, 512).transpose(0, 1), q[..., 128:], kv[:, :512], kv[:, 512:]
    elif layout == "packed":
        ql, qp, kc, kp = rnd(T, H, 512), rnd(T, H, 64), rnd(T, 512), rnd(T, 64)
    else:  # one row for every head, one row for every token
        ql, qp = rnd(T, 1, 512).expand(T, H, 512), rnd(T, 1, 64).expand(T, H, 64)
        kc, kp = rnd(1, 512).expand(T, 512), rnd(1, 64).expand(T, 64)
    pages = -(-(T + 40) // ps)
    ang = torch.arange(max_pos, dtype=torch.float64, device="cuda")[:, None] * \
        10000.0 ** (-torch.arange(32, dtype=torch.float64, device="cuda") / 32)
    cs = torch.cat([ang.cos(), ang.sin()], 1).float()
    slots = torch.randperm(pages * ps, generator=g, device="cuda")[:T]
    if padded:
        slots[torch.randperm(T, generator=g, device="cuda")[:padded]] = -1
    if fp8:
        cache = torch.randint(0, 255, (pages, ps, 576), generator=g, device="cuda").to(torch.uint8)
        scale = torch.tensor([0.0123], device="cuda")
    else:
        cache, scale = rnd(pages, ps, 576), None
    pos = torch.randint(0, max_pos, (T,), generator=g, device="cuda")
    return dict(ql=ql, qp=qp, kc=kc, kp=kp, pos=pos, cs=cs, slots=slots, cache=cache, scale=scale)


def rotated(x, cs, interleaved):
    """(value, magnitude of the two products) in 64 bits."""
    c, s = cs[..., :32], cs[..., 32:]
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :32], x[..., 32:])
    lo, hi = a * c - b * s, b * c + a * s
    mlo, mhi = np.abs(a * c) + np.abs(b * s), np.abs(b * c) + np.abs(a * s)
    if interleaved:
        return (np.stack([lo, hi], -1).reshape(x.shape), np.stack([mlo, mhi], -1).reshape(x.shape))
    return np.concatenate([lo, hi], -1), np.concatenate([mlo, mhi], -1)


def step_half(x, mant, min_exp):
    e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** min_exp)))
    return 2.0 ** (e - mant - 1)


def check(d, q_out, before, interleaved, fp8):
    import torch
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    T, H = d["qp"].shape[:2]
    cs = f(d["cs"])
    cs = cs[np.clip(d["pos"].cpu().numpy(), 0, len(cs) - 1)]  # clamped, as documented
    q = f(q_out)
    assert np.array_equal(q[..., :512], f(d["ql"]))
    ref, mag = rotated(f(d["qp"]), cs[:, None], interleaved)
    err = np.abs(q[..., 512:] - ref)
    fp32 = 3 * 2.0 ** -24 * mag
    assert np.all(err <= step_half(np.abs(ref) + fp32, 7, -126) + fp32)
    slots = d["slots"].cpu().numpy()
    kept = slots >= 0
    ref, mag = rotated(f(d["kp"]), cs, interleaved)
    fp32 = 3 * 2.0 ** -24 * mag
    row = np.concatenate([f(d["kc"]), ref], 1)[kept]
    slack = np.concatenate([np.zeros((T, 512)), fp32], 1)[kept]
    flat = d["cache"].reshape(-1, 576)
    untouched = np.ones(flat.shape[0], bool)
    untouched[slots[kept]] = False
    raw, was = flat.view(torch.uint8).cpu().numpy(), before.reshape(-1, 576).view(torch.uint8).cpu().numpy()
    assert np.array_equal(raw[untouched], was[untouched])
    if not fp8:
        got = f(flat)[slots[kept]]
        assert np.array_equal(got[:, :512], row[:, :512])
        assert np.all(np.abs(got - row) <= step_half(np.abs(row) + slack, 7, -126) + slack)
        return
    s = float(d["scale"])
    got = f(flat.view(torch.float8_e4m3fn))[slots[kept]]
    want = np.clip(row / s, -448, 448)
    slack = slack / s + 2.0 ** -24 * np.abs(want)
    assert np.all(np.abs(got - want) <= step_half(np.abs(want) + slack, 3, -6) + slack)


def call(d, interleaved, **kw):
    import torch
    import paged_mla_decode_latent_gb300 as mla
    T, H = d["qp"].shape[:2]
    q_out = torch.full((T, H, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
    mla.rope_epilogue(d["ql"], d["qp"], d["kc"], d["kp"], d["pos"], d["cs"], d["slots"], q_out,
                      d["cache"], d["scale"], interleaved=interleaved, **kw)
    return q_out


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("T,H,ps,padded,layout", [
    (1, 8, 64, 0, "views"), (1, 1, 1, 0, "packed"), (3, 128, 7, 1, "views"), (77, 12, 16, 5, "views"),
    (64, 128, 1, 0, "packed"), (65, 20, 64, 0, "expanded"), (1000, 5, 16, 999, "views"), (5, 16, 4, 5, "packed")])
def test_against_formula(T, H, ps, padded, layout, interleaved, fp8):
    d = inputs(T, H, ps, fp8, seed=T + H, padded=padded, layout=layout)
    before = d["cache"].clone()
    q = call(d, interleaved, inputs_early=bool(T % 2))
    check(d, q, before, interleaved, fp8)


def test_large_offsets():
    """A cache whose byte offsets pass 32 bits: 4.6 GB, the new rows at its end."""
    import torch
    import paged_mla_decode_latent_gb300 as mla
    d = inputs(9, 4, 16, False, seed=3)
    pages = 250_000
    cache = torch.zeros(pages, 16, 576, dtype=torch.bfloat16, device="cuda")
    d["slots"] = torch.arange(pages * 16 - 9, pages * 16, device="cuda")
    q = torch.empty(9, 4, 576, dtype=torch.bfloat16, device="cuda")
    mla.rope_epilogue(d["ql"], d["qp"], d["kc"], d["kp"], d["pos"], d["cs"], d["slots"], q, cache)
    assert torch.equal(cache.view(-1, 576)[-9:, :512], d["kc"])
    assert int((cache.view(-1, 576)[:-9] != 0).any(1).sum()) == 0


def test_flags():
    import torch
    import paged_mla_decode_latent_gb300 as mla
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    d = inputs(6, 3, 16, False, seed=1)
    d["slots"][2] = -1
    d["pos"][2] = 1 << 40  # padding: clamped, not flagged
    call(d, True, status=status)
    assert int(status) == 0
    d["pos"][1] = -7
    call(d, True, status=status)
    assert int(status) == mla.DEVFLAG_POSITION
    status.zero_()
    d["pos"][1] = 5000
    call(d, True, status=status)
    assert int(status) == mla.DEVFLAG_POSITION
    status.zero_()
    d["pos"][1] = 0
    d["slots"][4] = d["cache"].shape[0] * 16
    before = d["cache"].clone()
    q = call(d, True, status=status)
    assert int(status) == mla.DEVFLAG_BAD_PAGE
    d["slots"][4] = -1
    check(d, q, before, True, False)


def test_matches_the_plain_epilogue_at_position_zero():
    """cos 1, sin 0: every byte is mla_decode_epilogue's."""
    import torch
    import paged_mla_decode_latent_gb300 as mla
    for fp8 in (False, True):
        d = inputs(33, 16, 16, fp8, seed=2, padded=3, layout="packed")
        d["pos"].zero_()
        other = d["cache"].clone()
        q = call(d, False)
        q2 = torch.empty_like(q)
        mla.epilogue(d["ql"], d["qp"], d["kc"], d["kp"], d["slots"], q2, other, d["scale"])
        assert torch.equal(q, q2)
        assert torch.equal(d["cache"].view(torch.uint8), other.view(torch.uint8))


def test_graph_and_side_stream():
    import torch
    d = inputs(40, 16, 16, True, seed=5, padded=2)
    before = d["cache"].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    q = call(d, True, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    check(d, q, before, True, True)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q = call(d, True)
    d["pos"].add_(1)
    d["kc"].mul_(-1.0)
    d["cache"].copy_(before)
    g.replay()
    torch.cuda.synchronize()
    check(d, q, before, True, True)


# Generic scales, powers of two and sums of two (their quotients are ties often), ones whose
# reciprocal leaves the fp32 range, infinite, negative.
@pytest.mark.parametrize("scale", [0.0123, 1.0, 2.0 ** -7, 0.75, 1.0 / 448, 2.0 ** -101, 2.0 ** 101, 3e38,
                                   1e-40, float("inf"), -0.3])
def test_every_bf16_value_gets_the_code_of_its_fp32_quotient(scale):
    """Bit for bit: all 65536 values as latents of 128 tokens, NaN and infinities among them."""
    import torch
    import paged_mla_decode_latent_gb300 as mla
    d = inputs(128, 1, 16, True, seed=3, layout="packed")
    every = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).view(128, 512)
    d["kc"].copy_(every)
    d["scale"].fill_(scale)
    q = torch.empty(128, 1, 576, dtype=torch.bfloat16, device="cuda")
    mla.rope_epilogue(d["ql"], d["qp"], d["kc"], d["kp"], d["pos"], d["cs"], d["slots"], q, d["cache"], d["scale"])
    got = d["cache"].view(-1, 576)[d["slots"]][:, :512].cpu().view(torch.uint8)
    want = every.float() / torch.tensor(scale, dtype=torch.float32)
    want = torch.where(want.isnan(), want, want.clamp(-448, 448)).to(torch.float8_e4m3fn).view(torch.uint8)
    nan = want & 0x7F == 0x7F
    assert torch.equal(got & 0x7F == 0x7F, nan)
    assert torch.equal(got[~nan], want[~nan])


@pytest.mark.parametrize("fp8", [False, True])
def test_append_then_prefix_decode(fp8):
    """The two as a decode step uses them, captured: the new tokens of every sequence are rotated
    and inserted, then all rows attend to the shared prefix and to their own keys."""
    import torch
    import oracle
    import paged_mla_decode_latent_gb300 as mla
    B, Sq, H, P, ps = 5, 2, 16, 300, 16
    lens = [310, 302, 400, 331, 305]
    p = PrefixProblem(B, Sq, H, lens, P, ps, syn.KV_FP8_E4M3 if fp8 else syn.KV_BF16, True, seed=21)
    t, plan = p.to_device(), p.plan()
    ws = mla.workspace_for(plan)
    d = inputs(B * Sq, H, ps, fp8, seed=22)
    slots = torch.tensor([p.slots[b, n - Sq + i] for b, n in enumerate(lens) for i in range(Sq)],
                         dtype=torch.int64, device="cuda")
    pos = torch.tensor([n - Sq + i for n in lens for i in range(Sq)], device="cuda")
    q = torch.empty(B * Sq, H, 576, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(B, Sq, H, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(B, Sq, H, device="cuda")
    scale = t["scale"] if fp8 else None

    def step():
        mla.rope_epilogue(d["ql"], d["qp"], d["kc"], d["kp"], pos, d["cs"], slots, q, t["cache"], scale)
        mla.prefix_fwd(plan, q.view(B, Sq, H, 576), t["cache"], scale, t["pt"], t["bt"], t["lens"],
                       p.scale, out, lse, ws)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    d["qp"].mul_(-1.0)
    g.replay()
    torch.cuda.synchronize()
    assert mla.prefix_check(plan, ws) == 0
    # The reference attends with the inserted rows and the query rows as stored.
    d.update(pos=pos)
    p.q_bits = q.view(torch.int16).cpu().numpy().view(np.uint16).reshape(B, Sq, H, 576)
    c = t["cache"].cpu()
    p.cache = c.numpy() if fp8 else c.view(torch.int16).numpy().view(np.uint16)
    ref, mag = rotated(d["qp"].double().cpu().numpy(), d["cs"].double().cpu().numpy()[pos.cpu().numpy()][:, None], True)
    fp32 = 3 * 2.0 ** -24 * mag
    got = q[..., 512:].double().cpu().numpy()
    assert np.all(np.abs(got - ref) <= step_half(np.abs(ref) + fp32, 7, -126) + fp32)
    assert_close(out.double().cpu().numpy(), lse.double().cpu().numpy(), *p.reference(), "step")


@pytest.mark.parametrize("captured", [False, True])
def test_steps_back_to_back_read_what_the_step_before_left(captured):
    """Forty steps over the same buffers (rows inserted at the same slots, lengths and query rows
    rewritten) with nothing between them, against the same steps one at a time: the same bits."""
    import torch
    import paged_mla_decode_latent_gb300 as mla
    B, H, P, ps, N = 40, 16, 1000, 16, 40
    p = PrefixProblem(B, 1, H, [P + 20 + b for b in range(B)], P, ps, syn.KV_BF16, seed=23)
    t, plan = p.to_device(), p.plan()
    ws = mla.workspace_for(plan)
    g = torch.Generator(device="cuda").manual_seed(24)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    ql, qp, kc, kp = rnd(N, B, H, 512), rnd(N, B, H, 64), rnd(N, B, 512), rnd(N, B, 64)
    cs = torch.randn(5000, 64, generator=g, device="cuda")
    slots = torch.tensor([p.slots[b, P + 3] for b in range(B)], dtype=torch.int64, device="cuda")
    pos = torch.randint(0, 5000, (N, B), generator=g, device="cuda")
    lens = torch.stack([t["lens"] - int(i) for i in torch.randint(0, 20, (N,))])  # at least P + 1
    q = torch.empty(B, H, 576, dtype=torch.bfloat16, device="cuda")
    keep = t["cache"].clone()

    def steps(out, lse, wait):
        t["cache"].copy_(keep)
        for i in range(N):
            torch.add(lens[i], 0, out=t["lens"])
            mla.rope_epilogue(ql[i], qp[i], kc[i], kp[i], pos[i], cs, slots, q, t["cache"])
            mla.prefix_fwd(plan, q.view(B, 1, H, 576), t["cache"], None, t["pt"], t["bt"], t["lens"],
                           p.scale, out[i], lse[i], ws)
            if wait:
                torch.cuda.synchronize()

    new = lambda *s, dt: torch.full((N, B, 1, H, *s), float("nan"), dtype=dt, device="cuda")  # noqa: E731
    one, one_lse = new(512, dt=torch.bfloat16), new(dt=torch.float32)
    steps(one, one_lse, True)
    assert torch.isfinite(one_lse).all() and torch.isfinite(one).all()
    run, run_lse = new(512, dt=torch.bfloat16), new(dt=torch.float32)
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            steps(run, run_lse, False)
        graph.replay()
    else:
        steps(run, run_lse, False)
    torch.cuda.synchronize()
    assert mla.prefix_check(plan, ws) == 0
    assert torch.equal(run, one) and torch.equal(run_lse, one_lse)
