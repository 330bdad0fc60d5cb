"""A latent cache in 4 bits and the pages it lives in: what is timed and what is compared.

Five operators:

* ``attend``: decode attention over a paged latent cache whose rows hold 512
  e2m1 codes, 32 e4m3 scales (one for 16 dims) and 64 f16 rope dims.
* ``append``: the rotated query rows, and the insert of new tokens into that
  cache.
* ``resize``: one step of a server's page book: sequences end, grow and begin.
* ``fork``: each sequence goes on from a parent's pages (beams, samples).
* ``compact``: live pages move to the front of the cache.

``own`` false: plain torch operations in 32 bits.  ``own`` true: the
framework's entry points.  ``exact`` is the definition in 64 bits.
"""
import math
import random

import torch

own = False

DEV = "cuda"
D_QK, D_V, D_ROPE = 576, 512, 64
ROW4, SCALES, ROPE = 416, 256, 288       # bytes of a 4-bit row; where its scales and its rope dims begin
SCALE = 1.0 / math.sqrt(192.0)


def listed():
    return [
        # A handful of chats on an odd shard: 3 speculative tokens under the mask, pages of 7, one sequence empty.
        {"name": "attend_b13_h12_sq3_c999_odd", "op": "attend", "batch": 13, "heads": 12, "sq": 3, "ctx": 999,
         "page": 7, "causal": True, "ragged": True, "empty": 1},
        # One 16-head shard, a handful of short chats: latency counts.
        {"name": "attend_b4_h16_c512", "op": "attend", "batch": 4, "heads": 16, "sq": 1, "ctx": 512,
         "page": 64, "causal": False, "ragged": True, "empty": 0},
        # The same shard over long documents: what 4 bits are for.
        {"name": "attend_b8_h16_c109440", "op": "attend", "batch": 8, "heads": 16, "sq": 1, "ctx": 109440,
         "page": 64, "causal": False, "ragged": False, "empty": 0},
        # All 128 heads, batch 64, 8192 tokens, page size 1.
        {"name": "attend_b64_h128_c8192", "op": "attend", "batch": 64, "heads": 128, "sq": 1, "ctx": 8192,
         "page": 1, "causal": False, "ragged": False, "empty": 0},
        # One new token on an 8-head shard: a launch and little else.
        {"name": "append_t1_h8", "op": "append", "tokens": 1, "heads": 8, "page": 64, "interleaved": True, "padded": 0},
        # A prefill chunk of 8192 tokens, all heads, half-split rotation, padding behind it.
        {"name": "append_t8192_h128", "op": "append", "tokens": 8192, "heads": 128, "page": 16, "interleaved": False,
         "padded": 5},
        # A decode step of 64 chats: two end, two begin with a prompt, the others grow by a token.
        {"name": "resize_b64_c2000", "op": "resize", "batch": 64, "ctx": 2000, "page": 64, "tokens": 1, "ended": 2,
         "begun": 2, "spare": 1.0},
        # The same at page size 1 and 256 sequences of up to 8192 tokens, a pool that runs out.
        {"name": "resize_b256_c8192_tight", "op": "resize", "batch": 256, "ctx": 8192, "page": 1, "tokens": 4,
         "ended": 9, "begun": 11, "spare": 0.4},
        # One step of 8 beams over a short context in one layer.
        {"name": "fork_b8_c700", "op": "fork", "beams": 8, "ctx": 700, "prompt": 300, "page": 16, "layers": 1, "fp8": True},
        # One step of 64 beams over 4000 tokens, pages of 64, eight layers.
        {"name": "fork_b64_c4000", "op": "fork", "beams": 64, "ctx": 4000, "prompt": 2000, "page": 64, "layers": 8,
         "fp8": False},
        # A small pool with odd pages.
        {"name": "compact_p1111_odd", "op": "compact", "pages": 1111, "page": 7, "layers": 1, "live": 0.4, "fp8": True},
        # A big one: two layers of 16384 pages of 64 tokens, 60% live.
        {"name": "compact_p16384", "op": "compact", "pages": 16384, "page": 64, "layers": 2, "live": 0.6, "fp8": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["attend", "attend", "attend", "append", "resize", "fork", "compact"])
    page = rng.choice([1, 7, 16, 64])
    if kind == "attend":
        heads = rng.choice([rng.randint(1, 128), 8, 12, 16, 16, 20, 32, 64, 128])
        sq = rng.choice([1, 1, 2, 3, 4]) if heads <= 64 else 1
        batch = _log(rng, 1, 128)
        most = min(109440, 64 * 128 * 8192 // (batch * max(16, heads * sq)), 875520 // batch)
        return {"op": kind, "batch": batch, "heads": heads, "sq": sq, "ctx": _log(rng, sq, most), "page": page,
                "causal": sq > 1, "ragged": rng.random() < 0.6, "empty": rng.choice([0, 0, 1]) if batch > 1 else 0}
    if kind == "append":
        tokens = _log(rng, 1, 8192)
        return {"op": kind, "tokens": tokens, "heads": rng.choice([rng.randint(1, 128), 8, 16, 128]), "page": page,
                "interleaved": rng.random() < 0.5, "padded": min(rng.choice([0, 0, 1, 9]), tokens - 1)}
    if kind == "resize":
        batch = _log(rng, 2, 256)
        return {"op": kind, "batch": batch, "ctx": _log(rng, 8, 8192), "page": page, "tokens": rng.randint(1, 4),
                "ended": rng.randint(0, batch // 2), "begun": rng.randint(0, batch // 2),
                "spare": rng.choice([1.0, 1.0, 0.4])}
    if kind == "fork":
        ctx = _log(rng, 4, 4000)
        return {"op": kind, "beams": _log(rng, 2, 64), "ctx": ctx, "prompt": rng.randint(0, ctx // 2), "page": page,
                "layers": rng.randint(1, 8), "fp8": rng.random() < 0.5}
    pages = _log(rng, 16, 16384)
    return {"op": kind, "pages": pages, "page": page, "layers": rng.randint(1, 2), "live": rng.uniform(0.1, 0.9),
            "fp8": rng.random() < 0.5}


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) & 0x7FFFFFFFFFFFFFFF)


# ---------------------------------------------------------------- 4-bit rows ---

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _quantised(x, rope, kv_scale):
    """4-bit rows of latent values `x` [n, 512] and rope dims [n, 64], both in 32 bits."""
    q = (x / kv_scale).view(-1, 32, 16)
    top = q.abs().amax(2)
    s = (top / torch.full_like(top, 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)
    d = s.to(torch.float32)[..., None]
    v = torch.where(d > 0, q / d, torch.zeros_like(q))
    a = v.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = (code + 8 * (v < 0)).to(torch.uint8).view(-1, 256, 2)
    r = (rope / kv_scale).clamp(-65504.0, 65504.0).to(torch.float16)
    return torch.cat([code[..., 0] | code[..., 1] << 4, s.view(torch.uint8), r.view(torch.uint8).view(-1, 128)], 1)


def _pairs():
    """The two values of each byte of codes, as one 64-bit word of two 32-bit values."""
    one = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=DEV)
    byte = torch.arange(256, device=DEV)
    return torch.stack([one[byte & 15], one[byte >> 4]], 1).contiguous().view(torch.int64).view(-1)


def _latent(rows, pairs):
    """The values (without kv_scale) that the codes and scales of 4-bit rows [..., 416] stand for, in 32 bits."""
    v = pairs[rows[..., :SCALES].to(torch.int32)].view(torch.float32)
    s = rows[..., SCALES:ROPE].contiguous().view(torch.float8_e4m3fn).to(torch.float32)
    return (v.unflatten(-1, (32, 16)) * s[..., None]).flatten(-2)


def _rope(rows):
    return rows[..., ROPE:].contiguous().view(torch.float16)


# -------------------------------------------------------------------- attend ---

def _prepare_attend(c, g):
    B, H, Sq, ps, ctx = c["batch"], c["heads"], c["sq"], c["page"], c["ctx"]
    lens = torch.full((B,), ctx, dtype=torch.int32, device=DEV)
    if c["ragged"]:  # log-uniform up to ctx, the first one of that length
        u = torch.rand(B, generator=g, device=DEV)
        lo = float(max(Sq, ctx // 16))
        lens = torch.exp(math.log(lo) + u * (math.log(ctx + 1.0) - math.log(lo))).floor().clamp(Sq, max(Sq, ctx)).to(torch.int32)
        lens[0] = ctx
    if c["empty"]:
        lens[B - c["empty"]:] = 0
    per = -(-ctx // ps)
    pages = B * per
    table = torch.randperm(pages, generator=g, device=DEV).to(torch.int32).view(B, per)
    x = torch.randn(pages * ps, D_QK, generator=g, device=DEV)
    # Latent channels of a trained model differ in size.
    x[:, :D_V] *= torch.exp(0.3 * torch.randn(D_V, generator=g, device=DEV))
    kv_scale = (x.abs().max() / 2688.0).reshape(1)
    cache = _quantised(x[:, :D_V].contiguous(), x[:, D_V:].contiguous(), kv_scale).view(pages, ps, ROW4)
    s = {"op": "attend", "case": c, "cache": cache, "kv_scale": kv_scale, "table": table, "lens": lens, "pairs": _pairs(),
         "q": torch.randn(B, Sq, H, D_QK, generator=g, device=DEV).to(torch.bfloat16),
         "out": torch.empty(B, Sq, H, D_V, dtype=torch.bfloat16, device=DEV),
         "lse": torch.empty(B, Sq, H, dtype=torch.float32, device=DEV)}
    if own:
        import paged_mla_decode_latent_gb300 as mla
        s["plan"] = mla.plan(lens.cpu(), H, Sq, ps, mla.KV_FP4_E2M1, c["causal"])
        s["workspace"] = mla.workspace_for(s["plan"])
    return s


def _plain_attend(s):
    c, ps = s["case"], s["case"]["page"]
    q = s["q"].to(torch.float32)
    B, Sq, H, _ = q.shape
    ctx = s["lens"].to(torch.int64)
    j = torch.arange(c["ctx"], device=DEV)
    at = torch.where(j < ctx[:, None], j, 0)
    rows = s["cache"][s["table"].to(torch.int64).gather(1, at // ps), at % ps]
    keys = torch.cat([_latent(rows, s["pairs"]), _rope(rows).to(torch.float32)], -1) * s["kv_scale"]
    tok = torch.arange(Sq, device=DEV)
    seen = ctx[:, None] - Sq + tok + 1 if c["causal"] else ctx[:, None].expand(B, Sq)
    seen = seen.clamp(min=0).repeat_interleave(H, 1)
    z = torch.bmm(q.reshape(B, Sq * H, D_QK), keys.transpose(1, 2)).mul_(SCALE).masked_fill_(j >= seen[..., None], -math.inf)
    top = z.amax(2)
    w = z.sub_(top.clamp(min=-3e38)[..., None]).exp_()
    total = w.sum(2)
    o = torch.bmm(w, keys[..., :D_V]) / total.clamp(min=1e-30)[..., None]
    return {"out": o.to(torch.bfloat16).view(B, Sq, H, D_V), "lse": (top + total.log()).view(B, Sq, H)}


def _exact_attend(c, seed):
    s = prepare(c, seed)
    B, H, Sq, ps = c["batch"], c["heads"], c["sq"], c["page"]
    flat = s["cache"].view(-1, ROW4)
    value = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
    out = torch.zeros(B, Sq, H, D_V, dtype=torch.float64, device=DEV)
    lse = torch.full((B, Sq, H), -math.inf, dtype=torch.float64, device=DEV)
    for b, n in enumerate(s["lens"].tolist()):
        k = torch.arange(n, device=DEV)
        r = flat[s["table"][b][k // ps].to(torch.int64) * ps + k % ps]
        keys = torch.empty(n, D_QK, dtype=torch.float64, device=DEV)
        for half in range(2):
            nib = (r[:, :SCALES] >> (4 * half)) & 15
            keys[:, half:D_V:2] = value[(nib & 7).to(torch.int64)] * (1.0 - 2.0 * (nib >> 3).to(torch.float64))
        step = r[:, SCALES:ROPE].contiguous().view(torch.float8_e4m3fn).to(torch.float64)
        keys[:, :D_V] *= step.repeat_interleave(16, 1)
        keys[:, D_V:] = _rope(r).to(torch.float64)
        keys *= s["kv_scale"].to(torch.float64)
        for i in range(Sq):
            m = max(0, n - Sq + i + 1) if c["causal"] else n
            if m:
                z = (s["q"][b, i].to(torch.float64) @ keys[:m].t()) / math.sqrt(192.0)
                lse[b, i] = torch.logsumexp(z, 1)
                out[b, i] = torch.exp(z - lse[b, i][:, None]) @ keys[:m, :D_V]
    return {"out": out, "lse": lse}


# -------------------------------------------------------------------- append ---

def _prepare_append(c, g):
    T, H, ps = c["tokens"], c["heads"], c["page"]
    pages = -(-max(2 * T, 64) // ps)
    table = 65536
    freq = 10000.0 ** (-torch.arange(0, D_ROPE, 2, dtype=torch.float64, device=DEV) / D_ROPE)
    angle = torch.arange(table, dtype=torch.float64, device=DEV)[:, None] * freq
    cos_sin = torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32)
    # The projections as they leave their products: q is one tensor of 192 dims a head whose last 64 are
    # rotated, the latent and its rotated part are one row of 576, the absorbed query is [heads, tokens, 512].
    q = torch.randn(T, H, 192, generator=g, device=DEV).to(torch.bfloat16)
    kv = torch.randn(T, D_QK, generator=g, device=DEV).to(torch.bfloat16)
    ql = torch.randn(H, T, D_V, generator=g, device=DEV).to(torch.bfloat16)
    slots = torch.randperm(pages * ps, generator=g, device=DEV)[:T]
    if c["padded"]:
        slots[T - c["padded"]:] = -1
    x = torch.randn(pages * ps, D_QK, generator=g, device=DEV)
    kv_scale = (x.abs().max() / 2688.0).reshape(1)
    cache = _quantised(x[:, :D_V].contiguous(), x[:, D_V:].contiguous(), kv_scale).view(pages, ps, ROW4)
    return {"op": "append", "case": c, "q_pe": q[..., 128:], "ql_nope": ql.transpose(0, 1), "kv_c": kv[:, :D_V],
            "k_pe": kv[:, D_V:], "positions": torch.randint(0, table, (T,), generator=g, device=DEV),
            "cos_sin": cos_sin, "slots": slots, "cache": cache, "kv_scale": kv_scale, "pairs": _pairs(),
            "q_out": torch.empty(T, H, D_QK, dtype=torch.bfloat16, device=DEV)}


def _rotate(x, cs, interleaved):
    cos, sin = cs[..., :D_ROPE // 2], cs[..., D_ROPE // 2:]
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    a, b = x[..., :D_ROPE // 2], x[..., D_ROPE // 2:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _appended(s, q):
    """What the cache holds, as values: the codes times their scales, and the rope dims."""
    return {"q": q, "latent": _latent(s["cache"], s["pairs"]), "rope": _rope(s["cache"])}


def _plain_append(s):
    c = s["case"]
    cs = s["cos_sin"][s["positions"]]
    q_pe = _rotate(s["q_pe"].to(torch.float32), cs[:, None], c["interleaved"])
    n = c["tokens"] - c["padded"]
    row = _quantised(s["kv_c"][:n].to(torch.float32).contiguous(),
                     _rotate(s["k_pe"][:n].to(torch.float32), cs[:n], c["interleaved"]), s["kv_scale"])
    s["cache"].view(-1, ROW4)[s["slots"][:n]] = row
    return _appended(s, torch.cat([s["ql_nope"], q_pe.to(torch.bfloat16)], -1))


def _exact_append(c, seed):
    s = prepare(c, seed)
    T, half = c["tokens"], D_ROPE // 2
    cs = s["cos_sin"][s["positions"]].to(torch.float64)
    turn = torch.complex(cs[:, :half], cs[:, half:])

    def rotated(x, by):
        x = x.to(torch.float64)
        z = torch.complex(x[..., 0::2].contiguous(), x[..., 1::2].contiguous()) if c["interleaved"] else \
            torch.complex(x[..., :half].contiguous(), x[..., half:].contiguous())
        z = z * by
        return torch.view_as_real(z).flatten(-2) if c["interleaved"] else torch.cat([z.real, z.imag], -1)

    def fl32(v):  # a quotient of two 32-bit values, rounded to 32 bits (once: 53 bits are more than 2 * 24 + 2)
        return v.to(torch.float32).to(torch.float64)

    keep = s["slots"] >= 0
    by = s["kv_scale"].to(torch.float64)
    x = fl32(s["kv_c"][keep].to(torch.float64) / by).view(-1, 32, 16)
    top = fl32(x.abs().amax(2) / 6.0)
    unit = torch.exp2(torch.floor(torch.log2(top.clamp(min=2.0 ** -30))).clamp(min=-6.0) - 3.0)
    step = (torch.round(top / unit) * unit).clamp(max=448.0)             # torch.round: ties to even
    v = torch.where(step[..., None] > 0, fl32(x / step[..., None].clamp(min=2.0 ** -20)), torch.zeros_like(x))
    grid = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
    # Nearest of the grid; of two equally near ones the even code, which is made a hair nearer.
    far = (v.abs()[..., None] - grid).abs() + 1e-12 * (torch.arange(8, device=DEV) % 2)
    latent = torch.empty(*s["cache"].shape[:2], D_V, dtype=torch.float64, device=DEV)
    rope = _rope(s["cache"]).to(torch.float64)
    latent[:] = _latent(s["cache"], s["pairs"])                          # rows that the call leaves as they were
    latent.view(-1, D_V)[s["slots"][keep]] = (grid[far.argmin(-1)] * torch.sign(v) * step[..., None]).flatten(1)
    rope.view(-1, D_ROPE)[s["slots"][keep]] = rotated(s["k_pe"], turn)[keep] / by
    q = torch.empty(T, c["heads"], D_QK, dtype=torch.float64, device=DEV)
    q[..., :D_V] = s["ql_nope"]
    q[..., D_V:] = rotated(s["q_pe"], turn[:, None])
    return {"q": q, "latent": latent, "rope": rope}


# --------------------------------------------------------------------- pages ---

def _count(table, lens, ps, pages):
    """Holders of each page, from the tables."""
    j = torch.arange(table.shape[1], device=DEV)
    held = j < ((lens.to(torch.int64) + ps - 1) // ps)[:, None]
    refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
    return refs.scatter_add_(0, table[held].to(torch.int64), torch.ones(1, dtype=torch.int32, device=DEV).expand(int(held.sum())))


def _cache(c, pages, g):
    shape = (c["layers"], pages, c["page"], D_QK)
    if c["fp8"]:  # codes of all finite values
        x = torch.randint(0, 254, shape, generator=g, device=DEV, dtype=torch.uint8)
        return x + (x >= 127).to(torch.uint8)
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)


def _seen(cache):
    return cache.view(torch.float8_e4m3fn) if cache.dtype is torch.uint8 else cache


def _pages_of(lens, ps):
    return (lens.to(torch.int64) + ps - 1) // ps


def _lengths(c, n, key):
    """n lengths between half of c["ctx"] and all of it: the same ones whatever the seed."""
    r = random.Random("%s %s" % (key, sorted(c.items())))
    return [r.randint(max(1, c["ctx"] // 2), c["ctx"]) for _ in range(n)]


def _prepare_resize(c, g):
    B, ps, ctx = c["batch"], c["page"], c["ctx"]
    old = torch.tensor(_lengths(c, B, "old"), dtype=torch.int32)
    new = old + c["tokens"]
    old[:c["begun"]] = 0
    new[:c["begun"]] = torch.tensor(_lengths(c, B, "new"), dtype=torch.int32)[:c["begun"]]
    new[B - c["ended"]:] = 0
    width = -(-(ctx + c["tokens"]) // ps)
    held = int(_pages_of(old, ps).sum())
    more = int((_pages_of(new, ps) - _pages_of(old, ps)).clamp(min=0).sum())
    less = int((_pages_of(old, ps) - _pages_of(new, ps)).clamp(min=0).sum())
    pages = held + max(8, int(more * c["spare"]) - (less if c["spare"] < 1.0 else 0))
    order = torch.randperm(B, generator=g, device=DEV)  # which row does which
    old, new = old.to(DEV)[order], new.to(DEV)[order]
    pool = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.zeros(B, width, dtype=torch.int32, device=DEV)
    table[torch.arange(width, device=DEV) < _pages_of(old, ps)[:, None]] = pool[:held]
    s = {"op": "resize", "case": c, "refs0": _count(table, old, ps, pages), "table0": table, "lens0": old, "new": new,
         "slots": torch.empty(B, c["tokens"], dtype=torch.int64, device=DEV)}
    s |= {"refs": s["refs0"].clone(), "table": table.clone(), "lens": old.clone()}
    if own:
        import paged_mla_decode_latent_gb300 as mla
        s["workspace"] = mla.pages_workspace(pages, B)
    return s


def _plain_resize(s):
    c, ps, refs, table = s["case"], s["case"]["page"], s["refs"], s["table"]
    old, new = s["lens"].to(torch.int64), s["new"].to(torch.int64)
    po, pn = _pages_of(old, ps), _pages_of(new, ps)
    j = torch.arange(table.shape[1], device=DEV)
    gone = (j >= pn[:, None]) & (j < po[:, None])
    refs.scatter_add_(0, table.to(torch.int64).flatten(), -gone.flatten().to(torch.int32))
    free = (refs == 0).nonzero().flatten()
    need = (pn - po).clamp(min=0)
    end = need.cumsum(0)
    given = (need == 0) | (end <= free.numel())
    taken = (j >= po[:, None]) & (j < pn[:, None]) & given[:, None]
    page = free[((end - need)[:, None] + j - po[:, None])[taken]]
    table[taken] = page.to(torch.int32)
    refs[page] = 1
    lens = torch.where(given, new, old)
    at = lens[:, None] - c["tokens"] + torch.arange(c["tokens"], device=DEV)
    slot = table.to(torch.int64).gather(1, at.clamp(min=0) // ps) * ps + at % ps
    s["slots"].copy_(torch.where(at >= old[:, None], slot, -1))
    s["lens"].copy_(lens)


def _prepare_fork(c, g):
    B, ps, ctx = c["beams"], c["page"], c["ctx"]
    # A prompt's whole pages are shared by all beams; each beam's further pages are its own.
    shared = c["prompt"] // ps
    lens = torch.tensor(_lengths(c, B, "beams"), dtype=torch.int32, device=DEV)
    lens = lens[torch.randperm(B, generator=g, device=DEV)]
    width = -(-ctx // ps)
    held = _pages_of(lens, ps)
    pages = shared + int((held - shared).sum()) + B + 8
    pool = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.zeros(B, width, dtype=torch.int32, device=DEV)
    table[:, :shared] = pool[:shared]
    j = torch.arange(width, device=DEV)
    mine = (j >= shared) & (j < held[:, None])
    table[mine] = pool[shared:shared + int(mine.sum())]
    s = {"op": "fork", "case": c, "refs0": _count(table, lens, ps, pages), "table": table, "lens": lens,
         "parents": torch.randint(0, B, (B,), generator=g, device=DEV, dtype=torch.int32),
         "cache": _cache(c, pages, g), "table_out": torch.zeros_like(table), "lens_out": torch.zeros_like(lens)}
    s["refs"] = s["refs0"].clone()
    if own:
        import paged_mla_decode_latent_gb300 as mla
        s["workspace"] = mla.pages_workspace(pages, B)
    return s


def _plain_fork(s):
    ps, refs, cache, table = s["case"]["page"], s["refs"], s["cache"], s["table"].to(torch.int64)
    B, W = table.shape
    lens, parents = s["lens"].to(torch.int64), s["parents"].to(torch.int64)
    i, j = torch.arange(B, device=DEV), torch.arange(W, device=DEV)
    children = torch.zeros(B, dtype=torch.int64, device=DEV).scatter_add_(0, parents, torch.ones_like(parents))
    first = torch.full((B,), B, dtype=torch.int64, device=DEV).scatter_reduce_(0, parents, i, "amin")
    whole, held = lens // ps, _pages_of(lens, ps)
    change = torch.where(j < whole[:, None], children[:, None] - 1, (children[:, None] > 0).to(torch.int64) - 1)
    change = torch.where(j < held[:, None], change, 0)
    refs.scatter_add_(0, table.flatten(), change.flatten().to(torch.int32))
    part = (lens % ps)[parents]
    copies = ((part > 0) & (first[parents] != i)).nonzero().flatten()
    page = (refs == 0).nonzero().flatten()[:copies.numel()]
    source, last = parents[copies], whole[parents[copies]]
    used = (torch.arange(ps, device=DEV) < part[copies][:, None])[None, :, :, None]
    cache[:, page] = torch.where(used, cache[:, table[source, last]], cache[:, page])
    refs[page] = 1
    held_by = j < held[parents][:, None]
    s["table_out"].copy_(torch.where(held_by, table[parents], s["table_out"].to(torch.int64)))
    s["table_out"][copies, last] = page.to(torch.int32)
    s["lens_out"].copy_(lens[parents])


def _prepare_compact(c, g):
    pages, ps = c["pages"], c["page"]
    live = max(1, int(pages * c["live"]))
    B = max(1, min(64, live // 4))
    width = -(-live // B)
    pool = torch.randperm(pages, generator=g, device=DEV)[:live].to(torch.int32)
    table = torch.zeros(B, width, dtype=torch.int32, device=DEV)
    table.view(-1)[:live] = pool                 # the last rows may be shorter, or empty
    held = (live - width * torch.arange(B, device=DEV)).clamp(0, width)
    lens = (held * ps - torch.randint(0, ps, (B,), generator=g, device=DEV) * (held > 0)).to(torch.int32)
    s = {"op": "compact", "case": c, "refs0": _count(table, lens, ps, pages), "table0": table, "lens": lens,
         "cache": _cache(c, pages, g), "page_map": torch.empty(pages, dtype=torch.int32, device=DEV),
         "n_live": torch.zeros(1, dtype=torch.int32, device=DEV)}
    s |= {"refs": s["refs0"].clone(), "table": table.clone()}
    if own:
        import paged_mla_decode_latent_gb300 as mla
        s["workspace"] = mla.pages_workspace(pages, B)
    return s


def _plain_compact(s):
    ps, refs, cache, table = s["case"]["page"], s["refs"], s["cache"], s["table"]
    live = refs > 0
    p = torch.arange(refs.numel(), device=DEV)
    n = live.sum()
    hole, high = (~live & (p < n)).nonzero().flatten(), (live & (p >= n)).nonzero().flatten()
    cache[:, hole] = cache[:, high]
    s["page_map"].copy_(torch.where(live, p, -1))
    s["page_map"][high] = hole.to(torch.int32)
    refs[hole] = refs[high]
    refs[high] = 0
    held = torch.arange(table.shape[1], device=DEV) < _pages_of(s["lens"], ps)[:, None]
    table.copy_(torch.where(held, s["page_map"][table.to(torch.int64)], table))
    s["n_live"].copy_(n)


# ----------------------------------------------------------------------- all ---

def prepare(case, seed):
    return {"attend": _prepare_attend, "append": _prepare_append, "resize": _prepare_resize, "fork": _prepare_fork,
            "compact": _prepare_compact}[case["op"]](case, _gen(seed))


def run(s):
    op = s["op"]
    if own:
        import paged_mla_decode_latent_gb300 as mla
    if op == "attend":
        if not own:
            return _plain_attend(s)
        mla.fwd(s["plan"], s["q"], s["cache"], s["kv_scale"], s["table"], s["lens"], SCALE, s["out"], s["lse"], s["workspace"])
        mla.combine(s["plan"], s["lens"], s["out"], s["lse"], s["workspace"])
        return {"out": s["out"], "lse": s["lse"]}
    if op == "append":
        if not own:
            return _plain_append(s)
        mla.rope_epilogue(s["ql_nope"], s["q_pe"], s["kv_c"], s["k_pe"], s["positions"], s["cos_sin"], s["slots"],
                          s["q_out"], s["cache"], s["kv_scale"], interleaved=s["case"]["interleaved"])
        return _appended(s, s["q_out"])
    s["refs"].copy_(s["refs0"])                  # every pass starts from the same book
    if op == "resize":
        s["table"].copy_(s["table0"])
        s["lens"].copy_(s["lens0"])
        if own:
            mla.pages_resize(s["refs"], s["table"], s["lens"], s["new"], s["case"]["page"], s["workspace"], s["slots"])
        else:
            _plain_resize(s)
        return {"refs": s["refs"], "table": s["table"], "lens": s["lens"], "slots": s["slots"]}
    if op == "fork":
        if own:
            mla.pages_fork(s["refs"], s["table"], s["lens"], s["parents"], s["table_out"], s["lens_out"], s["cache"],
                           s["workspace"])
        else:
            _plain_fork(s)
        return {"refs": s["refs"], "table": s["table_out"], "lens": s["lens_out"], "cache": _seen(s["cache"])}
    s["table"].copy_(s["table0"])
    if own:
        mla.pages_compact(s["refs"], s["table"], s["lens"], s["cache"], s["page_map"], s["n_live"], s["workspace"])
    else:
        _plain_compact(s)
    return {"refs": s["refs"], "table": s["table"], "map": s["page_map"], "n_live": s["n_live"], "cache": _seen(s["cache"])}


def work(case):
    c = case
    if c["op"] == "attend":
        B, rows, ctx = c["batch"], c["heads"] * c["sq"], float(c["ctx"])
        lo = float(max(c["sq"], c["ctx"] // 16))
        mean = ctx if not c["ragged"] or ctx <= lo else (ctx - lo) / math.log(ctx / lo)    # of a log-uniform length
        keys = ctx + (B - 1 - c["empty"]) * mean if B > c["empty"] else 0.0
        return {"bytes": int(keys * (ROW4 + 4 / c["page"]) + B * rows * (D_QK * 2 + D_V * 2 + 4)),
                "flops": int(2 * (D_QK + D_V) * rows * keys)}
    if c["op"] == "append":
        T, H = c["tokens"], c["heads"]
        # q in and out; the row in and out; the rotation's row, the position and the slot; the values read back.
        slots = -(-max(2 * T, 64) // c["page"]) * c["page"]
        return {"bytes": 2 * T * H * D_QK * 2 + T * D_QK * 2 + (T - c["padded"]) * ROW4 + T * (256 + 16)
                + slots * (ROW4 + 4 * D_V + 2 * D_ROPE), "flops": 6 * 32 * T * (H + 1) + 4 * D_V * T}
    if c["op"] == "resize":
        B, ps = c["batch"], c["page"]
        held = 0.75 * c["ctx"] * B / ps
        moved = 0.75 * c["ctx"] * (c["ended"] + c["begun"]) / ps + B * c["tokens"] / ps
        # The book is set back (refs and tables read and written); refs read, the changed entries and refs written.
        return {"bytes": int(held * (8 + 8 + 4) + moved * 8 + B * (8 + 4 * 4 + 8 * c["tokens"])), "flops": 0}
    row = D_QK * (1 if c["fp8"] else 2)
    if c["op"] == "fork":
        B, ps = c["beams"], c["page"]
        copies = B * (1 - 0.632) * (ps - 1) / max(1, ps)          # beams that share a parent's partly filled page
        entries = 0.75 * c["ctx"] * B / ps
        return {"bytes": int(2 * copies * c["layers"] * row * ps / 2 + entries * (4 + 4 + 8 + 8)), "flops": 0}
    moves = c["pages"] * c["live"] * (1 - c["live"])
    return {"bytes": int(2 * moves * c["layers"] * c["page"] * row + c["pages"] * (8 + 8 + 4 + 16 * c["live"])), "flops": 0}


def exact(case, seed):
    if case["op"] == "attend":
        return _exact_attend(case, seed)
    return _exact_append(case, seed) if case["op"] == "append" else None  # whole numbers and rows moved as they are
