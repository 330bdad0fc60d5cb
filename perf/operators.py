"""The serving operators around a shared prefix: what is timed and what is compared.

Two operators of the paged latent cache:

* ``prefix``: decode attention for a batch whose sequences share their first
  ``prefix_len`` tokens.  The shared keys are scored by the query rows of the
  whole batch at once; each sequence's own keys follow; the two are one softmax.
* ``append``: the insert of new tokens into the paged cache with the position
  rotation applied on the way, together with the rotated query rows.

``own`` false: plain torch operations in 32 bits.  ``own`` true: the
framework's entry points.  ``exact`` is the definition in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
D_QK, D_V, D_ROPE = 576, 512, 64
SCALE = 1.0 / math.sqrt(192.0)


def listed():
    return [
        # A handful of chats behind a short system prompt on a 16-head shard: latency counts.
        {"name": "prefix_b4_h16_p512", "op": "prefix", "batch": 4, "heads": 16, "sq": 1, "prefix": 512,
         "suffix": 64, "page": 64, "fp8": False, "causal": False, "outliers": False},
        # One head-parallel shard, long shared document, fp8 cache, 64-key pages.
        {"name": "prefix_b32_h16_p32000_fp8", "op": "prefix", "batch": 32, "heads": 16, "sq": 1, "prefix": 32000,
         "suffix": 1024, "page": 64, "fp8": True, "causal": False, "outliers": False},
        # All 128 heads, batch 64, a prompt of 8192 tokens at page size 1.
        {"name": "prefix_b64_h128_p8192", "op": "prefix", "batch": 64, "heads": 128, "sq": 1, "prefix": 8192,
         "suffix": 512, "page": 1, "fp8": False, "causal": False, "outliers": False},
        # Speculative tokens under the causal mask, 1% outlier rows in the cache.
        {"name": "prefix_b32_h16_sq4_p8192", "op": "prefix", "batch": 32, "heads": 16, "sq": 4, "prefix": 8192,
         "suffix": 256, "page": 16, "fp8": False, "causal": True, "outliers": True},
        # Odd everything: 13 sequences, 12 heads, 3 tokens, pages of 7 keys, a prefix that ends inside a page.
        {"name": "prefix_odd_b13_h12_sq3_p4999_fp8", "op": "prefix", "batch": 13, "heads": 12, "sq": 3, "prefix": 4999,
         "suffix": 333, "page": 7, "fp8": True, "causal": True, "outliers": False},
        # The largest: 128 sequences of 128 heads behind 23333 shared tokens.
        {"name": "prefix_b128_h128_p23333", "op": "prefix", "batch": 128, "heads": 128, "sq": 1, "prefix": 23333,
         "suffix": 512, "page": 16, "fp8": False, "causal": False, "outliers": False},
        # One new token on an 8-head shard: a launch and little else.
        {"name": "append_t1_h8", "op": "append", "tokens": 1, "heads": 8, "page": 64, "fp8": False,
         "interleaved": True, "padded": 0},
        # A decode step of 64 sequences, all heads, fp8 cache.
        {"name": "append_t64_h128_fp8", "op": "append", "tokens": 64, "heads": 128, "page": 1, "fp8": True,
         "interleaved": True, "padded": 0},
        # An odd step: half-split rotation, pages of 7, padding tokens behind the batch.
        {"name": "append_t77_h12_padded", "op": "append", "tokens": 77, "heads": 12, "page": 7, "fp8": False,
         "interleaved": False, "padded": 5},
        # A prefill chunk of 8192 tokens, all heads.
        {"name": "append_t8192_h128", "op": "append", "tokens": 8192, "heads": 128, "page": 16, "fp8": False,
         "interleaved": True, "padded": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.6:
        heads = rng.choice([rng.randint(1, 128), 8, 12, 16, 20, 32, 64, 96, 128])
        sq = rng.choice([1, 1, 2, 3, 4]) if heads <= 64 else 1
        batch = _log(rng, 1, 128)
        rows = batch * heads * sq
        return {"op": "prefix", "batch": batch, "heads": heads, "sq": sq,
                "prefix": min(_log(rng, 1, 65536), 128 * 128 * 23333 // rows), "suffix": _log(rng, sq, 1024),
                "page": rng.choice([1, 7, 16, 64]), "fp8": rng.random() < 0.4, "causal": sq > 1,
                "outliers": rng.random() < 0.2}
    return {"op": "append", "tokens": _log(rng, 1, 8192), "heads": rng.choice([rng.randint(1, 128), 8, 16, 128]),
            "page": rng.choice([1, 7, 16, 64]), "fp8": rng.random() < 0.4, "interleaved": rng.random() < 0.6,
            "padded": rng.choice([0, 0, 1, 9])}


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) & 0x7FFFFFFFFFFFFFFF)


def _codes(x):
    """fp8 codes of x and the scale they stand on: x is about codes * scale."""
    scale = (x.abs().max() / 448.0).reshape(1)
    return (x / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8), scale


def _prepare_prefix(c, g):
    B, H, Sq, P, ps = c["batch"], c["heads"], c["sq"], c["prefix"], c["page"]
    # Each sequence's own tokens, the new ones among them: log-uniform up to c["suffix"].
    u = torch.rand(B, generator=g, device=DEV)
    lo, hi = float(Sq), float(max(c["suffix"], Sq))
    suffix = torch.exp(math.log(lo) + u * (math.log(hi + 1.0) - math.log(lo))).floor().clamp(lo, hi).to(torch.int32)
    lens = (P + suffix).to(torch.int32)
    pre_pages = -(-P // ps)
    first = P // ps                                    # the first page that a sequence has for itself
    per = -(-(P + int(hi)) // ps) - first              # own pages that each table has room for
    pool = torch.randperm(pre_pages + B * per, generator=g, device=DEV).to(torch.int32)
    prefix_table = pool[:pre_pages].contiguous()
    own_pages = pool[pre_pages:].view(B, per)
    block_table = torch.cat([prefix_table[:first].expand(B, first), own_pages], 1).contiguous()
    cache = torch.randn(pre_pages + B * per, ps, D_QK, generator=g, device=DEV)
    if c["outliers"]:
        cache *= 1.0 + 7.0 * (torch.rand(cache.shape[0], ps, 1, generator=g, device=DEV) < 0.01)
    kv_scale = None
    if c["fp8"]:
        cache, kv_scale = _codes(cache)
    else:
        cache = cache.to(torch.bfloat16)
    s = {"op": "prefix", "case": c, "cache": cache, "kv_scale": kv_scale, "prefix_table": prefix_table,
         "block_table": block_table, "lens": lens, "prefix": P,
         "q": torch.randn(B, Sq, H, D_QK, generator=g, device=DEV).to(torch.bfloat16)}
    if own:
        import paged_mla_decode_latent_gb300 as mla
        s["plan"] = mla.prefix_plan(lens.cpu(), P, H, Sq, ps, mla.KV_FP8_E4M3 if c["fp8"] else mla.KV_BF16, c["causal"])
        s["workspace"] = mla.workspace_for(s["plan"])
        s["out"] = torch.empty(B, Sq, H, D_V, dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty(B, Sq, H, dtype=torch.float32, device=DEV)
    return s


def _prepare_append(c, g):
    T, H, ps = c["tokens"], c["heads"], c["page"]
    pages = -(-max(2 * T, 512) // ps)
    table = 65536
    # The rotation's table: angles in 64 bits, rounded once.
    freq = 10000.0 ** (-torch.arange(0, D_ROPE, 2, dtype=torch.float64, device=DEV) / D_ROPE)
    angle = torch.arange(table, dtype=torch.float64, device=DEV)[:, None] * freq
    cos_sin = torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32)
    # The projections as they leave their products: q is one tensor of 192 dims a head whose last 64 are
    # rotated, the latent and its rotated part are one row of 576, the absorbed query is [heads, tokens, 512].
    q = torch.randn(T, H, 192, generator=g, device=DEV).to(torch.bfloat16)
    kv = torch.randn(T, D_QK, generator=g, device=DEV).to(torch.bfloat16)
    ql = torch.empty(H, T, D_V, dtype=torch.bfloat16, device=DEV)
    for h0 in range(0, H, 16):
        n = min(16, H - h0)
        ql[h0:h0 + n] = torch.randn(n, T, D_V, generator=g, device=DEV).to(torch.bfloat16)
    slots = torch.randperm(pages * ps, generator=g, device=DEV)[:T]
    if c["padded"]:
        slots[max(0, T - c["padded"]):] = -1
    cache = torch.randn(pages, ps, D_QK, generator=g, device=DEV)
    if c["fp8"]:
        cache, kv_scale = _codes(cache)
    else:
        cache, kv_scale = cache.to(torch.bfloat16), None
    s = {"op": "append", "case": c, "q_pe": q[..., 128:], "ql_nope": ql.transpose(0, 1), "kv_c": kv[:, :D_V],
         "k_pe": kv[:, D_V:], "positions": torch.randint(0, table, (T,), generator=g, device=DEV),
         "cos_sin": cos_sin, "slots": slots, "cache": cache, "kv_scale": kv_scale}
    if own:
        import paged_mla_decode_latent_gb300  # noqa: F401  (the calls are made in run)
        s["q_out"] = torch.empty(T, H, D_QK, dtype=torch.bfloat16, device=DEV)
    return s


def prepare(case, seed):
    return (_prepare_prefix if case["op"] == "prefix" else _prepare_append)(case, _gen(seed))


def _rows(cache, kv_scale, page, slot):
    """Latent rows in 32 bits."""
    x = cache[page, slot]
    return x.to(torch.float32) if kv_scale is None else x.view(torch.float8_e4m3fn).to(torch.float32) * kv_scale


def _plain_prefix(s):
    c, q, P, ps = s["case"], s["q"].to(torch.float32), s["prefix"], s["case"]["page"]
    B, Sq, H, _ = q.shape
    ctx = s["lens"].to(torch.int64)
    tok = torch.arange(Sq, device=DEV)
    seen = ctx[:, None] - Sq + tok + 1 if c["causal"] else ctx[:, None].expand(B, Sq)
    seen = seen.clamp(min=0).repeat_interleave(H, 1)                       # [B, rows] visible keys
    q = q.reshape(B, Sq * H, D_QK)
    # The shared keys, for every row of the batch at once.
    j = torch.arange(P, device=DEV)
    kp = _rows(s["cache"], s["kv_scale"], s["prefix_table"].to(torch.int64)[j // ps], j % ps)
    zp = (q.reshape(-1, D_QK) @ kp.t()).mul_(SCALE)
    zp.masked_fill_(j >= seen.reshape(-1, 1), -math.inf)
    # Each sequence's own keys.
    most = s["block_table"].shape[1] * ps
    k = torch.arange(P, min(most, P + max(c["suffix"], Sq)), device=DEV)
    at = torch.where(k < ctx[:, None], k, P)
    ks = _rows(s["cache"], s["kv_scale"], s["block_table"].to(torch.int64).gather(1, at // ps), at % ps)
    zs = torch.bmm(q, ks.transpose(1, 2)).mul_(SCALE).masked_fill_(k >= seen[..., None], -math.inf)
    top = torch.maximum(zp.amax(1).view(B, -1), zs.amax(2))
    wp = zp.sub_(top.reshape(-1, 1)).exp_()
    ws = zs.sub_(top[..., None]).exp_()
    total = wp.sum(1).view(B, -1) + ws.sum(2)
    o = (wp @ kp[:, :D_V]).view(B, -1, D_V) + torch.bmm(ws, ks[..., :D_V])
    out = (o / total[..., None]).to(torch.bfloat16).view(B, Sq, H, D_V)
    return {"out": out, "lse": (top + total.log()).view(B, Sq, H)}


def _rotate(x, cs, interleaved):
    cos, sin = cs[..., :D_ROPE // 2], cs[..., D_ROPE // 2:]
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    a, b = x[..., :D_ROPE // 2], x[..., D_ROPE // 2:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _plain_append(s):
    c = s["case"]
    cs = s["cos_sin"][s["positions"]]
    q_pe = _rotate(s["q_pe"].to(torch.float32), cs[:, None], c["interleaved"])
    q_out = torch.cat([s["ql_nope"], q_pe.to(torch.bfloat16)], -1)
    row = torch.cat([s["kv_c"].to(torch.float32), _rotate(s["k_pe"].to(torch.float32), cs, c["interleaved"])], -1)
    n = max(0, c["tokens"] - c["padded"])
    slots = s["slots"][:n]
    flat = s["cache"].view(-1, D_QK)
    if c["fp8"]:
        flat[slots] = (row[:n] / s["kv_scale"]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        return {"q": q_out, "cache": s["cache"].view(torch.float8_e4m3fn)}
    flat[slots] = row[:n].to(torch.bfloat16)
    return {"q": q_out, "cache": s["cache"]}


def run(s):
    if own:
        import paged_mla_decode_latent_gb300 as mla
        if s["op"] == "prefix":
            mla.prefix_fwd(s["plan"], s["q"], s["cache"], s["kv_scale"], s["prefix_table"], s["block_table"], s["lens"],
                           SCALE, s["out"], s["lse"], s["workspace"])
            return {"out": s["out"], "lse": s["lse"]}
        mla.rope_epilogue(s["ql_nope"], s["q_pe"], s["kv_c"], s["k_pe"], s["positions"], s["cos_sin"], s["slots"],
                          s["q_out"], s["cache"], s["kv_scale"], interleaved=s["case"]["interleaved"])
        return {"q": s["q_out"], "cache": s["cache"].view(torch.float8_e4m3fn) if s["case"]["fp8"] else s["cache"]}
    return _plain_prefix(s) if s["op"] == "prefix" else _plain_append(s)


def _sequences(c, seed):
    s = prepare(c, seed)
    return s, [int(n) for n in s["lens"].tolist()]


def work(case):
    c = case
    if c["op"] == "append":
        T, H = c["tokens"], c["heads"]
        kept = max(0, T - c["padded"])
        # q in and out; the row in and out; the rotation's row, the position and the slot.
        return {"bytes": 2 * T * H * D_QK * 2 + T * D_QK * 2 + kept * D_QK * (1 if c["fp8"] else 2) + T * (256 + 16),
                "flops": 6 * 32 * T * (H + 1)}
    B, rows = c["batch"], c["heads"] * c["sq"]
    lo, hi = c["sq"], max(c["suffix"], c["sq"])
    mean = lo if hi == lo else (hi - lo) / math.log(hi / lo)     # of a log-uniform length
    keys = c["prefix"] + B * mean                                # cache rows, each read once
    row = D_QK * (1 if c["fp8"] else 2)
    return {"bytes": int(keys * (row + 4 / c["page"]) + B * rows * (D_QK * 2 + D_V * 2 + 4)),
            "flops": int(2 * (D_QK + D_V) * B * rows * (c["prefix"] + mean))}


def _exact_prefix(c, seed):
    s, lens = _sequences(c, seed)
    B, H, Sq, P, ps = c["batch"], c["heads"], c["sq"], c["prefix"], c["page"]
    flat = s["cache"].reshape(-1, D_QK)
    scale = 1.0 if s["kv_scale"] is None else float(s["kv_scale"])

    def rows(table, keys):
        x = flat[table[keys // ps].to(torch.int64) * ps + keys % ps]
        return (x.view(torch.float8_e4m3fn) if c["fp8"] else x).to(torch.float64) * scale

    shared = rows(s["prefix_table"], torch.arange(P, device=DEV))
    out = torch.empty(B, Sq, H, D_V, dtype=torch.float64, device=DEV)
    lse = torch.empty(B, Sq, H, dtype=torch.float64, device=DEV)
    for b in range(B):
        keys = torch.cat([shared, rows(s["block_table"][b], torch.arange(P, lens[b], device=DEV))])
        for i in range(Sq):
            n = lens[b] - Sq + i + 1 if c["causal"] else lens[b]
            z = (s["q"][b, i].to(torch.float64) @ keys[:n].t()) / math.sqrt(192.0)
            lse[b, i] = torch.logsumexp(z, 1)
            out[b, i] = torch.exp(z - lse[b, i][:, None]) @ keys[:n, :D_V]
    return {"out": out, "lse": lse}


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

    cache = (s["cache"].view(torch.float8_e4m3fn) if c["fp8"] else s["cache"]).to(torch.float64)
    keep = s["slots"] >= 0
    row = torch.cat([s["kv_c"].to(torch.float64), rotated(s["k_pe"], turn)], 1)[keep]
    if c["fp8"]:
        row = (row / s["kv_scale"].to(torch.float64)).clamp(-448.0, 448.0)
    cache.view(-1, D_QK)[s["slots"][keep]] = row
    q = torch.empty(T, c["heads"], D_QK, dtype=torch.float64, device=DEV)
    q[..., :D_V] = s["ql_nope"]
    q[..., D_V:] = rotated(s["q_pe"], turn[:, None])
    return {"q": q, "cache": cache}


def exact(case, seed):
    return (_exact_prefix if case["op"] == "prefix" else _exact_append)(case, seed)
