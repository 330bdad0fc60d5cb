"""The 4-bit cache row in numpy, 64 bits: values, codes, and a decode over them."""
from __future__ import annotations

import numpy as np

import mla_synth as syn

ROW = 416
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3_value(code):
    """Values of OCP E4M3FN codes."""
    code = np.asarray(code, np.uint8).astype(np.int64)
    e, m = (code >> 3) & 15, code & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((code & 127) == 127, np.nan, v)
    return np.where(code & 128, -v, v)


def e4m3_code(x):
    """Nearest code of x >= 0 (ties to the even one), at most 448."""
    grid = e4m3_value(np.arange(127))
    x = np.minimum(np.asarray(x, np.float64), 448.0)
    hi = np.minimum(np.searchsorted(grid, x), 126)
    lo = np.maximum(hi - 1, 0)
    d_lo, d_hi = x - grid[lo], grid[hi] - x
    up = (d_hi < d_lo) | ((d_hi == d_lo) & (hi % 2 == 0))
    return np.where(up, hi, lo).astype(np.uint8)


def e2m1_code(v):
    """Nearest code (ties to the even one), saturating."""
    a = np.abs(np.asarray(v, np.float64))
    mid = (E2M1[1:] + E2M1[:-1]) / 2
    c = np.zeros(a.shape, np.uint8)
    for k, m in enumerate(mid):  # from code k to k + 1; the tie goes to the even one
        c += (a > m) if k % 2 == 0 else (a >= m)
    return c + 8 * np.signbit(v).astype(np.uint8)


def f32_quotient(x, by):
    """x / by rounded once to 32 bits (both of 32 bits or fewer)."""
    with np.errstate(all="ignore"):
        return (np.asarray(x, np.float64) / np.asarray(by, np.float64)).astype(np.float32).astype(np.float64)


def encode(latent, rope, kv_scale):
    """4-bit rows (uint8 [n, 416]) of latent [n, 512] and rope [n, 64]."""
    kv_scale = np.float32(kv_scale)
    n = latent.shape[0]
    q = f32_quotient(latent, kv_scale).reshape(n, 32, 16)
    bad = np.isnan(q).any(2)
    top = np.where(bad, 0.0, np.nanmax(np.abs(np.where(np.isnan(q), 0.0, q)), axis=2))
    s = np.where(bad, 0x7F, e4m3_code(f32_quotient(top, np.float32(6.0)))).astype(np.uint8)
    d = np.where(bad, 1.0, e4m3_value(s))[..., None]
    zero = (bad | (s == 0))[..., None]
    c = np.where(zero, 0, e2m1_code(f32_quotient(np.where(zero, 0.0, q), np.where(zero, 1.0, d)))).astype(np.uint8)
    c = c.reshape(n, 256, 2)
    with np.errstate(all="ignore"):
        r = np.clip(f32_quotient(rope, kv_scale), -65504.0, 65504.0).astype(np.float32).astype(np.float16)
    return np.concatenate([c[..., 0] | c[..., 1] << 4, s, r.view(np.uint8).reshape(n, 128)], 1)


def decode_rows(rows):
    """The values of rows [..., 416] without kv_scale, in 64 bits: [..., 576]."""
    codes = rows[..., :256]
    value = np.concatenate([E2M1, -E2M1])
    v = np.stack([value[codes & 15], value[codes >> 4]], -1).reshape(*rows.shape[:-1], 512)
    v = v * np.repeat(e4m3_value(rows[..., 256:288]), 16, axis=-1)
    r = np.ascontiguousarray(rows[..., 288:]).view(np.float16).astype(np.float64)
    return np.concatenate([v, r], -1)


class Fp4Problem:
    """A decode over a 4-bit cache of N(0, 1) rows; `outliers`: that share of rows times 8."""

    def __init__(self, batch, sq, heads, lens, page, causal=False, seed=0, outliers=0.0, poison=True, raw=False):
        p = syn.make_problem(batch, sq, heads, lens, page, syn.KV_BF16, causal, seed, outlier_frac=outliers, poison=False)
        self.batch, self.sq, self.heads, self.page, self.causal = batch, sq, heads, page, causal
        self.lens, self.q_bits, self.table = p.seq_lens, p.q_bits, p.block_table
        self.scale = p.softmax_scale
        x = syn.bf16_bits_to_f32(p.cache).reshape(-1, 576)
        self.kv_scale = np.float32(np.abs(x).max() / 2688.0)
        if raw:  # every code and every finite scale, whatever a writer would choose
            rng = np.random.default_rng(seed)
            self.cache = rng.integers(0, 256, (x.shape[0], ROW), dtype=np.uint8)
            s = self.cache[:, 256:288]
            s[(s & 127) > 0x48] = 0x48  # up to 4: sums stay within fp32's and bf16's reach
            self.cache[:, 288:] = x[:, 512:].astype(np.float16).view(np.uint8)
            self.kv_scale = np.float32(0.25)
        else:
            self.cache = encode(x[:, :512], x[:, 512:], self.kv_scale)
        self.cache = self.cache.reshape(p.num_pages, page, ROW)
        if poison:  # what no call may read: NaN scales and NaN rope behind every sequence's end, and unused entries
            for b, n in enumerate(self.lens):
                pages = -(-int(n) // page)
                if n % page:
                    tail = self.cache[self.table[b, pages - 1], n % page:]
                    tail[:, 256:] = 0x7F
                self.table[b, pages:] = -1

    def keys(self, b):
        n = int(self.lens[b])
        j = np.arange(n)
        return decode_rows(self.cache[self.table[b, j // self.page], j % self.page]) * np.float64(self.kv_scale)

    def reference(self):
        q = syn.bf16_bits_to_f32(self.q_bits).astype(np.float64)
        B, Sq, H = self.batch, self.sq, self.heads
        out, lse = np.zeros((B, Sq, H, 512)), np.full((B, Sq, H), -np.inf)
        for b in range(B):
            keys, n = self.keys(b), int(self.lens[b])
            for i in range(Sq):
                m = max(0, n - Sq + i + 1) if self.causal else n
                if m == 0:
                    continue
                z = (q[b, i] @ keys[:m].T) * self.scale
                top = z.max(1, keepdims=True)
                w = np.exp(z - top)
                lse[b, i] = top[:, 0] + np.log(w.sum(1))
                out[b, i] = (w / w.sum(1, keepdims=True)) @ keys[:m, :512]
        return out, lse

    def to_device(self):
        import torch
        return {"q": torch.from_numpy(self.q_bits.view(np.int16)).view(torch.bfloat16).cuda(),
                "cache": torch.from_numpy(self.cache).cuda(), "bt": torch.from_numpy(self.table).cuda(),
                "lens": torch.from_numpy(self.lens).cuda(), "scale": torch.tensor([self.kv_scale], device="cuda")}

    def run(self, num_sms=0, t=None):
        """plan + fwd + combine; (out, lse, plan, status)."""
        import torch
        import paged_mla_decode_latent_gb300 as mla
        t = t or self.to_device()
        plan = mla.plan(self.lens, self.heads, self.sq, self.page, mla.KV_FP4_E2M1, self.causal, num_sms)
        ws = mla.workspace_for(plan)
        out = torch.full((self.batch, self.sq, self.heads, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
        lse = torch.full((self.batch, self.sq, self.heads), float("nan"), device="cuda")
        mla.fwd(plan, t["q"], t["cache"], t["scale"], t["bt"], t["lens"], self.scale, out, lse, ws)
        mla.combine(plan, t["lens"], out, lse, ws)
        status = mla.check(plan, ws)
        return out.double().cpu().numpy(), lse.double().cpu().numpy(), plan, status
