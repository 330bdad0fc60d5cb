"""Problems whose sequences share a prefix, for the tests of the shared-prefix
decode: the paged inputs the library takes, and the same keys as the fp64
oracle takes them (one table of single-key pages per sequence)."""
from __future__ import annotations

import numpy as np

import mla_synth as syn


class PrefixProblem:
    def __init__(self, batch, sq, heads, lens, prefix, page_size, kv_dtype=syn.KV_BF16,
                 causal=False, seed=0, outlier_frac=0.0, scale=syn.DEFAULT_SCALE, q_mult=1.0):
        lens = np.asarray(lens, np.int32).reshape(batch)
        pre_pages = -(-prefix // page_size)
        first = prefix // page_size
        own = [max(0, -(-int(n) // page_size) - first) if n > prefix else 0 for n in lens]
        n_pages = max(1, pre_pages + sum(own))
        base = syn.make_problem(batch, sq, heads, [0] * batch, page_size, kv_dtype, causal, seed,
                                softmax_scale=scale, outlier_frac=outlier_frac,
                                extra_pages=n_pages)
        rng = np.random.default_rng(seed + 17)
        pool = rng.permutation(n_pages).astype(np.int32)
        cache = base.cache
        nan = np.uint16(0x7FC0) if kv_dtype == syn.KV_BF16 else np.uint8(0x7F)
        used = np.zeros((n_pages, page_size), bool)
        self.prefix_table = pool[:pre_pages].copy()
        for j in range(prefix):
            used[self.prefix_table[j // page_size], j % page_size] = True
        width = max(1, first + max(own + [0]), -(-int(lens.max() if batch else 0) // page_size))
        # Entries before the own pages and past the last one are -1: never read.
        bt = np.full((batch, width), -1, np.int32)
        slots = np.zeros((batch, max(1, int(lens.max()))), np.int32)
        at = pre_pages
        for b, n in enumerate(lens):
            bt[b, first:first + own[b]] = pool[at:at + own[b]]
            at += own[b]
            for j in range(int(n)):
                page = self.prefix_table[j // page_size] if j < prefix else bt[b, j // page_size]
                slots[b, j] = page * page_size + j % page_size
                used[page, j % page_size] = True
        cache[~used] = nan  # poison: slots no sequence holds
        self.batch, self.sq, self.heads, self.prefix = batch, sq, heads, prefix
        self.lens, self.page_size, self.kv_dtype, self.causal = lens, page_size, kv_dtype, causal
        self.q_bits, self.cache, self.kv_scale, self.scale = base.q_bits, cache, base.kv_scale, scale
        if q_mult != 1.0:
            self.q_bits = syn.f32_to_bf16_bits(syn.bf16_bits_to_f32(self.q_bits) * np.float32(q_mult))
        self.block_table, self.slots = bt, slots

    def reference(self):
        import oracle
        oracle.build()
        flat = self.cache.reshape(-1, 1, syn.D_QK)
        return oracle.decode(self.q_bits, flat, self.kv_dtype, self.kv_scale, 1, self.slots,
                             self.lens, self.scale, self.causal)

    def to_device(self, device="cuda"):
        import torch
        c = torch.from_numpy(self.cache.view(np.int16)).view(torch.bfloat16) \
            if self.kv_dtype == syn.KV_BF16 else torch.from_numpy(self.cache)
        return dict(q=torch.from_numpy(self.q_bits.view(np.int16)).view(torch.bfloat16).to(device),
                    cache=c.to(device), scale=torch.tensor([self.kv_scale], dtype=torch.float32, device=device),
                    pt=torch.from_numpy(self.prefix_table).to(device) if self.prefix else None,
                    bt=torch.from_numpy(self.block_table).to(device),
                    lens=torch.from_numpy(self.lens).to(device))

    def plan(self, num_sms=0):
        import paged_mla_decode_latent_gb300 as mla
        return mla.prefix_plan(self.lens, self.prefix, self.heads, self.sq, self.page_size,
                               self.kv_dtype, self.causal, num_sms)

    def run(self, t=None, plan=None, num_sms=0, workspace=None):
        """(out f64, lse f64, plan, status) through the C ABI; outputs start as NaN."""
        import torch
        import paged_mla_decode_latent_gb300 as mla
        t = t or self.to_device()
        plan = plan or self.plan(num_sms)
        ws = workspace if workspace is not None else mla.workspace_for(plan)
        out = torch.full((self.batch, self.sq, self.heads, 512), float("nan"), dtype=torch.bfloat16,
                         device="cuda")
        lse = torch.full((self.batch, self.sq, self.heads), float("nan"), device="cuda")
        mla.prefix_fwd(plan, t["q"], t["cache"], t["scale"], t["pt"], t["bt"], t["lens"],
                       self.scale, out, lse, ws)
        status = mla.prefix_check(plan, ws)
        return out.double().cpu().numpy(), lse.double().cpu().numpy(), plan, status
