"""The shared-prefix decode on inputs whose scores are exact, at bounds derived from the arithmetic:
what is left is the rounding of the weights, the exponentials and the sums.

Queries and keys are small integers, so every product and sum of a score is
exact in fp32 in any order.  Per row, with s the largest |c2 s_j| (log2 units; c2 = c log2 e), T the
tiles it spans and n its keys:
  exponent     c2 is rounded twice (2^-23 s); c2 s_j + base once, base = 7 - m, |m| <= s + 8:
               2^-24 (2 s + 15); times ln 2
  exponential  2^-22 relative
  row sum      16 sums in a chain, then 3, then one a tile and one an exchange: 2^-24 (24 + 2 T)
  log          log2 of up to 2^40 within an ulp (2^-18), m - 7 + log2 l and the product with ln 2
               rounded once each: 2^-24 (2 s + 64)
  merge        expf, logf and sums over at most 77 partials: 2^-22 + 2^-24 (77 + 2 |lse|)
They add up to lse_bound.  An output adds the f16 weights, half a step of 2^-11 relative each, the
fp32 sum over n keys (truncated at most: 2^-23 n), all relative to sum_j w_j |v_j|, and its own
rounding to bf16, 2^-8 of the value."""
import numpy as np
import pytest

import mla_synth as syn
from prefix_problems import PrefixProblem

pytestmark = pytest.mark.gpu

LN2 = np.log(2.0)


def lse_bound(s, tiles, lse):
    return (LN2 * (2.0 ** -23 * s + 2.0 ** -24 * (2 * s + 15)) + 2.0 ** -22 + 2.0 ** -24 * (24 + 2 * tiles)
            + LN2 * (2.0 ** -18 + 2.0 ** -24 * (2 * s + 64)) + 2.0 ** -22 + 2.0 ** -24 * (77 + 2 * abs(lse)))


def rows(p):
    """(b, i, h, scores, values, softmax weights, lse) of every row that sees a key, in 64 bits."""
    q = syn.bf16_bits_to_f32(p.q_bits).astype(np.float64)
    flat = syn.bf16_bits_to_f32(p.cache.reshape(-1, 576)).astype(np.float64)
    for b in range(p.batch):
        k = flat[p.slots[b, :p.lens[b]]]
        for i in range(p.sq):
            n = int(p.lens[b]) - p.sq + i + 1 if p.causal else int(p.lens[b])
            if n <= 0:
                continue
            z = q[b, i] @ k[:n].T * p.scale
            top = z.max(1, keepdims=True)
            w = np.exp(z - top)
            lse = top[:, 0] + np.log(w.sum(1))
            for h in range(p.heads):
                yield b, i, h, z[h] / LN2, k[:n, :512], w[h] / w[h].sum(), lse[h]


def check(p, out, lse, weight_step=2.0 ** -11):
    worst_o = worst_l = 0.0
    for b, i, h, z2, v, w, ref_lse in rows(p):
        s = np.abs(z2).max()
        tiles = p.prefix // 256 + 1 + (p.batch * max(0, int(p.lens.max()) - p.prefix)) // 256 + 1
        lb = lse_bound(s, tiles, ref_lse)
        ref, mass = w @ v, w @ np.abs(v)
        ob = 2.0 ** -8 * np.abs(ref) + 1.01 * (weight_step + 2 * lb + 2.0 ** -23 * len(w)) * mass
        worst_l = max(worst_l, abs(lse[b, i, h] - ref_lse) / lb)
        worst_o = max(worst_o, (np.abs(out[b, i, h] - ref) / np.maximum(ob, 1e-300)).max())
    return worst_o, worst_l


@pytest.mark.parametrize("args,sms", [
    ((2, 1, 16, [700, 760], 700, 16, syn.KV_BF16, False), 0),
    ((3, 2, 20, [300, 290, 100], 256, 7, syn.KV_BF16, True), 0),
    ((3, 2, 20, [300, 290, 100], 256, 7, syn.KV_BF16, True), 2),
    ((1, 1, 128, [2600], 2500, 16, syn.KV_BF16, False), 0),
    ((5, 1, 8, [1, 2, 3, 130, 0], 128, 1, syn.KV_BF16, False), 0)])
def test_integer_scores(args, sms):
    p = PrefixProblem(*args, seed=3, scale=2.0 ** -6)
    rng = np.random.default_rng(4)
    p.q_bits = syn.f32_to_bf16_bits(rng.integers(-2, 3, p.q_bits.shape).astype(np.float32))
    p.cache = syn.f32_to_bf16_bits(rng.integers(-2, 3, p.cache.shape).astype(np.float32))
    out, lse, plan, status = p.run(num_sms=sms)
    assert status == 0 and (plan.own_folded or plan.own_splits == 0)
    worst_o, worst_l = check(p, out, lse)
    print(f"of the bounds: out {worst_o:.3f}, lse {worst_l:.3f}")
    assert worst_o <= 1 and worst_l <= 1


def two_keys(prefix):
    """Two keys of opposite values and nearly equal weights, p = e^(-a / 512) for a = 1 .. 200 by
    head: an output is (1 - p) / (1 + p), small against the weights whose rounding it shows."""
    p = PrefixProblem(2, 1, 100, [2, 2], prefix, 1, seed=5, scale=2.0 ** -9)
    q = np.zeros((2, 1, 100, 576), np.float32)
    q[..., 512] = np.arange(1, 201).reshape(2, 1, 100)
    p.q_bits = syn.f32_to_bf16_bits(q)
    row = np.ones(576, np.float32)
    row[512:] = 0
    flat = p.cache.reshape(-1, 576)
    for b in range(2):
        flat[p.slots[b, 0]] = syn.f32_to_bf16_bits(row)
        other = -row
        other[512] = -1.0
        flat[p.slots[b, 1]] = syn.f32_to_bf16_bits(other)
    return p


def emulated(p, dtype):
    """The two keys' outputs with their weights rounded to `dtype`, all else exact."""
    import torch
    out, lse = np.zeros((2, 1, 100, 512)), np.zeros((2, 1, 100))
    for b, i, h, z2, v, w, ref_lse in rows(p):
        x = np.exp2(z2 - z2.max() + 7)
        out[b, i, h] = torch.from_numpy(x).to(dtype).double().numpy() @ v / x.sum()
        lse[b, i, h] = ref_lse
    return out, lse


@pytest.mark.parametrize("prefix", [1, 2])
def test_weights_keep_eleven_bits(prefix):
    import torch
    p = two_keys(prefix)
    assert check(p, *emulated(p, torch.float16))[0] <= 1
    assert check(p, *emulated(p, torch.bfloat16))[0] > 1.2  # the bound tells the two apart
    out, lse, _, status = p.run()
    assert status == 0
    worst_o, worst_l = check(p, out, lse)
    assert worst_o <= 1 and worst_l <= 1
