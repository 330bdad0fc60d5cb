"""The shared-prefix decode on rows of small magnitude, which f16 holds only scaled.

Bar: parity.py's (relative Frobenius error 4e-3, LSE 1e-3), here for every query row by itself, so
that rows over large keys hide nothing.  What a row's 512 outputs are off by: half a bf16 step each,
2^-8 / sqrt(3) of the value at most in the mean square (2.3e-3; 1.65e-3 over all mantissas), weights
of 11 bits (3e-4), and the staging, 2^-17 of a key's largest latent value."""
import numpy as np
import pytest

import mla_synth as syn
from prefix_problems import PrefixProblem

pytestmark = pytest.mark.gpu

BF16, FP8 = syn.KV_BF16, syn.KV_FP8_E4M3


def scale_bits(bits, by):
    """bf16 bits times powers of two (exact, but for the subnormals that it meets)."""
    return syn.f32_to_bf16_bits(syn.bf16_bits_to_f32(bits) * np.float32(by) if np.isscalar(by)
                                else syn.bf16_bits_to_f32(bits) * by.astype(np.float32))


def check_rows(p, out, lse, what=""):
    ref, ref_lse = p.reference()
    some = np.isfinite(ref_lse)
    assert np.array_equal(np.isneginf(lse), ~some) and np.all(out[~some] == 0)
    assert np.isfinite(out).all()
    err = np.linalg.norm(out - ref, axis=-1)[some] / np.linalg.norm(ref, axis=-1)[some]
    assert err.max() <= 4e-3, f"{what}: a row's relative error {err.max():.2e}"
    e = np.abs(lse - ref_lse)[some].max()
    assert e <= 1e-3, f"{what}: lse {e:.2e}"


@pytest.mark.parametrize("k", [7, 9, 12, 14, 16, 18, 20, 24, 33, 48, 66])
def test_small_keys(k):
    """The whole cache times 2^-k, shared and own keys; scores of order one all the same."""
    up = min(k, 11)
    p = PrefixProblem(4, 2, 16, [300, 290, 100, 520], 256, 16, causal=True, seed=k, q_mult=2.0 ** up,
                      scale=syn.DEFAULT_SCALE * 2.0 ** (k - up))
    p.cache = scale_bits(p.cache, 2.0 ** -k)
    out, lse, plan, status = p.run()
    assert status == 0 and plan.own_folded
    check_rows(p, out, lse, f"2^-{k}")


@pytest.mark.parametrize("k", [9, 12, 16, 20, 40, 70])
@pytest.mark.parametrize("dtype", [BF16, FP8])
def test_small_queries(k, dtype):
    """Every query row times its own power of two down to 2^-k, softmax_scale up by 2^k: some rows
    of a block are scaled when staged and some are not."""
    p = PrefixProblem(3, 1, 40, [700, 690, 100], 640, 16, dtype, seed=k, scale=syn.DEFAULT_SCALE * 2.0 ** k)
    by = 2.0 ** -np.random.default_rng(k).integers(k - 2, k + 1, (3, 1, 40, 1)).astype(np.float64)
    p.q_bits = scale_bits(p.q_bits, by)
    out, lse, _, status = p.run()
    assert status == 0
    check_rows(p, out, lse, f"q 2^-{k}")


@pytest.mark.parametrize("sms", [0, 2, 6])
def test_keys_of_every_magnitude(sms):
    """Magnitudes 1 to 2^-40 key by key, in whole row blocks and cut ones.  Sequences that end before
    the large keys see small ones only."""
    p = PrefixProblem(6, 1, 32, [1500, 40, 300, 700, 1460, 1530], 1450, 1, seed=3, scale=0.02)
    rng = np.random.default_rng(5)
    slots = p.slots[5]  # the longest sequence's: position -> row
    flat = p.cache.reshape(-1, 576)
    k = np.where(np.arange(1450) < 320, rng.integers(16, 41, 1450), rng.integers(0, 41, 1450))
    flat[slots[:1450]] = scale_bits(flat[slots[:1450]], 2.0 ** -k[:, None].astype(np.float64))
    out, lse, _, status = p.run(num_sms=sms)
    assert status == 0
    check_rows(p, out, lse, f"mixed, {sms} SMs")


@pytest.mark.parametrize("first", [True, False])
def test_a_large_key_without_weight_leaves_the_small_ones_their_bits(first):
    """One key of order one that every query row scores at -60 or less, among keys of 2^-20: the
    output is the small keys', whether the large one comes first or in a later tile."""
    p = PrefixProblem(2, 1, 16, [600, 620], 590, 16, seed=6, scale=0.5)
    q = syn.bf16_bits_to_f32(p.q_bits)
    q[..., 3] = 16.0
    p.q_bits = syn.f32_to_bf16_bits(q)
    p.cache = scale_bits(p.cache, 2.0 ** -20)
    j = 0 if first else 580
    row = np.zeros(576, np.float32)
    row[3], row[100] = -8.0, 1.0
    p.cache[p.prefix_table[j // 16], j % 16] = syn.f32_to_bf16_bits(row)
    out, lse, _, status = p.run()
    assert status == 0
    ref, _ = p.reference()
    assert np.abs(ref).max() < 2.0 ** -18
    check_rows(p, out, lse, "large key without weight")


def test_small_latents_beside_ordinary_rope_dims():
    p = PrefixProblem(3, 1, 64, [500, 420, 300], 400, 16, seed=7)
    by = np.ones(576)
    by[:512] = 2.0 ** -20
    p.cache = scale_bits(p.cache, np.broadcast_to(by, p.cache.shape))
    p.q_bits[..., :512] = scale_bits(p.q_bits[..., :512], 2.0 ** 10)
    out, lse, _, status = p.run()
    assert status == 0
    check_rows(p, out, lse, "small latents")


def test_bad_and_small_keys_in_one_tile():
    """A NaN key spoils the rows that see it; the small keys beside it keep their bits for the others."""
    import paged_mla_decode_latent_gb300 as mla
    p = PrefixProblem(3, 1, 16, [300, 290, 100], 256, 16, seed=8, q_mult=2.0 ** 8, scale=syn.DEFAULT_SCALE * 2.0 ** 10)
    p.cache = scale_bits(p.cache, 2.0 ** -18)
    ref, ref_lse = p.reference()
    t = p.to_device()
    t["cache"][int(p.prefix_table[200 // 16]), 200 % 16, 9] = float("nan")
    out, lse, _, status = p.run(t=t)
    assert status == mla.DEVFLAG_KV_RANGE
    assert np.isnan(out[:2]).all() and np.isnan(lse[:2]).all()
    err = np.linalg.norm(out[2] - ref[2], axis=-1) / np.linalg.norm(ref[2], axis=-1)
    assert err.max() <= 4e-3 and np.abs(lse[2] - ref_lse[2]).max() <= 1e-3


def test_zero_rows_and_subnormals():
    """Rows of zeros (nothing to scale by) and of bf16's smallest values beside ordinary ones."""
    p = PrefixProblem(2, 1, 16, [300, 270], 256, 16, seed=9)
    flat = p.cache.reshape(-1, 576)
    flat[p.slots[0, 10:20]] = 0
    flat[p.slots[0, 20:30]] = 1  # 2^-133
    flat[p.slots[0, 256:260]] = 0
    p.q_bits[0, 0, 3] = 0
    p.q_bits[0, 0, 4] = 1
    out, lse, _, status = p.run()
    assert status == 0
    check_rows(p, out, lse, "zeros and subnormals")


@pytest.mark.parametrize("k", [8, 9, 10, 11, 12])
@pytest.mark.parametrize("flat", [False, True])
def test_keys_about_the_border_of_what_is_scaled(k, flat):
    """Thousands of keys of one magnitude, of which some are scaled when staged and some are not: their
    weights keep the same bits.  flat: scores near zero, so that every key counts."""
    p = PrefixProblem(6, 1, 64, [2203 - 30 * i for i in range(6)], 2158, 64, seed=k, q_mult=2.0 ** k,
                      scale=syn.DEFAULT_SCALE * (2.0 ** -10 if flat else 1.0))
    p.cache = scale_bits(p.cache, 2.0 ** -k)
    out, lse, _, status = p.run()
    assert status == 0
    check_rows(p, out, lse, f"2^-{k}")


def test_keys_of_two_magnitudes():
    """Half of the keys at 2^-10, half of order one, in rows whose scores favour either."""
    p = PrefixProblem(8, 1, 64, [2203 - i for i in range(8)], 2158, 64, seed=3)
    flat = p.cache.reshape(-1, 576)
    half = np.random.default_rng(4).random((flat.shape[0], 1)) < 0.5
    p.cache = scale_bits(flat, np.where(half, 2.0 ** -10, 1.0)).reshape(p.cache.shape)
    out, lse, _, status = p.run()
    assert status == 0
    check_rows(p, out, lse, "two magnitudes")


@pytest.mark.parametrize("spike", [2.0 ** -8, 2.0 ** -6, 2.0 ** -4, 1.0, 2.0 ** 6])
def test_many_light_small_keys_beside_a_heavy_one(spike):
    """2100 equal keys of magnitude 2^-10 with e^-8 of the weight of one that a single large value keeps
    from being scaled: together they hold a third of the output's other dims."""
    p = PrefixProblem(2, 1, 16, [2110, 2120], 2100, 1, seed=5, scale=1.0)
    rng = np.random.default_rng(6)
    row = np.zeros((2, 576), np.float32)
    row[:, :512] = rng.standard_normal((2, 512)).clip(-2, 2) * 2.0 ** -10
    row[0, 7], row[0, 512] = spike, 2.0 ** -9
    p.cache.reshape(-1, 576)[:] = syn.f32_to_bf16_bits(row[1])
    p.cache[p.prefix_table[50], 0] = syn.f32_to_bf16_bits(row[0])
    q = np.zeros(p.q_bits.shape, np.float32)
    q[..., 512] = 2.0 ** 12
    p.q_bits = syn.f32_to_bf16_bits(q)
    out, lse, _, status = p.run()
    assert status == 0
    ref, ref_lse = p.reference()
    rest = np.arange(512) != 7
    err = np.linalg.norm((out - ref)[..., rest], axis=-1) / np.linalg.norm(ref[..., rest], axis=-1)
    assert err.max() <= 4e-3 and np.abs(lse - ref_lse).max() <= 1e-3
