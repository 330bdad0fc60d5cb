"""The 4-bit row's definition against itself, and what the library refuses of it (no GPU)."""
import ctypes

import numpy as np
import pytest

import fp4_rows as f4
import paged_mla_decode_latent_gb300 as mla


@pytest.fixture(scope="module", autouse=True)
def built():
    mla.build()


def test_codes_are_the_nearest_and_ties_go_to_the_even_one():
    import torch
    x = np.concatenate([np.linspace(0, 500, 4001), f4.e4m3_value(np.arange(127)),
                        (f4.e4m3_value(np.arange(126)) + f4.e4m3_value(np.arange(1, 127))) / 2])
    ref = torch.from_numpy(np.minimum(x, 448).astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(f4.e4m3_code(x.astype(np.float32)), ref)
    for v, c in [(0, 0), (.25, 0), (.26, 1), (.75, 2), (.74, 1), (1.25, 2), (1.75, 4), (2.5, 4), (2.51, 5), (3.5, 6),
                 (5, 6), (5.1, 7), (6, 7), (100, 7), (np.inf, 7), (-.75, 10), (-0.0, 8)]:
        assert f4.e2m1_code(np.float64(v)) == c, v


def test_rows_keep_what_they_can():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((64, 576))
    y = f4.decode_rows(f4.encode(x[:, :512], x[:, 512:], np.float32(1.0)))
    # A block's scale is off by 2^-4 of itself at most, a code by half a step: 1 of 6 where the largest code is.
    top = np.abs(x[:, :512]).reshape(64, 32, 16).max(2)
    assert (np.abs(y - x)[:, :512].reshape(64, 32, 16) <= top[..., None] * (1 + 2 ** -4) / 6 + 1e-12).all()
    assert (np.abs(y - x)[:, 512:] <= np.abs(x[:, 512:]) * 2.0 ** -11 + 2.0 ** -25).all()


def test_plans_take_4_bit_caches():
    p = mla.plan([300, 20], 16, 1, 64, mla.KV_FP4_E2M1, num_sms=152)
    assert p.kv_dtype == mla.KV_FP4_E2M1 and p.key_tile == 128 and (p.grid_x, p.grid_y) == (1, 2)
    assert mla.plan([300, 20], 32, 1, 64, mla.KV_FP4_E2M1, num_sms=152).key_tile == 128
    p = mla.plan([300, 20], 33, 1, 64, mla.KV_FP4_E2M1, num_sms=152)
    assert p.key_tile == 64 and (p.grid_x, p.grid_y) == (2, 2)
    d = mla.dplan_info(2, 16, 2, 64, mla.KV_FP4_E2M1, False, 300, 152)
    assert d.key_tile == 128 and d.row_blocks == 1 and mla.dplan_info(2, 33, 1, 64, mla.KV_FP4_E2M1, False, 300, 152).key_tile == 64


@pytest.mark.parametrize("dtype", [2, 3, 5, -1])
def test_other_types_are_refused(dtype):
    with pytest.raises(mla.MLADecodeError) as e:
        mla.plan([300], 16, 1, 64, dtype, num_sms=152)
    assert e.value.status == mla.ERR_INVALID_ARG


def test_calls_without_a_4_bit_form_say_so():
    with pytest.raises(mla.MLADecodeError) as e:
        mla.prefix_plan([300], 100, 16, 1, 64, mla.KV_FP4_E2M1, num_sms=152)
    assert e.value.status == mla.ERR_UNSUPPORTED
    at = ctypes.c_void_p(1 << 20)  # never read: refused first
    st = mla.lib().mla_gather_kv_b_proj(at, 4, 16, mla.KV_FP4_E2M1, at, at, 4, at, at, 1, 64, at, 8, at, at, at, None)
    assert st == mla.ERR_UNSUPPORTED


def test_inserts_need_a_scale():
    at = ctypes.c_void_p(1 << 20)
    args = [at, at, at, at, at, 4, 8, at, at, 4, 16, mla.KV_FP4_E2M1, None, 0, None, None]
    assert mla.lib().mla_decode_epilogue(*args) == mla.ERR_INVALID_ARG
    p = mla.plan([64], 8, 1, 16, mla.KV_FP4_E2M1, num_sms=152)
    st = mla.lib().mla_decode_step(ctypes.byref(p), at, at, at, at, at, 0, at, at, 4, None, at, 4, at, 0.1, at, at, at,
                                   int(p.workspace_bytes), None)
    assert st == mla.ERR_INVALID_ARG


@pytest.mark.parametrize("dtype,shape", [("uint8", (4, 16, 576)), ("bfloat16", (4, 16, 576)), ("uint8", (4, 8, 416)),
                                         ("uint8", (64, 416)), ("bfloat16", (4, 16, 416))])
def test_a_plan_and_a_cache_of_other_rows(dtype, shape):
    import torch
    p = mla.plan([64], 8, 1, 16, mla.KV_FP4_E2M1, num_sms=152)
    d = mla.dplan_info(1, 8, 1, 16, mla.KV_FP4_E2M1, False, 64, 152)
    z, cache = torch.zeros(1, 64, dtype=torch.int32), torch.zeros(shape, dtype=getattr(torch, dtype))
    for call in (lambda: mla.fwd(p, z, cache, None, z, z, 0.1, z, z, z), lambda: mla.fwd_dplan(d, z, cache, None, z, 0.1, z, z, z),
                 lambda: mla.step(p, z, z, z, z, z, z, cache, None, z, z, 0.1, z, z, z)):
        with pytest.raises(mla.MLADecodeError) as e:
            call()
        assert e.value.status == mla.ERR_INVALID_ARG


def test_a_4_bit_cache_and_another_plan():
    import torch
    p = mla.plan([64], 8, 1, 16, mla.KV_FP8_E4M3, num_sms=152)
    z, cache = torch.zeros(1, 64, dtype=torch.int32), torch.zeros(4, 16, 416, dtype=torch.uint8)
    with pytest.raises(mla.MLADecodeError):
        mla.fwd(p, z, cache, None, z, z, 0.1, z, z, z)
