"""Host side of the shared-prefix decode: the plan and the refusals."""
import ctypes

import numpy as np
import pytest

import paged_mla_decode_latent_gb300 as mla


@pytest.fixture(scope="module", autouse=True)
def built():
    mla.build()


def share(total, pairs, i):
    return total * i // pairs


@pytest.mark.parametrize("batch,heads,sq,prefix,own,sms", [
    (1, 1, 1, 1, 0, 152), (4, 16, 1, 512, 64, 152), (64, 128, 1, 8192, 512, 152),
    (13, 12, 3, 4999, 333, 152), (128, 128, 1, 23333, 512, 152), (3, 100, 1, 255, 1, 2),
    (7, 128, 8, 100000, 10, 148), (2, 16, 1, 0, 90, 152), (5, 64, 1, 257, 0, 37),
    (64, 128, 1, 100, 20000, 152), (130, 1, 1, 600, 40, 152), (9, 5, 3, 700, 10, 152)])
def test_plan(batch, heads, sq, prefix, own, sms):
    lens = [prefix + (own * (b + 1)) // batch for b in range(batch)]
    p = mla.prefix_plan(lens, prefix, heads, sq, 16, mla.KV_BF16, sq > 1, sms)
    rows = heads * sq
    assert p.total_rows == batch * rows and p.row_blocks == -(-p.total_rows // 128)
    assert p.prefix_tiles == -(-prefix // 256) and p.max_ctx == max(lens)
    most = max(lens) - prefix
    seqs = max(min(batch - 1, (128 * j + 127) // rows) - 128 * j // rows + 1 for j in range(p.row_blocks))
    if p.own_folded:
        # Room for every sequence at its longest, in whole tiles; no decode of its own.
        assert prefix > 0 and p.own_splits == 0
        assert p.block_keys % 256 == 0 and p.block_keys >= seqs * most
        assert p.row_blocks * p.block_keys * 1152 < 2 ** 30
    else:
        assert p.block_keys == 0 and p.own_splits * p.own_chunk >= most
        assert p.own_chunk % p.key_tile == 0 and (p.own_splits == 0) == (most == 0)
    if prefix:
        own_keys = [sum(lens[b] - prefix for b in range(128 * j // rows, min(batch - 1, (128 * j + 127) // rows) + 1))
                    for j in range(p.row_blocks)]
        tiles = p.row_blocks * p.prefix_tiles + p.own_folded * sum(-(-k // 256) for k in own_keys)
        assert 1 <= p.pairs <= min(max(1, sms // 2), tiles)
    else:
        assert p.pairs == 0 and not p.own_folded
    segments = p.row_blocks + p.pairs if prefix else 0
    keys = 256 * p.prefix_tiles + p.row_blocks * p.block_keys
    offs = [p.ws_status_offset, p.ws_partition_offset, p.ws_keys_offset, p.ws_q_offset,
            p.ws_prefix_o_offset, p.ws_prefix_lse_offset, p.ws_own_o_offset, p.ws_own_lse_offset,
            p.workspace_bytes]
    sizes = [16 + (keys + p.total_rows if prefix else 0),
             20 * p.row_blocks + 16 * (p.pairs + 1) + (4 * p.row_blocks * seqs if p.own_folded else 0),
             keys * 1152 if prefix else 0, p.total_rows * 1152 if prefix else 0,
             segments * 128 * 2048, segments * 128 * 4,
             p.own_splits * p.total_rows * 2048, p.own_splits * p.total_rows * 4]
    for a, b, n in zip(offs, offs[1:], sizes):
        assert a % 256 == 0 and b - a >= n


def test_own_tiles_have_pairs_too():
    """Two shared tiles and seven of own keys: more than the two pairs that the shared ones could use."""
    p = mla.prefix_plan([512 + 200] * 8, 512, 16, 1, 16, 0, False, 152)
    assert p.own_folded and p.prefix_tiles == 2 and p.pairs > 4


def test_own_keys_fold_in_or_not():
    """Short own keys become tiles of their row blocks, long ones are decoded apart."""
    assert mla.prefix_plan([8192 + 80] * 64, 8192, 128, 1, 16, 0, False, 152).own_folded == 1
    assert mla.prefix_plan([1024 + 100000] * 16, 1024, 128, 1, 16, 0, False, 152).own_folded == 0


def test_folded_regions_stay_small():
    """Thousands of row blocks: a tile each for a key each would take gigabytes."""
    assert mla.prefix_plan([101] * 4000, 100, 128, 1, 16, 0, False, 152).own_folded == 1
    p = mla.prefix_plan([101] * 8000, 100, 128, 1, 16, 0, False, 152)
    assert p.own_folded == 0 and p.own_splits == 1


def test_struct_layout():
    assert ctypes.sizeof(mla.PrefixPlan) == 22 * 4 + 9 * 8


@pytest.mark.parametrize("kw", [
    dict(lens=[-1]), dict(lens=[]), dict(prefix=-1), dict(prefix=(1 << 22) + 1), dict(heads=0),
    dict(heads=129), dict(sq=0), dict(sq=17), dict(heads=128, sq=9), dict(page=0), dict(page=4097),
    dict(dtype=2)])
def test_plan_refuses(kw):
    a = dict(lens=[100], prefix=64, heads=16, sq=1, page=16, dtype=0)
    a.update(kw)
    with pytest.raises(mla.MLADecodeError) as e:
        mla.prefix_plan(a["lens"], a["prefix"], a["heads"], a["sq"], a["page"], a["dtype"], False, 152)
    assert e.value.status == mla.ERR_INVALID_ARG


def test_plan_refuses_too_many_rows():
    with pytest.raises(mla.MLADecodeError) as e:
        mla.prefix_plan([1] * 65535, 1, 128, 8, 1, 0, True, 152)
    assert e.value.status == mla.ERR_UNSUPPORTED


def fwd(plan, **kw):
    """mla_decode_prefix_fwd on made-up aligned addresses: every refusal comes before any use."""
    a = dict(q=1 << 20, cache=2 << 20, pages=64, scale=None, pt=3 << 20, bt=4 << 20, stride=16,
             lens=5 << 20, softmax=0.07, out=6 << 20, lse=7 << 20, ws=8 << 20,
             bytes=plan.workspace_bytes)
    a.update(kw)
    return mla.lib().mla_decode_prefix_fwd(
        ctypes.byref(plan), a["q"], a["cache"], a["pages"], a["scale"], a["pt"], a["bt"],
        a["stride"], a["lens"], a["softmax"], a["out"], a["lse"], a["ws"], a["bytes"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), -1), (dict(cache=None), -1), (dict(pt=None), -1), (dict(bt=None), -1),
    (dict(lens=None), -1), (dict(out=None), -1), (dict(lse=None), -1), (dict(q=(1 << 20) + 2), -1),
    (dict(cache=(1 << 20) + 8), -1), (dict(out=(1 << 20) + 8), -1), (dict(pt=(1 << 20) + 2), -1),
    (dict(scale=(1 << 20) + 1), -1), (dict(pages=0), -1), (dict(pages=1 << 30), -2),
    (dict(stride=6), -1), (dict(softmax=float("nan")), -1), (dict(softmax=float("inf")), -1),
    (dict(softmax=-1.0), -1), (dict(ws=None), -3), (dict(ws=(8 << 20) + 16), -3), (dict(bytes=100), -3)])
def test_fwd_refuses(kw, status):
    plan = mla.prefix_plan([100, 120], 64, 16, 1, 16, 0, False, 152)
    assert fwd(plan, **kw) == status


@pytest.mark.parametrize("field,value", [
    ("version", 0), ("batch", 0), ("rows", 17), ("total_rows", 33), ("prefix_len", 600),
    ("prefix_tiles", 2), ("pairs", 0), ("pairs", 100), ("pairs", -1), ("own_splits", 400),
    ("own_folded", 2), ("own_folded", 0), ("block_keys", 0), ("max_ctx", 1 << 29), ("own_chunk", 100),
    ("key_tile", 64), ("wait_limit_us", -1), ("kv_dtype", 7), ("page_size", 0),
    ("ws_q_offset", 256), ("workspace_bytes", 512)])
def test_fwd_refuses_an_edited_plan(field, value):
    plan = mla.prefix_plan([100, 120], 64, 16, 1, 16, 0, False, 152)
    setattr(plan, field, value)
    assert fwd(plan) == mla.ERR_INVALID_ARG


def test_plan_is_quick():
    import time
    t0 = time.perf_counter()
    for _ in range(3):
        mla.prefix_plan(np.full(128, 23500), 23333, 128, 1, 16, 0, False, 152)
    assert (time.perf_counter() - t0) / 3 < 0.25


def test_binding_refuses_host_tensors():
    import torch
    p = mla.prefix_plan([100, 120], 64, 16, 1, 16, 0, False, 152)
    z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t)  # noqa: E731
    with pytest.raises(mla.MLADecodeError) as e:
        mla.prefix_fwd(p, z(2, 1, 16, 576), z(20, 16, 576), None, z(4, t=torch.int32), z(2, 8, t=torch.int32),
                       z(2, t=torch.int32), 0.07, z(2, 1, 16, 512), z(2, 1, 16, t=torch.float32),
                       z(int(p.workspace_bytes), t=torch.uint8))
    assert e.value.status == mla.ERR_INVALID_ARG
