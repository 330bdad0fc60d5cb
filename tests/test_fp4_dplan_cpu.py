"""Sizes of the device plan: the shortest chunk that it names is the one that it cuts."""
import pytest

import paged_mla_decode_latent_gb300 as mla


@pytest.fixture(scope="module", autouse=True)
def built():
    mla.build()


# keys that a tile of the decode kernel has, two of which are the shortest chunk
@pytest.mark.parametrize("heads,sq,kv_dtype,tile", [
    (16, 1, mla.KV_FP4_E2M1, 128), (32, 1, mla.KV_FP4_E2M1, 128), (33, 1, mla.KV_FP4_E2M1, 256),
    (64, 1, mla.KV_FP4_E2M1, 256), (128, 1, mla.KV_FP4_E2M1, 256), (64, 16, mla.KV_FP4_E2M1, 256),
    (16, 1, mla.KV_BF16, 128), (128, 1, mla.KV_BF16, 64), (16, 1, mla.KV_FP8_E4M3, 128), (128, 1, mla.KV_FP8_E4M3, 64)])
def test_shortest_chunk(heads, sq, kv_dtype, tile):
    d = mla.dplan_info(4, heads, sq, 16, kv_dtype, False, 4096, 152)
    assert d.min_chunk_keys == 2 * tile
