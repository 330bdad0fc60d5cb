"""Limits of the shared-prefix plan: contexts near 2^31, and the deal of tiles to CTA pairs."""
import pytest

import paged_mla_decode_latent_gb300 as mla


@pytest.fixture(scope="module", autouse=True)
def built():
    mla.build()


@pytest.mark.parametrize("heads,dtype", [(128, mla.KV_BF16), (16, mla.KV_BF16), (8, mla.KV_FP8_E4M3)])
@pytest.mark.parametrize("batch", [1, 200])
@pytest.mark.parametrize("prefix", [0, 100, 1 << 22])
def test_own_keys_end_below_2_31(heads, dtype, batch, prefix):
    """The kernels count keys in int32: a chunk of own keys must not end past it."""
    planned = 0
    for n in (2 ** 31 - 1, 2 ** 31 - 65, 2 ** 31 - 2 ** 20, 2 ** 31 - 2 ** 26, 2 ** 30):
        try:
            p = mla.prefix_plan([n] * batch, prefix, heads, 1, 4096, dtype, False, 152)
        except mla.MLADecodeError as e:
            assert e.status == mla.ERR_UNSUPPORTED
            continue
        planned += 1
        assert p.own_chunk > 0
        assert p.prefix_len + p.own_splits * p.own_chunk < 2 ** 31
        assert p.own_splits * p.own_chunk >= n - prefix
    assert planned > 0 or batch > 1
