"""Compact writes neither into what it reads nor twice to one place: refused before anything is queued."""
import pytest

import paged_mla_decode_latent_gb300 as mla


@pytest.fixture(scope="module", autouse=True)
def built():
    mla.build()


def at(n):
    return n << 20


ARGS = dict(refs=at(1), pages=100, table=at(2), stride=10, width=10, lens=at(3), rows=4, ps=16, cache=at(7), layers=1,
            layer_stride=0, row=576, map=at(4), n=at(5), status=None, ws=at(8), nws=1 << 20)


@pytest.mark.parametrize("kw", [
    dict(map=at(1)), dict(map=at(1) + 4 * 99), dict(n=at(1)), dict(n=at(1) + 4 * 99),  # the counts
    dict(map=at(2)), dict(map=at(2) - 4 * 99), dict(n=at(2) + 4 * 39),  # the table
    dict(map=at(3)), dict(n=at(3) + 12),  # the lengths
    dict(n=at(4)), dict(n=at(4) + 4 * 99)])  # each other
def test_compact_refuses_overlaps(kw):
    assert mla.lib().mla_pages_compact(*{**ARGS, **kw}.values(), None) == mla.ERR_INVALID_ARG
