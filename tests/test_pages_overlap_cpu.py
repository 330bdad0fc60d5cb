"""Fork writes neither into what it reads nor twice to one place: refused before anything is queued."""
import pytest

import paged_mla_decode_latent_gb300 as mla


@pytest.fixture(scope="module", autouse=True)
def built():
    mla.build()


def at(n):
    return n << 20


ARGS = dict(refs=at(1), pages=100, table=at(2), stride=10, width=10, lens=at(3), rows=4, parents=at(4), out=at(5),
            out_stride=10, lens_out=at(6), out_rows=4, ps=16, cache=at(7), layers=1, layer_stride=0, row=576,
            status=None, ws=at(8), nws=1 << 20)


@pytest.mark.parametrize("kw", [
    dict(out=at(4)), dict(out=at(4) + 12), dict(out=at(4) - 4 * 39), dict(parents=at(5) + 4 * 39),  # parents
    dict(out=at(3)), dict(out=at(3) - 4 * 39),  # the old lengths
    dict(lens_out=at(2)), dict(lens_out=at(2) + 4 * 39),  # the old table
    dict(lens_out=at(5)), dict(lens_out=at(5) + 4 * 39), dict(lens_out=at(5) - 12),  # the new table
    dict(out=at(1)), dict(out=at(1) + 4 * 99), dict(lens_out=at(1)), dict(lens_out=at(1) + 4 * 99)])  # the counts
def test_fork_refuses_overlaps(kw):
    assert mla.lib().mla_pages_fork(*{**ARGS, **kw}.values(), None) == mla.ERR_INVALID_ARG
