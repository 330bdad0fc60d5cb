"""Refusals of the page calls (before anything is queued), and the plain book's own sums."""
import ctypes

import numpy as np
import pytest

import paged_mla_decode_latent_gb300 as mla
from pages_book import Book


@pytest.fixture(scope="module", autouse=True)
def built():
    mla.build()


def at(n):
    return n << 20


RESIZE = dict(refs=at(1), pages=100, table=at(2), stride=10, width=10, lens=at(3), new=at(4), rows=4, ps=16, slots=at(5),
              tokens=2, status=None, ws=at(6), nws=1 << 20)
FORK = dict(refs=at(1), pages=100, table=at(2), stride=10, width=10, lens=at(3), rows=4, parents=at(4), out=at(5),
            out_stride=10, lens_out=at(6), out_rows=4, ps=16, cache=at(7), layers=2, layer_stride=100 * 16 * 576, row=576,
            status=None, ws=at(8), nws=1 << 20)
COMPACT = dict(refs=at(1), pages=100, table=at(2), stride=10, width=10, lens=at(3), rows=4, ps=16, cache=at(7), layers=2,
               layer_stride=100 * 16 * 576, row=576, map=at(4), n=at(5), status=None, ws=at(8), nws=1 << 20)


def call(name, args, **kw):
    assert set(kw) <= set(args)
    return getattr(mla.lib(), name)(*{**args, **kw}.values(), None)


BOOK = [dict(refs=None), dict(refs=at(1) + 4), dict(pages=0), dict(pages=-1), dict(pages=2 ** 31 - 1), dict(ps=0), dict(ps=4097),
        dict(table=None), dict(table=at(2) + 2), dict(stride=9), dict(width=0), dict(lens=None), dict(lens=at(3) + 1),
        dict(rows=-1), dict(rows=65536), dict(status=at(9) + 2)]
CACHE = [dict(cache=None), dict(cache=at(7) + 8), dict(layers=0), dict(row=0), dict(row=24), dict(row=(1 << 20) + 16),
         dict(layer_stride=100 * 16 * 576 - 16), dict(layer_stride=100 * 16 * 576 + 8), dict(layer_stride=-(1 << 30))]


@pytest.mark.parametrize("kw", BOOK + [dict(new=None), dict(new=at(4) + 2), dict(new=at(3)), dict(new=at(3) + 4), dict(slots=None),
                                       dict(slots=at(5) + 4), dict(tokens=-1)])
def test_resize_refuses(kw):
    assert call("mla_pages_resize", RESIZE, **kw) == mla.ERR_INVALID_ARG


@pytest.mark.parametrize("kw", BOOK + CACHE + [
    dict(rows=0), dict(parents=None), dict(parents=at(4) + 1), dict(out=None), dict(out=at(5) + 2), dict(out=at(2)),
    dict(out=at(2) + 4 * 39), dict(out_stride=9), dict(lens_out=None), dict(lens_out=at(3)), dict(lens_out=at(4) + 4),
    dict(out_rows=-1), dict(out_rows=65536)])
def test_fork_refuses(kw):
    assert call("mla_pages_fork", FORK, **kw) == mla.ERR_INVALID_ARG


@pytest.mark.parametrize("kw", BOOK + CACHE + [dict(map=None), dict(map=at(4) + 2), dict(n=None), dict(n=at(5) + 2)])
def test_compact_refuses(kw):
    assert call("mla_pages_compact", COMPACT, **kw) == mla.ERR_INVALID_ARG


@pytest.mark.parametrize("name,args", [("mla_pages_resize", RESIZE), ("mla_pages_fork", FORK), ("mla_pages_compact", COMPACT)])
@pytest.mark.parametrize("kw", [dict(ws=None), dict(ws=at(8) + 128), dict(nws=64)])
def test_workspaces(name, args, kw):
    assert call(name, args, **kw) == mla.ERR_WORKSPACE


def test_a_workspace_of_the_size_that_is_named_fits():
    n = mla.lib().mla_pages_workspace_bytes(100, 4)
    assert n > 0 and call("mla_pages_resize", RESIZE, nws=n - 1) == mla.ERR_WORKSPACE
    assert call("mla_pages_resize", RESIZE, nws=mla.lib().mla_pages_workspace_bytes(100, 0), rows=0) == mla.OK
    for pages, rows in [(0, 4), (2 ** 31 - 1, 4), (100, -1), (100, 65536)]:
        assert mla.lib().mla_pages_workspace_bytes(pages, rows) == -1
    with pytest.raises(mla.MLADecodeError):
        mla.pages_workspace(0, 4)


def test_a_cache_past_any_memory():
    kw = dict(pages=2 ** 31 - 2, ps=4096, row=1 << 20, layers=1, nws=1 << 62)
    assert call("mla_pages_compact", COMPACT, **kw) == mla.ERR_UNSUPPORTED


def test_bindings_refuse_host_tensors():
    import torch
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    ws, cache = torch.zeros(1 << 16, dtype=torch.uint8), torch.zeros(10, 16, 576, dtype=torch.bfloat16)
    for f in (lambda: mla.pages_resize(i(10), i(2, 4), i(2), i(2), 16, ws),
              lambda: mla.pages_fork(i(10), i(2, 4), i(2), i(2), i(2, 4), i(2), cache, ws),
              lambda: mla.pages_compact(i(10), i(2, 4), i(2), cache, i(10), i(1), ws)):
        with pytest.raises(mla.MLADecodeError) as e:
            f()
        assert e.value.status == mla.ERR_INVALID_ARG


def test_the_plain_book_adds_up():
    b = Book(60, 4, 5, 12, layers=2, seed=1)
    b.resize([9, 0, 17, 4, 30])
    for r in range(5):
        for j in range(int(b.lens[r])):
            b.cache[:, b.table[r, j // 4], j % 4] = (17 * r + j) % 256
    want = [b.rows(r).copy() for r in range(5)]
    parents = [4, 0, 0, 2, -1, 0]
    b.fork(parents, np.full((6, 12), -9, np.int32))
    b.compact()
    for i, r in enumerate(parents):
        assert b.lens[i] == 0 if r < 0 else np.array_equal(b.rows(i), want[r])
    assert (b.refs > 0).sum() == np.flatnonzero(b.refs).max() + 1
    b.resize([0] * 6)
    assert not b.refs.any()
