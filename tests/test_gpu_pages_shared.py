"""A row cut back into a page that others hold: no token of its own goes there, and the way on is a copy by fork."""
import numpy as np
import pytest

from pages_book import Book, Gpu

pytestmark = pytest.mark.gpu

FORMS = [(60, 16, 8), (33000, 16, 8)]  # one launch a call, a kernel a step


def filled(b):
    """Every row's tokens say whose they are: of row r, token j, all bytes 40 r + j."""
    for r, n in enumerate(b.lens):
        for j in range(int(n)):
            b.cache[:, b.table[r, j // b.page], j % b.page] = (40 * r + j) % 251


def two_beams(pages, page, width):
    """Rows 0 and 1 share two whole pages and each has its own third; row 0 is then cut back into the second."""
    b = Book(pages, page, 2, width, 2, 32, seed=1)
    b.scatter(1, 0.3)
    b.resize([33, 0])
    filled(b)
    b.fork([0, 0], np.zeros((2, width), np.int32))
    b.resize([31, 33])
    assert b.refs[b.table[0, 1]] == 2 and b.table[0, 1] == b.table[1, 1]
    return b, Gpu(b)


@pytest.mark.parametrize("pages,page,width", FORMS)
@pytest.mark.parametrize("grow", [1, 3, 20])
def test_no_slot_in_a_page_that_others_hold(pages, page, width, grow):
    b, g = two_beams(pages, page, width)
    slots = g.resize([31 + grow, 33 + grow], grow).cpu().numpy()
    want, _ = b.resize([31 + grow, 33 + grow], grow)  # the plain book hands out that slot
    assert want[0, 0] == int(b.table[1, 1]) * page + 15  # row 1's token 31
    want[0, 0] = -1
    assert np.array_equal(slots, want)
    g.same_as(b)  # pages, counts and lengths are as ever
    assert g.flags() == g.mla.DEVFLAG_SHARED
    sibling = {int(p) * page + o for p in b.table[1, :2] for o in range(page)}
    assert not sibling & set(slots[0].tolist())


@pytest.mark.parametrize("pages,page,width", FORMS)
def test_what_is_given_back_in_the_same_call_is_not_shared(pages, page, width):
    b, g = two_beams(pages, page, width)
    slots = g.resize([32, 5], 1).cpu().numpy()
    want, _ = b.resize([32, 5], 1)
    assert want[0, 0] >= 0 and np.array_equal(slots, want) and g.flags() == 0
    g.same_as(b)


@pytest.mark.parametrize("pages,page,width", FORMS)
def test_two_rows_that_both_grow_in_one_page_get_no_slot(pages, page, width):
    b, g = two_beams(pages, page, width)
    for x in (b, g):
        x.resize([20, 29])
    g.flags()
    slots = g.resize([21, 30], 2).cpu().numpy()
    assert (slots == -1).all() and g.flags() == g.mla.DEVFLAG_SHARED and g.lens.tolist() == [21, 30]


@pytest.mark.parametrize("pages,page,width", FORMS)
def test_a_page_that_does_not_exist_gives_no_slot(pages, page, width):
    for bad in (-1, pages, 1 << 30):
        b, g = two_beams(pages, page, width)
        g.table[0, 1] = bad
        slots = g.resize([32, 33], 1).cpu().numpy()
        assert slots[0, 0] == -1 and g.flags() == g.mla.DEVFLAG_BAD_PAGE


@pytest.mark.parametrize("pages,page,width", FORMS)
def test_going_on_from_it_twice_gives_a_page_of_its_own(pages, page, width):
    """parents 0, 0, 1: the second child of row 0 has a copy; the first is let go by the next fork."""
    b, g = two_beams(pages, page, width)
    before = [b.rows(r).copy() for r in range(2)]
    for parents in ([0, 0, 1], [1, 2]):
        table = np.zeros((len(parents), width), np.int32)
        b.fork(parents, table.copy())
        g.fork(parents, table)
        g.same_as(b, parents)
    slots = g.resize([33, 34], 2).cpu().numpy()
    want, _ = b.resize([33, 34], 2)
    assert np.array_equal(slots, want) and (slots[0] >= 0).all() and g.flags() == 0
    for x in (b.cache, g.cache):
        for s in slots.ravel():
            if s >= 0:
                x[:, int(s) // page, int(s) % page] = 255
    g.same_as(b)
    for r, n in enumerate([31, 33]):
        assert np.array_equal(b.rows(r)[:, :n], before[r])
        assert (b.rows(r)[:, n:] == 255).all()
