"""What PagedCache.reorder costs the host, by the comparisons of pages that it makes."""
import pytest

from test_beams_host import Cache


class Page(int):
    """A page's number that counts how often it is compared with another one."""
    compared = 0

    def __eq__(self, other):
        Page.compared += 1
        return int(self) == int(other)

    __hash__ = int.__hash__


@pytest.mark.parametrize("beams,shared", [(4, 60), (8, 500), (16, 500)])
def test_the_cost_grows_with_the_pages_not_with_their_square(beams, shared):
    """Beams over a long shared context, half of which end: at most some comparisons for each page of each of them."""
    c = Cache(shared + 4 * beams)
    c._free = [Page(p) for p in c._free]
    names = list(range(beams))
    c.extend(0, shared * c.page_size + 1)
    c.fork(0, names[1:])
    Page.compared = 0
    c.reorder(names, [i // 2 for i in range(beams)])
    assert Page.compared <= 4 * beams * shared
    c.check()
    assert all(c.pages_of(n)[:shared] == c.pages_of(0)[:shared] for n in names)
    assert len({c.pages_of(n)[-1] for n in names}) == beams
