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


def said(c, names):
    return [c.said(n) if n in c._table else None for n in names]


def test_parents_of_several_requests_count_within_each():
    """[requests][keep], as ttq_beam_select gives them, in one call and one launch."""
    c = Cache(60)
    names = [f"{r}{w}" for r in "xy" for w in range(3)]
    for r, tokens in (("x", 6), ("y", 9)):
        for t in range(tokens):
            c.say(r + "0", r + str(t))
        c.fork(r + "0", [r + "1", r + "2"])
    for n in names:
        c.say(n, "of " + n)
    was = dict(zip(names, said(c, names)))
    launches = c.launches
    c.reorder(names, [[2, 0, 0], [1, 1, 2]])
    assert c.launches == launches + 1
    assert said(c, names) == [was[n] for n in ("x2", "x0", "x0", "y1", "y1", "y2")]
    c.check()
    was = dict(zip(names, said(c, names)))
    more = [f"{r}{w}" for r in "xy" for w in range(5)]  # more beams than before
    c.reorder(names, [[0, 1, 2, 0, 1], [0, 0, 0, 0, 0]], more)
    assert said(c, more) == [was[n] for n in ("x0", "x1", "x2", "x0", "x1") + ("y0",) * 5]
    c.check()


def test_beams_that_end():
    """A parent of -1: the name is left without a sequence, and is free to be one of seqs in the next step."""
    c = Cache(40)
    names = [f"{r}{w}" for r in "xy" for w in range(3)]
    for r in "xy":
        for t in range(6):
            c.say(r + "0", r + str(t))
        c.fork(r + "0", [r + "1", r + "2"])
    for n in names:
        c.say(n, "of " + n)
    was = dict(zip(names, said(c, names)))
    c.reorder(names, [[2, 2, -1], [-1, -1, -1]])
    assert said(c, names) == [was["x2"], was["x2"], None, None, None, None]
    c.check()
    c.say("x1", "last")
    was = dict(zip(names, said(c, names)))
    before = dict(c._table)
    for bad in ([[2, 0, 0], [-1, -1, -1]], [[0, 0, 0], [0, -1, -1]]):  # beams that have ended go on
        with pytest.raises(ValueError):
            c.reorder(names, bad)
        assert c._table == before
    c.reorder(names, [[1, 0, 1], [-1, -1, -1]])
    assert said(c, names) == [was["x1"], was["x0"], was["x1"], None, None, None]
    c.check()
    c.reorder(names, [[-1, -1, -1], [-1, -1, -1]])
    assert c.free_pages == 40
    c.reorder(names, [[-1, -1, -1], [-1, -1, -1]])


@pytest.mark.parametrize("parents,names", [
    ([[0, 1, 2], [0]], None), ([[0, 1], [0, 1], [0, 1], [0, 1]], "abcdefgh"), ([[0, 3, 1], [0, 1, 2]], None),
    ([[0, -2, 1], [0, 1, 2]], None), ([[0], [1]], None), ([[0], [1]], ["a", "a"]), ([[0], [1]], ["a", "other"]),
    ([[0, 1, 2], 3], None), ([0, [1, 2, 0]], None)])
def test_refused_parents_of_requests(parents, names):
    c = Cache(40)
    for n in "abcdef":
        c.extend(n, 5)
    c.extend("other", 5)
    was = dict(c._table), dict(c._len), list(c._owners), list(c._free)
    with pytest.raises((ValueError, TypeError)):
        c.reorder(list("abcdef"), parents, names)
    assert (dict(c._table), dict(c._len), list(c._owners), list(c._free)) == was


def test_tensors_of_parents():
    import torch
    c = Cache(40)
    for n in "abcd":
        c.say(n, n)
    c.reorder(list("abcd"), torch.tensor([[1, 1], [0, -1]]))
    assert said(c, "abcd") == [["b"], ["b"], ["c"], None]
    c.reorder(list("abc"), torch.tensor([2, 0, 0]))
    assert said(c, "abc") == [["c"], ["b"], ["b"]]
