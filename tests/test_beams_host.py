"""The host side of the beams: refusals of ttq_beam_select before any launch, and
the bookkeeping of PagedCache.reorder."""
import ctypes
import random

import pytest

import test_activation_aware_amd as ttq
from test_serving_host import ALIGN, INVALID, MIS, NULL, OK, P, SHAPE, lib  # noqa: F401


def test_refusals(lib):
    def f(x=P, dt=0, requests=2, beams=4, V=100, ldl=100, scores=P, keep=8, out=P, parents=P, tokens=P, history=P, ldh=10,
          length=10, oh=P, ldo=11, ws=P, n=1 << 40):
        return lib.ttq_beam_select(x, dt, requests, beams, V, ldl, scores, keep, out, parents, tokens, history, ldh, length,
                                   oh, ldo, ws, n, None)

    odd = ctypes.c_void_p((1 << 20) + 1)
    assert f(dt=7) == INVALID and f(beams=0) == SHAPE and f(beams=65) == SHAPE and f(requests=-1) == SHAPE
    assert f(requests=1 << 30) == SHAPE and f(V=0, ldl=0) == SHAPE and f(V=(1 << 23) + 1, ldl=1 << 24) == SHAPE
    assert f(ldl=99) == SHAPE and f(ldl=1 << 50) == SHAPE and f(keep=0) == INVALID and f(keep=65) == INVALID
    assert f(length=-1) == SHAPE and f(ldh=9) == SHAPE and f(ldo=10) == SHAPE and f(ldo=1 << 45) == SHAPE
    assert f(length=1 << 41, ldh=1 << 41, ldo=1 << 42) == SHAPE
    assert f(requests=1 << 25, beams=1, V=1, ldl=1) == SHAPE      # more threads than a launch holds
    assert f(x=None) == NULL and f(x=odd) == ALIGN and f(scores=None) == NULL and f(scores=MIS) == ALIGN
    assert f(out=None) == NULL and f(parents=None) == NULL and f(tokens=MIS) == ALIGN
    assert f(history=None) == NULL and f(oh=MIS) == ALIGN
    assert f(ws=None) == NULL and f(ws=MIS) == ALIGN
    need = lib.ttq_beam_select_workspace_bytes(2, 4, 100, 8)
    assert need > 0 and f(n=need - 1) == SHAPE and b"workspace" in lib.ttq_last_error()
    assert f(requests=0, x=None, scores=None) == OK
    for bad in ((0, 4, 100, 8), (2, 0, 100, 8), (2, 65, 100, 8), (2, 4, 0, 8), (2, 4, 100, 0), (2, 4, 100, 65), (1 << 40, 4, 100, 8)):
        assert lib.ttq_beam_select_workspace_bytes(*bad) == 0


class Cache(ttq.PagedCache):
    """Pages on the CPU; copies are written down, and moved in `held`."""

    def __init__(self, pages, page_size=4):
        super().__init__(1, pages, 1, 64, page_size=page_size, device="cpu")
        self.held = [[] for _ in range(pages)]
        self.launches, self.fail = 0, False

    def _copy(self, src, dst, table=None):
        assert not set(src) & set(dst) and len(set(dst)) == len(dst)
        if self.fail:
            raise RuntimeError("no launch")
        self.launches += 1
        for a, b in zip(src, dst):
            self.held[b] = list(self.held[a])

    def say(self, seq, token):
        at = self._len.get(seq, 0)
        self.extend(seq, 1)
        page = self.held[self.pages_of(seq)[at // self.page_size]]
        del page[at % self.page_size:]
        page.append(token)

    def said(self, seq):
        out = []
        for i, p in enumerate(self.pages_of(seq)):
            out += self.held[p][:min(self.page_size, self.length(seq) - i * self.page_size)]
        return out

    def check(self):
        count = [0] * self.pages
        for t in self._table.values():
            for p in t:
                count[p] += 1
        assert count == self._owners
        assert sorted(self._free) == [p for p in range(self.pages) if count[p] == 0]


@pytest.mark.parametrize("seed", range(6))
def test_beams_go_on(seed):
    r = random.Random(seed)
    c = Cache(60)
    names = [f"beam {i}" for i in range(r.choice([1, 3, 5]))]
    for t in range(r.randint(1, 9)):
        c.say(names[0], t)
    c.fork(names[0], names[1:])
    c.extend("other", 5)
    truth = {n: c.said(n) for n in names}
    token = 100
    for _ in range(40):
        parents = [r.randrange(len(names)) for _ in names]
        before = c.launches
        c.reorder(names, parents)
        assert c.launches <= before + 1
        truth = {n: list(truth[names[p]]) for n, p in zip(names, parents)}
        c.check()
        for n in names:
            if r.random() < 0.9:
                c.say(n, token)
                truth[n].append(token)
                token += 1
        assert {n: c.said(n) for n in names} == truth
        c.check()
        if len(truth[names[0]]) > 25:
            break


def test_other_numbers_and_names():
    c = Cache(20)
    for t in range(6):
        c.say("a", t)
    c.reorder(["a"], [0, 0, 0], names=["x", "y", "z"])
    assert [c.said(n) for n in "xyz"] == [list(range(6))] * 3 and "a" not in c._table
    c.check()
    c.reorder(["x", "y", "z"], [2], names=["x"])
    assert c.said("x") == list(range(6)) and c.free_pages == 18
    c.check()
    c.reorder(["x"], [], names=[])
    assert c.free_pages == 20


def test_copies_go_into_pages_that_become_free():
    c = Cache(4)
    for t in range(6):
        c.say("a", t)
    c.fork("a", ["b", "c"])            # one shared page, three last ones: the cache is full
    assert c.free_pages == 0
    c.reorder(["a", "b", "c"], [1, 1, 1])
    assert [c.said(n) for n in "abc"] == [list(range(6))] * 3
    c.check()


def test_refused_reorders_change_nothing():
    c = Cache(4)
    for t in range(6):
        c.say("a", t)
    c.fork("a", ["b"])
    c.extend("other", 2)

    def state():
        return dict(c._table), dict(c._len), list(c._owners), list(c._free)

    was = state()
    for seqs, parents, names in ((["a", "a"], [0, 0], None), (["a", "q"], [0, 1], None), (["a", "b"], [0], None), (["a", "b"], [0, 2], None),
                                 (["a", "b"], [0, -1], None), (["a", "b"], [0, 1], ["x", "x"]), (["a", "b"], [0, 1], ["a", "other"])):
        with pytest.raises(ValueError):
            c.reorder(seqs, parents, names)
        assert state() == was
    with pytest.raises(RuntimeError, match="free pages"):
        c.reorder(["a", "b"], [0, 0, 1], names=["a", "b", "x"])
    assert state() == was
    c.free("other")
    was = state()
    c.fail = True
    with pytest.raises(RuntimeError, match="no launch"):
        c.reorder(["a", "b"], [0, 0])
    with pytest.raises(RuntimeError, match="no launch"):
        c.reorder(["a", "b"], [0, 0, 1], names=["a", "b", "x"])
    got = state()
    assert got[:3] == was[:3] and sorted(got[3]) == sorted(was[3])
