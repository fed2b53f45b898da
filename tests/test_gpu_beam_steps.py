"""Selections whose every parent and token is settled by the definition, and steps of several requests with their pages."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import test_activation_aware_amd as ttq  # noqa: E402
from test_gpu_beams import check, make, want  # noqa: E402

pytestmark = pytest.mark.gpu


def test_large_and_far_logits():
    """Offsets of 3e6, where logits lie a quarter apart and two are alike, and rows near the ends of 32 bits."""
    x, scores = make(1, 4, 600, "f32")
    x[0] *= 1e30
    x[1] += 3e6
    x[2, 5] = 3e38
    x[3, :] = -3e38
    x[3, 9] = -2.9e38
    scores[0] = torch.tensor([-1.0, -2.5, -3.0, -4.0])
    total, parents, tokens, _ = want(x, scores, 5)
    assert parents[0].tolist() == [0, 2, 1, 1, 3] and tokens[0, 2] < tokens[0, 3]
    assert tokens[0, [0, 1, 4]].tolist() == [int(x[0].argmax()), 5, 9]
    assert np.allclose(total[0], [-1, -3, -3.9906, -3.9906, -4], atol=1e-4)
    for keep in (1, 2, 3, 4, 5):
        check(x, scores, keep)


@pytest.mark.parametrize("bits", [16, 4])
def test_steps_of_requests(bits):
    """Two requests, one of which runs out of allowed tokens: the selection's parents go to reorder as they are."""
    cache = ttq.PagedCache(1, 40, 2, 64, page_size=16, bits=bits)
    names = [(r, w) for r in range(2) for w in range(3)]
    for r in range(2):
        cache.extend((r, 0), 10)
        cache.write(0, *(torch.full((10, 128), float(r), device="cuda").half() for _ in range(2)), cache.batch([(r, 0)], [10]))
        cache.fork((r, 0), [(r, 1), (r, 2)])
    g = torch.Generator().manual_seed(0)
    scores, history = torch.zeros((2, 3), device="cuda"), torch.empty((6, 0), dtype=torch.int64, device="cuda")
    scores[:, 1:] = -float("inf")
    for step in range(12):
        x = torch.randn((6, 50), generator=g)
        if step == 4:
            x[3:, 1:] = -float("inf")   # one token is allowed: as many candidates as beams, of which two are gone
            scores[1, 1:] = -float("inf")
        if step == 8:
            x[3:] = -float("inf")
        scores, parents, tokens, history = ttq.ttq_beam_select(x.cuda(), scores, 3, history)
        cache.reorder(names, parents)
        alive = [n for n, t in zip(names, tokens.flatten().tolist()) if t >= 0]
        assert [n in cache._table for n in names] == [n in alive for n in names]
        assert len(alive) == (6 if step < 4 else 4 if step == 4 else 6 if step < 8 else 3)
        for n in alive:
            cache.extend(n, 1)
        rows = torch.stack([torch.full((128,), float(history[3 * r + w, -1])) for r, w in alive]).half().cuda()
        cache.write(0, rows, -rows, cache.batch(alive, [1] * len(alive)))
    for r, w in alive:
        pages = cache.pages_of((r, w))
        b = cache.batch([(r, w)], [22])
        if bits == 16:
            held = torch.stack([cache.k[0, pages[p // 16], 1, p % 16, 5] for p in range(22)])
        else:
            held = ttq.ttq_packed_read(cache.k[0], cache.v[0], b["block_table"], b["q_start"], b["kv_len"], 22)[0][:, 70]
        assert held.tolist() == [float(r)] * 10 + history[3 * r + w].double().tolist()
    used = sum(o > 0 for o in cache._owners)
    assert used + cache.free_pages == 40
