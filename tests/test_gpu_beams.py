"""The selection of beams against plain numpy in 64 bits.

Parents, tokens and histories have to be equal: logits are drawn so that no two
candidates of different beams are nearer than the rows' sums are exact (their
error is some 2^-24 of a log sum of 20 at most; the nearest two totals of a test
are looked at).  Scores are fp32 roundings of totals of up to 64 or so: half a
step of 2^-18, and the sum's error."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import test_activation_aware_amd as ttq  # noqa: E402

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def make(requests, beams, vocab, dtype, seed=0, spread=3.0, stride=0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((requests * beams, vocab + stride), generator=g) * spread).to(TYPES[dtype])
    scores = -torch.rand((requests, beams), generator=g) * 10
    return x, scores


def want(x, scores, keep, history=None):
    """(totals, parents, tokens, histories) by the definition; asserts that no order hangs on an error of 1e-6."""
    x, s = x.double().numpy(), scores.double().numpy()
    requests, beams = s.shape
    vocab = x.shape[1]
    out = []
    for r in range(requests):
        total = np.full((beams, vocab), -np.inf)
        for w in range(beams):
            if not np.isfinite(s[r, w]):
                continue
            row = x[r * beams + w]
            with np.errstate(all="ignore"):
                m = row.max()
                lse = m + np.log(np.exp(row - m).sum())
                total[w] = s[r, w] + (row - lse)
        total = np.where(total > -np.inf, total, -np.inf).reshape(-1)
        order = np.argsort(-total, kind="stable")[:keep + 1]
        best = order[:keep]
        for a, b in zip(order, order[1:]):
            near = np.isfinite(total[b]) and total[a] - total[b] < 1e-6
            # near ones are of one beam, whose order is exact, or of equal rows
            assert not near or a // vocab == b // vocab or np.array_equal(x[r * beams + a // vocab], x[r * beams + b // vocab])
        none = ~np.isfinite(total[best])
        t = np.where(none, -np.inf, total[best])
        p, v = np.where(none, -1, best // vocab), np.where(none, -1, best % vocab)
        miss = keep - len(best)
        t, p, v = (np.concatenate([a, np.full(miss, f)]) for a, f in ((t, -np.inf), (p, -1), (v, -1)))
        h = None
        if history is not None:
            old = history.numpy()[r * beams:(r + 1) * beams]
            h = np.stack([np.append(old[int(a)], b) if a >= 0 else np.full(old.shape[1] + 1, -1) for a, b in zip(p, v)])
        out.append((t, p, v, h))
    return [None if o[0] is None else np.stack(o) for o in zip(*out)]


def check(x, scores, keep, history=None, got=None, columns=None):
    columns = x.shape[1] if columns is None else columns
    if got is None:
        got = ttq.ttq_beam_select(x.cuda()[:, :columns], scores.cuda(), keep, None if history is None else history.cuda())
    t, p, v, h = want(x[:, :columns], scores, keep, history)
    assert np.array_equal(got[1].cpu().numpy(), p)
    assert np.array_equal(got[2].cpu().numpy(), v)
    gt = got[0].double().cpu().numpy()
    assert np.array_equal(np.isfinite(gt), np.isfinite(t))
    live = np.isfinite(t)
    assert (np.abs(gt[live] - t[live]) <= 2.0 ** -24 * np.abs(t[live]) + 2e-6).all()
    if history is not None:
        assert np.array_equal(got[3].cpu().numpy(), h.reshape(-1, history.shape[1] + 1))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("requests,beams,vocab,keep", [
    (1, 1, 1, 1), (1, 1, 5, 8), (3, 2, 31, 4), (2, 4, 33, 64), (1, 64, 100, 64), (7, 3, 500, 6), (40, 8, 1000, 16),
    (1, 4, 50257, 8), (2, 5, 50257, 10), (1, 1, 151936, 64), (3, 8, 151936, 16), (1, 64, 131072, 64), (300, 4, 2000, 8),
])
def test_sizes(requests, beams, vocab, keep, dtype):
    x, scores = make(requests, beams, vocab, dtype)
    check(x, scores, keep)


def test_many_lists():
    """64 beams whose rows are five chunks each: the most candidates that a request joins in LDS."""
    x, scores = make(1, 64, 1100000, "f32")
    check(x, scores * 0.1, 64)


@pytest.mark.parametrize("length", [0, 1, 7, 100, 5000])
def test_histories(length):
    x, scores = make(3, 4, 700, "f16")
    g = torch.Generator().manual_seed(1)
    check(x, scores, 8, torch.randint(0, 1 << 40, (12, length), generator=g))


def test_strides():
    x, scores = make(3, 4, 1001, "bf16", stride=7)
    history = torch.arange(12 * 20).reshape(12, 20)
    d = history.cuda()
    got = ttq.ttq_beam_select(x.cuda()[:, :1001], scores.cuda(), 5, d[:, 3:9])
    check(x, scores, 5, history[:, 3:9], got, columns=1001)


@pytest.mark.parametrize("vocab", [300, 120000])
def test_empty_beams_and_forbidden_tokens(vocab):
    x, scores = make(4, 4, vocab, "f32")
    scores[0, 1:] = -float("inf")            # a first step
    scores[1] = -float("inf")                # a request that has ended
    scores[2, 0], scores[2, 3] = float("nan"), float("inf")
    x[:, 7:] = torch.where(torch.arange(7, vocab) % 3 == 0, x[:, 7:], torch.tensor(-float("inf")))
    x[12] = -float("inf")                    # a beam with nothing allowed
    x[13, 5:] = -float("inf")
    x[1] = float("nan")                      # of an empty beam: not read
    history = torch.arange(16 * 3).reshape(16, 3)
    check(x, scores, 12, history)


def test_fewer_candidates_than_kept():
    x, scores = make(2, 2, 50, "f16")
    x[:, 3:] = -float("inf")
    x[2, 1:] = -float("inf")
    check(x, scores, 8, torch.arange(12).reshape(4, 3))


def test_rows_that_are_no_distribution():
    """NaN or +inf among the logits: the row's sum is no number, and it has no candidates."""
    x, scores = make(3, 3, 400, "bf16")
    x[0, 17] = float("nan")
    x[4, 399] = float("inf")
    x[6] = float("nan")
    x[7] = float("inf")
    x[8, 0] = -float("inf")
    check(x, scores, 9)


@pytest.mark.parametrize("vocab", [257, 100000])
def test_equal_logits_and_equal_beams(vocab):
    """Of equal totals the earlier beam, then the lower token."""
    x = torch.zeros((6, vocab), dtype=torch.float16)
    x[:, vocab // 2:] = 1.0
    scores = torch.zeros((2, 3))
    scores[1, 2] = 1.0
    check(x, scores, 64)
    x, scores = make(1, 1, vocab, "bf16", spread=0.5)  # many equal ones in a row
    check(x, scores, 64)
    check(x.repeat(4, 1), scores.repeat(1, 4), 64)


def test_large_and_far_logits():
    x, scores = make(2, 4, 600, "f32")
    x[0] *= 1e30
    x[1] += 3e6
    x[2, 5] = 3e38
    x[3, :] = -3e38
    x[3, 9] = -2.9e38
    x, scores = x[:4], scores[:1]
    scores[0] = torch.tensor([-1.0, -2.5, -3.0, -4.0])
    got = ttq.ttq_beam_select(x.cuda(), scores.cuda(), 4)
    # each beam's best token has probability 1, or nearly
    assert got[1].tolist()[0][0] == 0 and got[2].tolist()[0][0] == int(x[0].argmax())
    assert sorted(got[1].tolist()[0]) in ([0, 1, 2, 3], [0, 2, 3, 3], [0, 1, 2, 2], [0, 0, 2, 3], [0, 2, 3, 1], [0, 1, 1, 2])
    assert [t for p, t in zip(got[1].tolist()[0], got[2].tolist()[0]) if p == 2][:1] == [5]


def test_keys_beyond_what_lds_holds():
    """A vocabulary of several chunks for many beams: the lists stay in memory."""
    vocab = 1200000
    x, scores = make(1, 64, vocab, "f32", spread=2.0)
    got = ttq.ttq_beam_select(x.cuda(), scores.cuda(), 64)
    total = torch.log_softmax(x.cuda().double(), 1) + scores.cuda().double()[0, :, None]
    value, at = total.flatten().topk(65)
    gap = value[:-1] - value[1:]
    assert bool(((gap > 1e-6) | (at[:-1] // vocab == at[1:] // vocab)).all())
    assert torch.equal(got[1][0], at[:64] // vocab) and torch.equal(got[2][0], at[:64] % vocab)


def test_streams_graphs_and_workspaces():
    x, scores = make(2, 4, 100003, "bf16")
    history = torch.arange(8 * 40).reshape(8, 40)
    d = x.cuda(), scores.cuda(), history.cuda()
    need = ttq.load().ttq_beam_select_workspace_bytes(2, 4, 100003, 8)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    first = ttq.ttq_beam_select(d[0], d[1], 8, d[2], workspace=ws)
    check(x, scores, 8, history, first)
    with pytest.raises(ttq.TTQError):
        ttq.ttq_beam_select(d[0], d[1], 8, d[2], workspace=ws[:need - 1])
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        got = ttq.ttq_beam_select(d[0], d[1], 8, d[2])
    stream.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, first))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ttq.ttq_beam_select(d[0], d[1], 8, d[2], workspace=ws)
    for i in range(3):
        for t in got:
            t.fill_(3)
        ws.fill_(i)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, first))


def test_refused_tensors():
    x, scores = (t.cuda() for t in make(2, 3, 40, "f16"))
    ttq.ttq_beam_select(x, scores, 4)
    history = torch.zeros((6, 4), dtype=torch.int64, device="cuda")
    for bad, kind in ((dict(logits=x.double()), TypeError), (dict(logits=x.T), ValueError), (dict(logits=x[:5]), ValueError),
                      (dict(scores=scores.double()), TypeError), (dict(scores=scores.T), ValueError), (dict(scores=scores.cpu()), ValueError),
                      (dict(keep=0), ValueError), (dict(keep=65), ValueError), (dict(history=history.int()), TypeError),
                      (dict(history=history[:5]), ValueError), (dict(history=history.T), ValueError),
                      (dict(logits=torch.zeros((130, 9), device="cuda"), scores=torch.zeros((2, 65), device="cuda")), ttq.TTQError)):
        a = dict(logits=x, scores=scores, keep=4)
        a.update(bad)
        with pytest.raises(kind):
            ttq.ttq_beam_select(**a)
    assert ttq.ttq_beam_select(x[:0], scores[:0], 4)[0].shape == (0, 4)


@pytest.mark.parametrize("bits", [16, 4])
def test_reordered_pages(bits):
    """PagedCache.reorder: what each beam's pages hold follows its parent; copies are the beams' own."""
    cache = ttq.PagedCache(2, 60, 2, 64, page_size=16, bits=bits)
    g = torch.Generator().manual_seed(0)
    names = ["a", "b", "c", "d"]
    cache.extend("a", 20)
    b = cache.batch(["a"], [20])
    for layer in range(2):
        cache.write(layer, *(torch.randn((20, 128), generator=g).half().cuda() for _ in range(2)), b)
    cache.fork("a", names[1:])

    def row(token):
        return torch.full((1, 128), float(token)).half().cuda()

    said = {n: [] for n in names}
    for step, parents in enumerate(([0, 0, 1, 2], [3, 3, 3, 3], [0, 1, 2, 3], [1, 0, 0, 2], [2, 2, 0, 0]) * 4):
        cache.reorder(names, parents)
        said = {n: list(said[names[p]]) for n, p in zip(names, parents)}
        for i, n in enumerate(names):
            cache.extend(n, 1)
            said[n].append(100 * step + 10 * i)
        b = cache.batch(names, [1] * 4)
        rows = torch.cat([row(said[n][-1]) for n in names])
        for layer in range(2):
            cache.write(layer, rows, -rows, b)
        used = sum(o > 0 for o in cache._owners)
        assert used + cache.free_pages == 60
    for n in names:
        pages = cache.pages_of(n)
        for at, token in enumerate(said[n]):
            p = 20 + at
            if bits == 16:
                assert float(cache.k[1, pages[p // 16], 1, p % 16, 5]) == token
                assert float(cache.v[0, pages[p // 16], 0, p % 16, 9]) == -token
        if bits == 4:
            b = cache.batch([n], [len(said[n])])
            k, v = ttq.ttq_packed_read(cache.k[1], cache.v[1], b["block_table"], b["q_start"], b["kv_len"], len(said[n]))
            assert k[:, 70].tolist() == said[n] and v[:, 3].tolist() == [-t for t in said[n]]
