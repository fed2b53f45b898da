"""The serving operators on the GPU against plain statements of them in 64
bits on the CPU.

Tolerances, from the number formats.  Attention: a probability is rounded to
the operand type (unit roundoff u, half a unit of the last of 11 or 8 bits: 2^-11 fp16, 2^-8 bf16), the output once
more, so an output is off by at most 2 u A with A = sum_j p_j |v_j| >= |o|;
fp16 probabilities (relative to the largest, 1) also lose what lies below
2^-25, kv_len of them at most, over their sum l; the scores are fp32 sums of
exact products, their error times A stays below 2e-4 A at these sizes.  The
log sum: 1e-4 absolute (fp32 exponentials and sums of up to 4096 terms per
lane).  Log probabilities: fp32 sums of V / 256 terms per thread and chunk."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import test_activation_aware_amd as ttq  # noqa: E402

pytestmark = pytest.mark.gpu

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    ttq.load()
    yield
    torch.cuda.synchronize()


def say(*a):
    print(*a, flush=True)


class Batch:
    """A cache with pages in random order and a ragged batch over it; what no
    position occupies holds NaN."""

    def __init__(self, lens, kv_heads, dim, page, dtype, seed=0, interleaved=False, pages_apart=1):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.kvh, self.dim, self.page, self.dtype = lens, kv_heads, dim, page, dtype
        need = [-(-k // page) for _, k in lens]
        self.pages = max(1, sum(need) * pages_apart + 2)
        order = torch.randperm(self.pages, generator=g)[:sum(need)].to(torch.int32)
        blocks = max(need + [1]) + 1
        self.table = torch.full((len(lens), blocks), -1, dtype=torch.int32)
        at = 0
        shape = (self.pages, kv_heads, page, dim)
        if interleaved:
            both = torch.full((self.pages, 2) + shape[1:], float("nan"), dtype=dtype, device="cuda")
            self.k, self.v = both[:, 0], both[:, 1]
        else:
            self.k = torch.full(shape, float("nan"), dtype=dtype, device="cuda")
            self.v = torch.full(shape, float("nan"), dtype=dtype, device="cuda")
        self.K, self.V = [], []  # per sequence [kv][heads][dim], double
        for s, n in enumerate(need):
            self.table[s, :n] = order[at:at + n]
            at += n
            kv = lens[s][1]
            x = [(torch.randn((kv, kv_heads, dim), generator=g)).to(dtype) for _ in range(2)]
            self.K.append(x[0].double())
            self.V.append(x[1].double())
            for c, t in zip((self.k, self.v), x):
                for b in range(n):
                    part = t[b * page:(b + 1) * page]
                    c[int(self.table[s, b]), :, :part.shape[0]] = part.transpose(0, 1).cuda()
        starts = np.concatenate([[0], np.cumsum([q for q, _ in lens])]).astype(np.int32)
        self.total = int(starts[-1])
        self.q_start = torch.from_numpy(starts).cuda()
        self.kv_len = torch.tensor([k for _, k in lens], dtype=torch.int32).cuda()
        self.dtable = self.table.cuda()
        self.gen = g


def attention_ref(b, q, heads, scale, softcap=0.0, window=0, slopes=None, prefix=None):
    """(o, lse, A, l) in double: outputs, log sums, sum p|v|, sum of exp(z - max)."""
    group, d = heads // b.kvh, b.dim
    o = torch.zeros((b.total, heads, d), dtype=torch.float64)
    lse = torch.full((b.total, heads), -math.inf, dtype=torch.float64)
    A, l = torch.zeros_like(o), torch.ones((b.total, heads), dtype=torch.float64)
    at = 0
    for s, (ql, kl) in enumerate(b.lens):
        i = torch.arange(kl - ql, kl)[:, None]
        j = torch.arange(kl)[None, :]
        seen = j <= i
        if window:
            seen = seen & (i - j < window)
        if prefix is not None:
            seen = seen | (j < prefix[s])
        for h in range(heads):
            x = q[at:at + ql, h * d:(h + 1) * d].double()
            z = x @ b.K[s][:, h // group].T * scale
            if softcap:
                z = softcap * torch.tanh(z / softcap)
            if slopes is not None:
                z = z - float(slopes[h]) * (i - j).abs()
            z = z.masked_fill(~seen, -math.inf)
            some = seen.any(1)
            if not bool(some.any()):
                continue
            m = z[some].amax(1, keepdim=True)
            e = (z[some] - m).exp()
            t = e.sum(1, keepdim=True)
            V = b.V[s][:, h // group]
            rows = torch.arange(at, at + ql)[some]
            o[rows, h], A[rows, h] = e @ V / t, e @ V.abs() / t
            lse[rows, h], l[rows, h] = (m + t.log())[:, 0], t[:, 0]
        at += ql
    return o, lse, A, l


def check_attention(lens, heads, kv_heads, dim, page, dtype, seed=0, softcap=0.0, window=0, slopes=False, prefix=None,
                    strided=False, interleaved=False, bounds=None):
    b = Batch(lens, kv_heads, dim, page, dtype, seed, interleaved)
    q = torch.randn((b.total, heads * dim), generator=b.gen).mul(1.5).to(dtype)
    sl = torch.tensor([2.0 ** (-8.0 * (h + 1) / heads) for h in range(heads)]) if slopes else None
    pf = None if prefix is None else torch.tensor(prefix, dtype=torch.int32)
    dq = q.cuda()
    out = None
    if strided:  # a slice of a fused projection, rows of a wider output
        wide = torch.full((b.total, heads * dim + 64), float("nan"), dtype=dtype, device="cuda")
        wide[:, 32:32 + heads * dim] = dq
        dq = wide[:, 32:32 + heads * dim]
        out = torch.full((b.total, heads * dim + 8), 7.0, dtype=dtype, device="cuda")[:, :heads * dim]
    lse = torch.full((b.total, heads), 7.0, device="cuda")
    mq, mk = bounds or (max(x for x, _ in lens), max(x for _, x in lens))
    say(f"attention lens={lens if len(lens) < 9 else len(lens)} {heads}/{kv_heads}x{dim} page {page} {dtype} "
        f"cap={softcap} window={window} slopes={slopes} prefix={prefix}")
    how = dict(softcap=softcap, window=window, slopes=None if sl is None else sl.cuda(),
               prefix_len=None if pf is None else pf.cuda())
    got = ttq.ttq_paged_attention(dq, b.k, b.v, b.dtable, b.q_start, b.kv_len, mq, mk, out=out, lse=lse, **how)
    again = ttq.ttq_paged_attention(dq, b.k, b.v, b.dtable, b.q_start, b.kv_len, mq, mk, **how)
    assert torch.equal(got, again), "two calls differ"
    if strided:
        assert bool((out._base[:, heads * dim:] == 7.0).all()), "wrote past its columns"
    o, L, A, l = attention_ref(b, q, heads, dim ** -0.5, softcap, window, sl, prefix)
    got = got.cpu().double().reshape(b.total, heads, dim)
    assert bool(torch.isfinite(got).all())
    kv = torch.tensor([k for ql, k in lens for _ in range(ql)]).double()[:, None, None]
    vmax = max([float(v.abs().max()) for v in b.V if v.numel()] + [0.0])
    tol = (2 * U[dtype] + 2e-4) * A + kv * 2.0 ** -25 * vmax / l[..., None] + 1e-7
    worst = float(((got - o).abs() / tol).max()) if b.total else 0.0
    none = torch.isinf(L)
    assert bool((got[none] == 0).all())
    gl = lse.cpu().double()
    assert bool((gl[none] == -math.inf).all())
    dl = float((gl - L)[~none].abs().max()) if bool((~none).any()) else 0.0
    say(f"  worst error {worst:.3f} of its bound, log sums off by {dl:.2e}")
    assert worst <= 1.0 and dl <= 1e-4


F16, BF16 = torch.float16, torch.bfloat16


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("dim,heads,kv_heads,page", [(64, 12, 12, 16), (128, 16, 2, 64), (256, 6, 3, 32),
                                                     (128, 5, 1, 256), (64, 48, 1, 128)])
def test_attention_decode(dim, heads, kv_heads, page, dtype):
    """One token each: lengths around the tile and page edges, one of them a single key."""
    check_attention([(1, n) for n in (1, 2, 15, 16, 17, 63, 64, 65, 127, 300, 1025)], heads, kv_heads, dim, page, dtype)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("dim,heads,kv_heads,page", [(64, 4, 4, 16), (128, 8, 2, 32), (256, 2, 1, 64),
                                                     (128, 3, 1, 128), (64, 32, 2, 64)])
def test_attention_chunks(dim, heads, kv_heads, page, dtype):
    """Chunks of odd lengths over odd contexts, whole prompts, and decode tokens among them."""
    check_attention([(5, 5), (1, 77), (129, 129), (64, 200), (31, 333), (1, 1), (2, 64), (257, 300)], heads, kv_heads,
                    dim, page, dtype)


@pytest.mark.parametrize("mods", [dict(softcap=20.0), dict(slopes=True), dict(window=1), dict(window=70),
                                  dict(window=64, softcap=30.0, slopes=True), dict(prefix=[3, 64, 0, 150, 129]),
                                  dict(prefix=[5, 1, 40, 299, 10], window=33),
                                  dict(prefix=[2, 77, 100, 0, 65], window=40, slopes=True, softcap=50.0)])
@pytest.mark.parametrize("dim,dtype", [(128, F16), (64, BF16), (256, F16)])
def test_attention_scores_and_masks(mods, dim, dtype):
    lens = [(5, 5), (1, 77), (100, 129), (40, 300), (130, 130)]
    check_attention(lens, 4, 2, dim, 32, dtype, **mods)


@pytest.mark.parametrize("lens", [[(3, 0), (2, 5), (0, 0), (0, 40), (1, 1)],      # no keys; no tokens
                                  [(9, 4), (70, 3), (1, 130)],                    # tokens before position 0
                                  [(0, 0)] * 70 + [(1, 33)] + [(0, 10)] * 5 + [(2, 20)] * 66])  # many sequences
@pytest.mark.parametrize("dim", [64, 128])
def test_attention_empty_rows(lens, dim):
    check_attention(lens, 4, 2, dim, 16, F16)


def test_attention_window_and_prefix_leave_a_gap():
    """A long context of which only the prefix and the last window are seen."""
    check_attention([(1, 3000), (40, 2500), (300, 1500)], 8, 2, 128, 64, F16, window=100, prefix=[70, 10, 200])
    check_attention([(1, 3000)], 8, 8, 64, 16, BF16, window=1, prefix=[1])


def test_attention_split_along_the_keys():
    check_attention([(1, 20000)], 8, 1, 128, 64, F16)
    check_attention([(1, 9000), (1, 3), (1, 0), (3, 5000)], 4, 2, 256, 128, BF16)
    check_attention([(40, 7000)], 4, 4, 64, 16, F16, softcap=30.0)


def test_attention_strides_and_bounds():
    check_attention([(20, 100), (1, 300)], 4, 2, 128, 16, F16, strided=True)
    check_attention([(20, 100), (1, 300)], 4, 2, 64, 64, BF16, interleaved=True)
    # max lengths are bounds: larger ones change nothing but the split
    check_attention([(20, 100), (1, 300)], 4, 2, 128, 16, F16, bounds=(64, 8192))
    check_attention([(3, 700)], 4, 2, 128, 16, F16, bounds=(3, 100000))


def test_attention_large_scores():
    """Scores of several hundred: the running maximum has to follow."""
    b = Batch([(40, 300)], 2, 64, 16, F16, seed=5)
    q = torch.randn((40, 4 * 64), generator=b.gen).mul(40).to(F16)
    got = ttq.ttq_paged_attention(q.cuda(), b.k, b.v, b.dtable, b.q_start, b.kv_len, 40, 300).cpu().double()
    o, _, A, l = attention_ref(b, q, 4, 0.125)
    # a score of 300 is off by up to 64 * 2^-24 * sum |q k| ~ 2e-3 relative to the others
    assert float(((got.reshape(o.shape) - o).abs() - (2 * U[F16] + 5e-3) * A - 1e-4).max()) <= 0


def test_attention_masked_keys_hold_anything():
    """Keys past a query's own position, or outside its window: NaN and inf in K do not reach it."""
    b = Batch([(64, 64)], 2, 128, 16, F16)
    q = torch.randn((64, 4 * 128), generator=b.gen).to(F16).cuda()
    clean = ttq.ttq_paged_attention(q, b.k, b.v, b.dtable, b.q_start, b.kv_len, 64, 64)
    for pos, bad in ((63, float("nan")), (62, float("inf"))):
        b.k[int(b.table[0, pos // 16]), :, pos % 16] = bad
    got = ttq.ttq_paged_attention(q, b.k, b.v, b.dtable, b.q_start, b.kv_len, 64, 64)
    assert torch.equal(got[:62], clean[:62])


@pytest.mark.parametrize("dim,heads,kv_heads,dtype", [(64, 4, 2, BF16), (128, 4, 2, F16), (128, 6, 1, BF16),
                                                      (256, 2, 1, F16)])
@pytest.mark.parametrize("lens,how", [([(300, 300)], {}), ([(200, 333), (1, 40)], dict(window=40)),
                                      ([(1, 300), (1, 77)], dict(window=30)), ([(3, 5000)], {}),
                                      ([(150, 200), (9, 100)], dict(prefix=[170, 95])),
                                      ([(1100, 1100)], dict(window=500, prefix=[70]))])
def test_attention_masked_values_hold_anything(lens, how, dim, heads, kv_heads, dtype):
    """NaN and inf in V: the outputs of a query that does not see them keep their bits, also in the elements
    next to them; one that does see them gets what the sum over its keys gives."""
    page = 16
    b = Batch(lens, kv_heads, dim, page, dtype, seed=2)
    q = torch.randn((b.total, heads * dim), generator=b.gen).mul(0.5).to(dtype).cuda()
    how = dict(how)
    prefix = how.pop("prefix", None)
    pf = None if prefix is None else torch.tensor(prefix, dtype=torch.int32).cuda()
    mq, mk = max(x for x, _ in lens), max(x for _, x in lens)
    say(f"masked values lens={lens} {heads}/{kv_heads}x{dim} {dtype} {how} prefix={prefix}")

    def run():
        return ttq.ttq_paged_attention(q, b.k, b.v, b.dtable, b.q_start, b.kv_len, mq, mk, prefix_len=pf,
                                       **how).cpu().reshape(b.total, heads, dim)

    clean = run()
    want = clean.double()
    at, group = 0, heads // kv_heads
    for s, (ql, kl) in enumerate(lens):
        i = torch.arange(kl - ql, kl)
        for n, bad in enumerate((math.inf, math.nan, -math.inf, math.inf, -math.inf)):
            pos = kl - 1 - (0, 1, 17, 35, 64)[n]  # around the last rows' diagonal and the window's edge
            if pos < 0:
                continue
            h, d = n % kv_heads, (0, 37, 37, dim - 1, 6)[n]
            b.v[int(b.table[s, pos // page]), h, pos % page, d] = bad
            seen = pos <= i
            if how.get("window"):
                seen = seen & (i - pos < how["window"])
            if prefix is not None:
                seen = seen | (pos < prefix[s])
            rows = at + torch.nonzero(seen)[:, 0]
            want[rows, h * group:(h + 1) * group, d] += bad
        at += ql
    got = run()
    assert torch.equal(run().view(torch.int16), got.view(torch.int16))
    same = torch.isfinite(want)
    assert torch.equal(got[same].view(torch.int16), clean[same].view(torch.int16))
    assert bool((torch.isnan(got) == torch.isnan(want)).all())
    assert bool((torch.isposinf(got) == torch.isposinf(want)).all())
    assert bool((torch.isneginf(got) == torch.isneginf(want)).all())


def test_attention_pages_past_4_gib():
    """Page offsets beyond 32 bits, for the write and the read."""
    page, kvh, dim = 256, 8, 128
    n = (5 << 30) // (page * kvh * dim * 2)
    k = torch.empty((n, kvh, page, dim), dtype=F16, device="cuda")
    v = torch.empty((n, kvh, page, dim), dtype=F16, device="cuda")
    lens = [(300, 300), (1, 1)]
    b = Batch(lens, kvh, dim, page, F16)
    table = torch.tensor([[n - 1, n - 3], [n - 2, 0]], dtype=torch.int32).cuda()
    kk = torch.cat([x for x in b.K]).reshape(301, -1).to(F16).cuda()
    vv = torch.cat([x for x in b.V]).reshape(301, -1).to(F16).cuda()
    ttq.ttq_cache_write(kk, vv, k, v, table, b.q_start, b.kv_len)
    q = torch.randn((301, 8 * 128), generator=b.gen).to(F16).cuda()
    got = ttq.ttq_paged_attention(q, k, v, table, b.q_start, b.kv_len, 300, 300)
    want = ttq.ttq_paged_attention(q, b.k, b.v, b.dtable, b.q_start, b.kv_len, 300, 300)
    assert torch.equal(got, want)


def test_attention_bad_pages_are_not_followed():
    """Page numbers outside the cache and lengths past the table: no fault, other sequences untouched."""
    b = Batch([(1, 100), (1, 50)], 2, 64, 16, F16)
    q = torch.randn((2, 4 * 64), generator=b.gen).to(F16).cuda()
    want = ttq.ttq_paged_attention(q, b.k, b.v, b.dtable, b.q_start, b.kv_len, 1, 100)
    t = b.dtable.clone()
    t[0, 1], t[0, 2] = 1 << 30, -7
    kv = b.kv_len.clone()
    kv[0] = 1 << 30
    got = ttq.ttq_paged_attention(q, b.k, b.v, t, b.q_start, kv, 1, 100)
    assert torch.equal(got[1], want[1])


def test_operators_on_another_stream():
    b = Batch([(40, 100), (1, 300)], 2, 128, 16, F16)
    q = torch.randn((41, 4 * 128), generator=b.gen).to(F16).cuda()
    x = torch.randn((5, 1000), device="cuda")
    tok = torch.arange(5, device="cuda")
    want = ttq.ttq_paged_attention(q, b.k, b.v, b.dtable, b.q_start, b.kv_len, 40, 300)
    lp = ttq.ttq_token_logprobs(x, tok, top=3)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = ttq.ttq_paged_attention(q, b.k, b.v, b.dtable, b.q_start, b.kv_len, 40, 300)
        lp2 = ttq.ttq_token_logprobs(x, tok, top=3)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and all(torch.equal(a, c) for a, c in zip(lp, lp2))


@pytest.mark.parametrize("lens", [[(1, 300), (1, 2500), (1, 1)], [(40, 100), (1, 300), (200, 260)]])
def test_operators_in_a_graph(lens):
    """A step captured once and replayed with other contents in the same buffers, the program's own work in between."""
    heads, kvh, dim, V = 8, 2, 128, 5000
    b = Batch(lens, kvh, dim, 16, F16)
    mq, mk = max(x for x, _ in lens), max(x for _, x in lens)
    k, v = torch.zeros_like(b.k), torch.zeros_like(b.v)
    new = torch.zeros((b.total, 2 * kvh * dim), dtype=F16, device="cuda")
    q = torch.zeros((b.total, heads * dim), dtype=F16, device="cuda")
    x = torch.zeros((b.total, V), device="cuda")
    tok = torch.zeros(b.total, dtype=torch.int64, device="cuda")
    src = torch.tensor([int(b.table[0, 0])], dtype=torch.int32).cuda()
    spare = [p for p in range(b.pages) if p not in b.table.flatten().tolist()]
    dst = torch.tensor(spare[:1], dtype=torch.int32).cuda()

    def step():
        ttq.ttq_cache_write(new[:, :kvh * dim], new[:, kvh * dim:], k, v, b.dtable, b.q_start, b.kv_len)
        ttq.ttq_cache_copy_pages(k, v, src, dst)
        o = ttq.ttq_paged_attention(q, k, v, b.dtable, b.q_start, b.kv_len, mq, mk)
        return (o, k, v) + tuple(ttq.ttq_token_logprobs(x, tok, top=4))

    def fill(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        for t in (k, v, new, q, x):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        tok.copy_(torch.randint(0, V, tok.shape, generator=g, device="cuda"))

    fill(0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in range(1, 5):
        fill(seed)
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        fill(seed)
        graph.replay()
        got = [t.clone() for t in held]
        torch.cuda.synchronize()
        say(f"replay {seed} of lens={lens}")
        for a, c in zip(got, want):
            assert torch.equal(a, c)


# -- the cache -------------------------------------------------------------
@pytest.mark.parametrize("dim,kv_heads,page,dtype", [(64, 12, 16, F16), (128, 8, 64, BF16), (256, 1, 256, F16),
                                                     (128, 3, 32, F16)])
def test_cache_write(dim, kv_heads, page, dtype):
    lens = [(1, 40), (17, 17), (0, 9), (3, 2), (100, 500), (1, 16), (1, 17)]   # (3, 2): its first row has no place
    b = Batch(lens, kv_heads, dim, page, dtype)
    wide = torch.randn((b.total, 2 * kv_heads * dim), generator=b.gen).to(dtype)
    k, v = b.k.clone(), b.v.clone()
    wk, wv = k.clone(), v.clone()
    at = 0
    for s, (ql, kl) in enumerate(lens):
        for i in range(ql):
            p = kl - ql + i
            if p >= 0:
                page_id = int(b.table[s, p // page])
                wk[page_id, :, p % page] = wide[at + i, :kv_heads * dim].reshape(kv_heads, dim).cuda()
                wv[page_id, :, p % page] = wide[at + i, kv_heads * dim:].reshape(kv_heads, dim).cuda()
        at += ql
    dw = wide.cuda()
    ttq.ttq_cache_write(dw[:, :kv_heads * dim], dw[:, kv_heads * dim:], k, v, b.dtable, b.q_start, b.kv_len)
    assert torch.equal(k.view(torch.int16), wk.view(torch.int16))
    assert torch.equal(v.view(torch.int16), wv.view(torch.int16))


@pytest.mark.parametrize("layers,pages,pairs,kv_heads,page,dim", [(1, 8, 3, 1, 16, 64), (3, 40, 13, 5, 32, 128),
                                                                  (2, 6000, 2900, 1, 16, 64), (2, 9, 4, 8, 256, 128)])
def test_copy_pages(layers, pages, pairs, kv_heads, page, dim):
    g = torch.Generator().manual_seed(3)
    shape = (layers, pages, kv_heads, page, dim)
    k = torch.randint(-30000, 30000, shape, dtype=torch.int16, device="cuda").view(torch.float16)
    v = torch.randint(-30000, 30000, shape, dtype=torch.int16, device="cuda").view(torch.float16)
    order = torch.randperm(pages, generator=g).to(torch.int32)
    src, dst = order[:pairs].clone(), order[pairs:2 * pairs].clone()
    table = torch.randint(-1, pages, (37, 301), generator=g).to(torch.int32)
    wk, wv, wt = k.clone(), v.clone(), table.clone()
    wk[:, dst.long()], wv[:, dst.long()] = k[:, src.long()], v[:, src.long()]
    to = {int(a): int(c) for a, c in zip(src, dst)}
    wt = torch.tensor([[to.get(int(x), int(x)) for x in r] for r in table], dtype=torch.int32)
    wide = torch.full((37, 310), -5, dtype=torch.int32, device="cuda")
    wide[:, :301] = table.cuda()
    ttq.ttq_cache_copy_pages(k, v, src.cuda(), dst.cuda(), table=wide[:, :301])
    assert torch.equal(k.view(torch.int16), wk.view(torch.int16)) and torch.equal(v.view(torch.int16), wv.view(torch.int16))
    assert torch.equal(wide[:, :301].cpu(), wt) and bool((wide[:, 301:] == -5).all())


def test_copy_pages_skips_and_shared_sources():
    """One page to several; pairs outside the cache; of equal sources the first decides the table."""
    k = torch.randn((6, 2, 16, 64), device="cuda").half()
    v = torch.randn((6, 2, 16, 64), device="cuda").half()
    wk, wv = k.clone(), v.clone()
    src = torch.tensor([1, 1, 6, 2, -1], dtype=torch.int32).cuda()
    dst = torch.tensor([3, 4, 5, 6, 0], dtype=torch.int32).cuda()
    for d in (3, 4):
        wk[d], wv[d] = k[1], v[1]
    table = torch.tensor([[0, 1, 2, -1, 1, 6]], dtype=torch.int32).cuda()
    ttq.ttq_cache_copy_pages(k, v, src, dst, table=table)
    assert torch.equal(k, wk) and torch.equal(v, wv)
    assert table.tolist() == [[0, 3, 2, -1, 3, 6]]


def test_paged_cache_life():
    """Write, fork, decode, free and compact: the sequences' keys stay what was written."""
    cache = ttq.PagedCache(2, 40, 2, 64, page_size=16)
    g = torch.Generator().manual_seed(1)
    kept = {}

    def append(step):
        seqs, new = list(step), [n for n in step.values()]
        for s, n in step.items():
            cache.extend(s, n)
        b = cache.batch(seqs, new)
        rows = torch.randn((sum(new), 2 * 2 * 64), generator=g).half()
        dr = rows.cuda()
        for layer in range(2):
            cache.write(layer, dr[:, :128] + layer, dr[:, 128:] - layer, b)
        at = 0
        for s, n in step.items():
            kept[s] = torch.cat([kept.get(s, rows[:0]), rows[at:at + n]])
            at += n
        return b

    def look():
        for s, rows in kept.items():
            for layer in range(2):
                for c, want in ((cache.k, rows[:, :128].cuda() + layer), (cache.v, rows[:, 128:].cuda() - layer)):
                    got = c[layer, cache.pages_of(s)].transpose(1, 2).reshape(-1, 128)[:cache.length(s)]
                    assert torch.equal(got, want), (s, layer)

    append({"a": 37, "b": 16})
    cache.fork("a", ["c", "d"])
    kept["c"], kept["d"] = kept["a"], kept["a"]
    append({"a": 1, "c": 20, "d": 1, "b": 1})
    look()
    for s in ("a", "b"):
        cache.free(s)
        del kept[s]
    b = cache.batch(["c", "d"], [1, 1])
    q = torch.randn((2, 4 * 64), generator=g).half().cuda()
    before = cache.attend(1, q, b)
    assert cache.compact(table=b["block_table"]) > 0
    look()
    again = cache.batch(["c", "d"], [1, 1])
    assert torch.equal(again["block_table"], b["block_table"])
    assert torch.equal(cache.attend(1, q, again), before)


# -- log probabilities -----------------------------------------------------
def logprobs_ref(x, tokens, top):
    x = x.double().cpu()
    lp = torch.log_softmax(x, 1)
    p = lp.exp()
    ent = torch.where(p > 0, -p * lp, torch.zeros_like(p)).sum(1)
    tok = tokens.cpu()
    ok = (tok >= 0) & (tok < x.shape[1])
    got = torch.where(ok, lp.gather(1, tok.clamp(0, x.shape[1] - 1)[:, None])[:, 0], 0.0)
    ids = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :top]
    return got, ent, ids, lp.gather(1, ids)


def check_logprobs(x, tokens, top):
    T, V = x.shape
    say(f"logprobs T={T} V={V} top={top} {x.dtype}")
    got = ttq.ttq_token_logprobs(x, tokens, top=top)
    again = ttq.ttq_token_logprobs(x, tokens, top=top)
    assert all(torch.equal(a.view(torch.int32), b.view(torch.int32)) for a, b in zip(got, again))
    lp, ent, ids, tlp = logprobs_ref(x, tokens, top)
    tol = (V / 256 + 64) * 2.0 ** -24 + 2.0 ** -20
    near = lambda a, b, t: bool(((a.cpu().double() - b).abs() <= t * (1 + torch.where(torch.isfinite(b), b.abs(), torch.ones_like(b))))[torch.isfinite(b)].all())  # noqa: E731
    assert near(got[0], lp, tol) and near(got[1], ent, 2 * tol)
    same_inf = lambda a, b: torch.equal(torch.isinf(a.cpu()), torch.isinf(b))  # noqa: E731
    assert same_inf(got[0], lp)
    if top:
        assert torch.equal(got[2].cpu(), ids)
        assert near(got[3], tlp, tol) and same_inf(got[3], tlp)


@pytest.mark.parametrize("dtype", [torch.float32, F16, BF16])
@pytest.mark.parametrize("T,V,top", [(1, 1, 1), (3, 5, 5), (2, 31, 7), (4, 33, 20), (7, 500, 64), (1, 4097, 10),
                                     (5, 50257, 20), (2, 151936, 64), (1, 300001, 5), (600, 3001, 3), (2000, 257, 0)])
def test_token_logprobs(T, V, top, dtype):
    g = torch.Generator().manual_seed(T * 1000 + V)
    x = (torch.randn((T, V), generator=g) * 4).to(dtype).cuda()
    tokens = torch.randint(0, V, (T,), generator=g).cuda()
    check_logprobs(x, tokens, top)


def test_token_logprobs_ties():
    """Equal logits everywhere: the lowest indices, in order."""
    g = torch.Generator().manual_seed(9)
    tokens = torch.tensor([5, 100, 60000])
    x = torch.randint(-2, 3, (3, 70001), generator=g).float()
    x[1] = 1.5
    x[2, 1::2] = -0.0
    x[2, ::2] = 0.0
    for dtype in (torch.float32, BF16):
        check_logprobs(x.to(dtype).cuda(), tokens.cuda(), 64)
        check_logprobs(x[:, :1000].to(dtype).cuda().contiguous(), torch.tensor([5, 100, 600]).cuda(), 20)


def test_token_logprobs_large_row_offset_and_masked_vocabulary():
    g = torch.Generator().manual_seed(2)
    x = torch.randn((6, 40000), generator=g)
    x[0] += 5000.0                                  # a common offset
    x[1, 100:] = -math.inf                          # only a hundred tokens are allowed
    x[2, :] = -math.inf
    x[2, 777] = 3.0                                 # a single one
    x[3] = x[3] * 1e-3
    x[4, 39999] = 60.0                              # nearly certain
    x[5, ::2] = -math.inf
    tokens = torch.tensor([1, 50, 777, 5, 39999, 0]).cuda()
    check_logprobs(x.cuda(), tokens, 10)
    x[0] = 0
    check_logprobs(x.to(BF16).cuda(), tokens, 64)


def test_token_logprobs_special_rows():
    x = torch.randn((5, 9000), device="cuda")
    x[0] = -math.inf
    x[1, 17] = math.nan
    x[2] = math.nan
    x[3, 4000] = math.inf
    tokens = torch.tensor([3, 5, 5, 5, -100]).cuda()
    lp, ent, ids, tlp = ttq.ttq_token_logprobs(x, tokens, top=4)
    assert lp[0].item() == -math.inf and ent[0].item() == 0 and ids[0].tolist() == [0, 1, 2, 3]
    assert bool((tlp[0] == -math.inf).all())
    assert bool(torch.isnan(lp[1:4]).all()) and bool(torch.isnan(ent[1:4]).all())
    assert lp[4].item() == 0 and math.isfinite(ent[4].item())
    assert ids[2].tolist() == [0, 1, 2, 3] and ids[3, 0].item() == 4000
    order = torch.sort(torch.nan_to_num(x[1], nan=-1e30), descending=True, stable=True).indices[:4]
    assert torch.equal(ids[1], order)
    lp2, _ = ttq.ttq_token_logprobs(x[4:], torch.tensor([9000]).cuda())
    assert lp2.item() == 0


@pytest.mark.parametrize("dtype", [torch.float32, F16])
def test_token_logprobs_strided_and_unaligned(dtype):
    g = torch.Generator().manual_seed(4)
    wide = (torch.randn((9, 5003), generator=g) * 3).to(dtype).cuda()
    tokens = torch.randint(0, 4099, (9,), generator=g).cuda()
    check_logprobs(wide[:, 3:4102], tokens, 12)
    check_logprobs(wide[:1, 1:], torch.tensor([5001]).cuda(), 5)


def test_token_logprobs_rows_past_2_gib():
    """Row offsets beyond 32 bits."""
    T, V = 5000, 150001
    x = torch.empty((T, V), dtype=BF16, device="cuda")
    x.fill_(-3.0)
    x[:, 7] = 4.0
    x[T - 1, V - 1] = 9.0
    tokens = torch.full((T,), 7, device="cuda")
    lp, ent, ids, _ = ttq.ttq_token_logprobs(x, tokens, top=2)
    assert ids[T - 1].tolist() == [V - 1, 7] and ids[T - 2].tolist() == [7, 0]
    want = torch.log_softmax(x[T - 1].double(), 0)[7].item()
    assert abs(lp[T - 1].item() - want) < 1e-3 and abs(lp[0].item() - lp[T - 2].item()) == 0


# -- refusals of the Python functions ----------------------------------------
def test_python_refusals():
    b = Batch([(2, 20), (1, 5)], 2, 64, 16, F16)
    q = torch.zeros((3, 4 * 64), dtype=F16, device="cuda")
    rest = (b.dtable, b.q_start, b.kv_len, 2, 20)
    call = ttq.ttq_paged_attention
    with pytest.raises(TypeError, match="Q must be Half"):
        call(q.float(), b.k, b.v, *rest)
    with pytest.raises(ValueError, match="Q must be"):
        call(q[:, ::2], b.k, b.v, *rest)
    with pytest.raises(ValueError, match="Q must be"):
        call(q[:, :100], b.k, b.v, *rest)
    with pytest.raises(ttq.TTQError, match="multiple of n_kv_heads"):
        call(q[:, :3 * 64], b.k, b.v, *rest)
    with pytest.raises(ttq.TTQError, match="16-byte aligned"):
        call(torch.zeros((3, 304), dtype=F16, device="cuda")[:, 1:257], b.k, b.v, *rest)
    with pytest.raises(TypeError, match="vcache must be"):
        call(q, b.k, b.v.float(), *rest)
    with pytest.raises(ValueError, match="one shape"):
        call(q, b.k, b.v[:-1], *rest)
    with pytest.raises(ValueError, match="dense"):
        call(q, b.k.transpose(1, 2).contiguous().transpose(1, 2), b.v.transpose(1, 2).contiguous().transpose(1, 2), *rest)
    with pytest.raises(TypeError, match="block_table must be Int"):
        call(q, b.k, b.v, b.dtable.long(), b.q_start, b.kv_len, 2, 20)
    with pytest.raises(ValueError, match="q_start must be a dense vector of 3"):
        call(q, b.k, b.v, b.dtable, b.q_start[:2], b.kv_len, 2, 20)
    with pytest.raises(ValueError, match="must be on the GPU"):
        call(q, b.k, b.v, b.table, b.q_start, b.kv_len, 2, 20)
    with pytest.raises(ttq.TTQError, match="window"):
        call(q, b.k, b.v, *rest, window=-1)
    with pytest.raises(ttq.TTQError, match="head_dim"):
        call(torch.zeros((3, 4 * 32), dtype=F16, device="cuda"), b.k.reshape(-1, 2, 32, 32), b.v.reshape(-1, 2, 32, 32), *rest)
    with pytest.raises(ValueError, match="slopes"):
        call(q, b.k, b.v, *rest, slopes=torch.zeros(3, device="cuda"))
    with pytest.raises(ValueError, match="lse"):
        call(q, b.k, b.v, *rest, lse=torch.zeros(3, device="cuda"))
    with pytest.raises(ValueError, match="out must be"):
        call(q, b.k, b.v, *rest, out=q[:2])
    with pytest.raises(ValueError, match="K must be"):
        ttq.ttq_cache_write(q, q, b.k, b.v, *rest[:3])
    with pytest.raises(TypeError, match="src must be Int"):
        ttq.ttq_cache_copy_pages(b.k, b.v, torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda"))
    x = torch.zeros((2, 10), device="cuda")
    with pytest.raises(TypeError, match="logits must be Float"):
        ttq.ttq_token_logprobs(x.double(), torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(TypeError, match="tokens must be Long"):
        ttq.ttq_token_logprobs(x, torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ttq.TTQError, match="top=11 exceeds"):
        ttq.ttq_token_logprobs(x, torch.zeros(2, dtype=torch.int64, device="cuda"), top=11)
    with pytest.raises(ttq.TTQError, match="workspace"):
        ttq.ttq_token_logprobs(torch.zeros((1, 100000), device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda"),
                               workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


# -- all of them together ----------------------------------------------------
def test_example_scores_and_decodes():
    """The example's answers against the same model fed the whole text again:
    decoding over forked, freed and compacted pages gives what a prompt gives."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "score_and_decode.py")
    spec = importlib.util.spec_from_file_location("score_and_decode", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    got = ex.run(tokens=300, answers=4, steps=10, show=say)
    # 4-bit weights move the perplexity of this model by a few percent; a wrong operator by far more
    assert abs(got["perplexity"] / got["dense_perplexity"] - 1) < 0.15
    model, text = got["model"], got["text"]
    for name in got["kept"]:
        said = torch.tensor(got["said"][name], device="cuda")
        whole = torch.cat([text, said[:-1]])
        # the prompt's quantisation, the whole text at once through every projection and the attention
        x = model.embed[whole]
        qkv = model.proj["qkv"].linear(x)
        att = model.attend(qkv, [name + " again"], [len(whole)])
        logits = model.proj["head"].linear(x + model.proj["out"].linear(att))
        lp, _ = ttq.ttq_token_logprobs(logits[len(text) - 1:].contiguous(), said)
        # fp16 activations between the layers: a few units in the last place of logits of about 10
        assert abs(float(lp.sum()) - got["score"][name]) < 0.02 * len(said)
        model.cache.free(name + " again")
