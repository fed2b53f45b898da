"""Each form of the paged attention, by sizes whose plan is asserted: tiles of
128 rows that share their keys (one and two halves of a workgroup, split and
not), tiles of 32 rows whose waves have keys of their own (one, two and four
waves, split and not), with every kind of score and mask in each."""
import math

import pytest

torch = pytest.importorskip("torch")
import test_activation_aware_amd as ttq  # noqa: E402
import test_gpu_serving as base  # noqa: E402
from attention_plan import plan  # noqa: E402
from test_gpu_serving import BF16, F16, U, Batch, attention_ref, check_attention, say  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    ttq.load()
    yield
    torch.cuda.synchronize()


# Sequences of odd lengths: prompts, chunks, decode tokens, tiles that end inside 32 and inside 128 rows.
RAGGED = [(5, 5), (1, 77), (129, 129), (64, 200), (31, 333), (1, 1), (2, 64), (257, 300)]
MASKS = [(5, 5), (1, 77), (100, 129), (40, 300), (130, 130)]
MODS = [dict(softcap=20.0), dict(softcap=100.0), dict(slopes=True), dict(window=1), dict(window=70),
        dict(window=64, softcap=30.0, slopes=True), dict(prefix=[3, 64, 0, 150, 129]),
        dict(prefix=[5, 1, 40, 299, 10], window=33),
        dict(prefix=[2, 77, 100, 0, 65], window=40, slopes=True, softcap=50.0),
        dict(prefix=[2, 77, 100, 0, 65], window=40, slopes=True, softcap=200.0)]
# Query heads and key heads by which these reach a form: (dim, waves) -> for RAGGED, for MASKS.
HEADS = {(64, 8): ((48, 16), (96, 16)), (64, 4): ((128, 64), (256, 64)), (128, 8): ((48, 16), (96, 16)),
         (128, 4): ((64, 32), (128, 32)), (256, 8): ((48, 16), (96, 16)), (256, 4): ((64, 32), (128, 32))}


def check(form, lens, heads, kv_heads, dim, page, dtype, **how):
    asked = {k: v for k, v in how.items() if k in ("window", "prefix", "bounds")}
    assert plan(lens, heads, kv_heads, dim, **asked) == form
    check_attention(lens, heads, kv_heads, dim, page, dtype, **how)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("dim,waves", HEADS)
def test_rows(dim, waves, dtype):
    heads, kv_heads = HEADS[dim, waves][0]
    check(("rows", waves, 1), RAGGED, heads, kv_heads, dim, 32, dtype)


@pytest.mark.parametrize("mods", MODS)
@pytest.mark.parametrize("dim,waves", HEADS)
def test_rows_scores_and_masks(dim, waves, mods):
    heads, kv_heads = HEADS[dim, waves][1]
    check(("rows", waves, 1), MASKS, heads, kv_heads, dim, 16, BF16 if dim == 128 else F16, **mods)


@pytest.mark.parametrize("dim,waves", HEADS)
def test_rows_strides(dim, waves):
    heads, kv_heads = HEADS[dim, waves][1]
    check(("rows", waves, 1), MASKS, heads, kv_heads, dim, 64, F16, strided=True)
    check(("rows", waves, 1), MASKS, heads, kv_heads, dim, 256, BF16, interleaved=True)


EMPTY = [[(3, 0), (2, 5), (0, 0), (0, 40), (1, 1), (140, 0), (33, 33), (260, 64)],
         [(9, 4), (170, 3), (1, 130), (140, 139)],
         [(0, 0)] * 70 + [(1, 33)] + [(0, 10)] * 5 + [(2, 20)] * 66 + [(0, 0)] * 64 + [(50, 50)]]


@pytest.mark.parametrize("lens", EMPTY)
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_rows_empty(lens, dim):
    """Bounds far above the lengths bring few rows here; rows that see nothing, sequences without tokens or keys."""
    bounds = (max(q for q, _ in lens), 1 << 20)
    assert plan(lens, 8, 4, dim, bounds=bounds)[0] == "rows"
    check_attention(lens, 8, 4, dim, 16, F16, bounds=bounds)
    check_attention(lens, 8, 4, dim, 16, BF16, bounds=bounds, window=20, softcap=30.0)


@pytest.mark.parametrize("dim,heads,kv_heads,lens,mods", [
    (64, 64, 8, [(112, 8300)], {}),
    (64, 64, 8, [(100, 8300), (1, 3), (12, 900), (1, 0), (5, 5)], dict(softcap=30.0, slopes=True)),
    (128, 64, 8, [(70, 6700)], {}),
    (128, 64, 8, [(70, 6700), (1, 40), (20, 1500)], dict(prefix=[700, 3, 20], window=3000)),
    (256, 32, 4, [(40, 5600)], {}),
    (256, 32, 4, [(40, 5600), (1, 40), (20, 1500)], dict(softcap=90.0)),
])
def test_rows_split(dim, heads, kv_heads, lens, mods):
    asked = {k: v for k, v in mods.items() if k in ("window", "prefix")}
    form = plan(lens, heads, kv_heads, dim, **asked)
    assert form[:2] == ("rows", 8) and form[2] > 2
    check_attention(lens, heads, kv_heads, dim, 64, F16 if dim != 128 else BF16, **mods)


@pytest.mark.parametrize("dim,waves", HEADS)
def test_rows_large_scores(dim, waves):
    """Scores of several hundred: the running maximum has to follow, in both halves."""
    heads, kv_heads = HEADS[dim, waves][1]
    assert plan(MASKS, heads, kv_heads, dim) == ("rows", waves, 1)
    b = Batch(MASKS, kv_heads, dim, 16, F16, seed=5)
    q = torch.randn((b.total, heads * dim), generator=b.gen).mul(40).to(F16)
    got = ttq.ttq_paged_attention(q.cuda(), b.k, b.v, b.dtable, b.q_start, b.kv_len, 130, 300).cpu().double()
    o, _, A, _ = attention_ref(b, q, heads, dim ** -0.5)
    # a score of 300 is off by up to dim * 2^-24 * sum |q k| ~ 2e-3 relative to the others (dim 256: 8e-3)
    assert float(((got.reshape(o.shape) - o).abs() - (2 * U[F16] + 5e-3 * dim / 64) * A - 1e-4).max()) <= 0


VALUES = [(64, 8, 128, 64, BF16, [(300, 300)], {}), (64, 4, 128, 64, F16, [(700, 700), (600, 650)], dict(window=200)),
          (64, 8, 128, 64, F16, [(200, 333), (100, 140)], dict(window=40)),
          (128, 8, 96, 16, F16, [(200, 333), (1, 40)], dict(window=40)),
          (128, 4, 128, 32, BF16, [(300, 320), (9, 100), (1, 64)], dict(prefix=[170, 95, 3])),
          (256, 8, 96, 16, F16, [(300, 300)], dict(window=100, prefix=[70])),
          (256, 4, 128, 32, BF16, [(300, 320), (9, 100), (1, 64)], {})]


@pytest.mark.parametrize("dim,waves,heads,kv_heads,dtype,lens,how", VALUES)
def test_rows_masked_values_hold_anything(dim, waves, heads, kv_heads, dtype, lens, how):
    """NaN and infinities in V next to what a query sees, as in the key form's test of it."""
    assert plan(lens, heads, kv_heads, dim, **how) == ("rows", waves, 1)
    base.test_attention_masked_values_hold_anything(lens, dict(how), dim, heads, kv_heads, dtype)


def test_rows_split_masked_values_hold_anything():
    lens = [(70, 7000)]
    form = plan(lens, 64, 8, 128, window=6700)
    assert form[0] == "rows" and form[2] > 2
    base.test_attention_masked_values_hold_anything(lens, dict(window=6700), 128, 64, 8, F16)


@pytest.mark.parametrize("dim,waves", HEADS)
def test_rows_masked_keys_hold_anything(dim, waves):
    heads, kv_heads = HEADS[dim, waves][0]
    assert plan(RAGGED, heads, kv_heads, dim) == ("rows", waves, 1)
    b = Batch(RAGGED, kv_heads, dim, 16, F16)
    q = torch.randn((b.total, heads * dim), generator=b.gen).to(F16).cuda()
    rest = (b.dtable, b.q_start, b.kv_len, 257, 333)
    clean = ttq.ttq_paged_attention(q, b.k, b.v, *rest)
    at = b.total - 257  # the last sequence's first row, its last keys seen by its last rows only
    for pos, bad in ((299, math.nan), (298, math.inf), (297, -math.inf)):
        b.k[int(b.table[7, pos // 16]), :, pos % 16] = bad
    got = ttq.ttq_paged_attention(q, b.k, b.v, *rest)
    assert torch.equal(got[:at + 254], clean[:at + 254])
    assert bool(torch.isnan(got[at + 256]).all())


# -- the key form: what the other tests do not reach -------------------------------
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("dim,heads,kv_heads", [(64, 32, 8), (128, 24, 8), (256, 8, 8)])
def test_keys_one_wave(dim, heads, kv_heads, dtype):
    """Many short sequences, a wave an item; some without keys, some of a few tokens."""
    lens = [(1, n) for n in (1, 2, 31, 32, 33, 63, 64, 65, 200, 499, 900)] * 6 + [(1, 0), (0, 9), (5, 40), (8, 7)]
    for mods in ({}, dict(softcap=30.0, window=40), dict(softcap=80.0), dict(slopes=True, prefix=[7] * len(lens))):
        prefix = mods.get("prefix")
        if prefix is not None:
            mods = dict(mods, prefix=[min(7, k) for _, k in lens])
        check(("keys", 1, 1), lens, heads, kv_heads, dim, 16, dtype, **mods)


@pytest.mark.parametrize("dim,heads,kv_heads,dtype", [(64, 32, 8, BF16), (128, 24, 8, F16), (256, 8, 8, BF16)])
def test_keys_one_wave_masked_values(dim, heads, kv_heads, dtype):
    lens = [(1, 300), (1, 77), (5, 100)] * 25
    assert plan(lens, heads, kv_heads, dim, window=30) == ("keys", 1, 1)
    base.test_attention_masked_values_hold_anything(lens, dict(window=30), dim, heads, kv_heads, dtype)


@pytest.mark.parametrize("dim,waves", [(64, 4), (128, 4), (256, 2)])
def test_keys_split(dim, waves):
    """Every kind of score in split keys, sequences of one share beside them."""
    lens = [(1, 9000), (1, 3), (1, 0), (3, 5000)]
    for mods in ({}, dict(softcap=30.0), dict(softcap=80.0, slopes=True), dict(slopes=True), dict(window=3000),
                 dict(prefix=[4000, 1, 0, 50], window=700)):
        asked = {k: v for k, v in mods.items() if k in ("window", "prefix")}
        form = plan(lens, 4, 2, dim, **asked)
        assert form[:2] == ("keys", waves) and form[2] > 1
        check_attention(lens, 4, 2, dim, 64, BF16 if dim == 64 else F16, **mods)


@pytest.mark.parametrize("dim,lens,heads,kv_heads", [(64, RAGGED, 48, 16), (64, RAGGED, 128, 64), (128, RAGGED, 64, 32),
                                                    (256, RAGGED, 48, 16), (128, [(70, 6700)], 64, 8),
                                                    (128, [(1, 100), (1, 33)] * 40, 16, 8)])
def test_forms_in_a_graph(dim, lens, heads, kv_heads):
    """Captured once, replayed with other contents, other work between the replays."""
    say(f"graph {plan(lens, heads, kv_heads, dim)}")
    b = Batch(lens, kv_heads, dim, 32, F16)
    q = torch.zeros((b.total, heads * dim), dtype=F16, device="cuda")
    max_q, max_kv = max(x for x, _ in lens), max(x for _, x in lens)

    def step():
        return ttq.ttq_paged_attention(q, b.k, b.v, b.dtable, b.q_start, b.kv_len, max_q, max_kv, softcap=40.0)

    def fill(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        for t in (b.k, b.v, q):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))

    fill(0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in range(1, 4):
        fill(seed)
        want = step().clone()
        torch.cuda.synchronize()
        fill(seed)
        graph.replay()
        got = held.clone()
        torch.cuda.synchronize()
        assert torch.equal(got, want)


SEEN = [("keys", 4, 64, 12, 4, [(1, 333), (20, 700)]), ("keys", 2, 256, 4, 2, [(1, 333), (9, 700)]),
        ("keys", 1, 128, 16, 8, [(1, 100), (1, 333)] * 40), ("keys", 4, 128, 8, 1, [(1, 20000)]),
        ("rows", 8, 128, 96, 16, [(200, 333), (70, 700)]), ("rows", 4, 128, 128, 32, [(300, 320), (129, 500), (1, 64)]),
        ("rows", 8, 64, 96, 16, [(200, 333), (70, 700)]), ("rows", 4, 256, 128, 32, [(300, 320), (129, 500), (1, 64)]),
        ("rows", 8, 128, 64, 8, [(70, 6700)])]


@pytest.mark.parametrize("form,waves,dim,heads,kv_heads,lens", SEEN)
def test_seen_infinities_of_no_weight(form, waves, dim, heads, kv_heads, lens):
    """An infinity in V that a query sees gives that infinity, opposite ones NaN, in whichever tile it lies, also where
    its probability is far below what 32 bits hold (a score of about -600 beside 0)."""
    say(plan(lens, heads, kv_heads, dim))
    assert plan(lens, heads, kv_heads, dim)[:2] == (form, waves)
    page, s = 16, max(range(len(lens)), key=lambda i: lens[i][1])
    b = Batch(lens, kv_heads, dim, page, F16, seed=8)
    q = torch.randn((b.total, heads * dim), generator=b.gen).half().cuda()
    max_q, max_kv = max(x for x, _ in lens), max(x for _, x in lens)
    row, kl = sum(x for x, _ in lens[:s + 1]) - 1, lens[s][1]  # the last token of the longest sequence
    h, group = kv_heads - 1, heads // kv_heads
    head = h * group + group - 1
    mine = q[row, head * dim:(head + 1) * dim]

    def place(pos):
        return int(b.table[s, pos // page]), h, pos % page

    at = [0, 17, 40, kl // 2, kl - 70, kl - 2, kl - 1]
    for pos in at:
        b.k[place(pos)] = -100 * mine.sign()

    def run():
        o = ttq.ttq_paged_attention(q, b.k, b.v, b.dtable, b.q_start, b.kv_len, max_q, max_kv)
        return o[row, head * dim:(head + 1) * dim].cpu()

    clean = run()
    assert bool(torch.isfinite(clean).all())
    for n, pos in enumerate(at):
        keep = b.v[place(pos)].clone()
        want = clean.clone()
        for d, bad in ((0, math.inf), (n + 3, -math.inf), (dim - 1, math.nan)):
            b.v[place(pos)][d] = bad
            want[d] = bad
        got = run()
        assert torch.equal(got.nan_to_num(7e4, 6e4, -6e4), want.nan_to_num(7e4, 6e4, -6e4)), (pos, got, want)
        other = at[n - 1]
        was = b.v[place(other)][0].clone()
        b.v[place(other)][0] = -math.inf
        got = run()
        assert bool(torch.isnan(got[0])) and torch.equal(got[1:-1], want[1:-1])
        b.v[place(other)][0] = was
        b.v[place(pos)] = keep
    assert torch.equal(run(), clean)
