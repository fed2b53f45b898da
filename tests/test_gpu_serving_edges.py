"""The serving operators at the edges of their ranges, on the GPU, against the
same plain statements in 64 bits as the other tests of them."""
import math

import pytest

torch = pytest.importorskip("torch")
import test_activation_aware_amd as ttq  # noqa: E402
from test_gpu_serving import BF16, F16, U, Batch, attention_ref, check_attention, say  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need an MI355X"
    ttq.load()
    yield
    torch.cuda.synchronize()


# -- attention -----------------------------------------------------------------
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 40, 2 ** 30])
@pytest.mark.parametrize("lens", [[(70, 3), (9, 4), (1, 130)], [(3, 0), (200, 100)]])
def test_attention_windows_beyond_every_position(lens, window):
    """With tokens before position 0, whose distance to the window's begin passes 32 bits."""
    check_attention(lens, 4, 2, 64, 16, F16, window=window)
    check_attention(lens, 4, 2, 128, 16, BF16, window=window, prefix=[2, 0, 50][:len(lens)])


@pytest.mark.parametrize("softcap", [1e-39, 1e-30, 0.3, 64.0, 65.0, 1e3, 1e5, 1e7, 1e30, 1e38, 3.4e38])
@pytest.mark.parametrize("dim,dtype,mods", [(64, F16, {}), (128, BF16, dict(slopes=True, window=50)), (256, F16, {})])
def test_attention_caps_of_any_size(softcap, dim, dtype, mods):
    """From caps that flatten every score to caps that change none."""
    check_attention([(5, 5), (1, 77), (40, 300)], 4, 2, dim, 32, dtype, softcap=softcap, **mods)


@pytest.mark.parametrize("softcap", [30.0, 100.0, 1000.0, 1e6])
def test_attention_caps_of_large_scores(softcap):
    """Scores of several hundred on both sides of the cap, and on both sides of half of it."""
    b = Batch([(40, 300)], 2, 64, 16, F16, seed=5)
    q = torch.randn((40, 4 * 64), generator=b.gen).mul(40).to(F16)
    got = ttq.ttq_paged_attention(q.cuda(), b.k, b.v, b.dtable, b.q_start, b.kv_len, 40, 300,
                                  softcap=softcap).cpu().double()
    o, _, A, _ = attention_ref(b, q, 4, 0.125, softcap=softcap)
    # as without a cap: a score of 300 is off by up to 64 * 2^-24 * sum |q k| ~ 2e-3, and a capped one by 2^-20 of it
    assert float(((got.reshape(o.shape) - o).abs() - (2 * U[F16] + 5e-3) * A - 1e-4).max()) <= 0


@pytest.mark.parametrize("dim,heads,kv_heads,lens", [(64, 2, 2, [(64, 300)]), (128, 4, 1, [(40, 900)]),
                                                    (256, 2, 1, [(64, 700)]), (64, 48, 16, [(130, 300), (300, 700)]),
                                                    (128, 64, 32, [(200, 600), (300, 900)])])
def test_attention_bits_of_a_query_are_its_own(dim, heads, kv_heads, lens):
    """A key that only the last token sees, and that token's query, grow large: the others keep their bits."""
    b = Batch(lens, kv_heads, dim, 16, F16, seed=6)
    q = torch.randn((b.total, heads * dim), generator=b.gen).half().cuda()
    max_q, max_kv = max(x for x, _ in lens), max(x for _, x in lens)

    def run():
        return ttq.ttq_paged_attention(q, b.k, b.v, b.dtable, b.q_start, b.kv_len, max_q, max_kv)

    clean, pos = run(), lens[-1][1] - 1
    own = q[-1].reshape(kv_heads, -1, dim)[:, 0]
    b.k[int(b.table[len(lens) - 1, pos // 16]), :, pos % 16] = 8 * own
    got = run()
    assert torch.equal(got[:-1], clean[:-1]) and not torch.equal(got[-1], clean[-1])
    q[-1] *= 30
    got = run()
    assert torch.equal(got[:-1], clean[:-1])


@pytest.mark.parametrize("lens,heads,kv_heads,dim", [([(1, 20000)], 8, 1, 128), ([(40, 300), (1, 9)], 4, 2, 64),
                                                    ([(70, 6700)], 64, 8, 128), ([(130, 300)], 96, 32, 64)])
def test_rows_of_no_sequence_are_left_alone(lens, heads, kv_heads, dim):
    """Tensors with more rows than the sequences have, as a captured step with room for more tokens passes them: in
    both forms, keys split and not, whatever the workspace holds."""
    b = Batch(lens, kv_heads, dim, 64, F16, seed=7)
    max_q, max_kv, more = max(x for x, _ in lens), max(x for _, x in lens), b.total + 3
    q = torch.randn((more, heads * dim), generator=b.gen).half().cuda()
    want = ttq.ttq_paged_attention(q[:b.total], b.k, b.v, b.dtable, b.q_start, b.kv_len, max_q, max_kv)
    out = torch.full((more, heads * dim), 7.0, dtype=F16, device="cuda")
    lse = torch.full((more, heads), 7.0, device="cuda")
    for fill in (0, 2, -1):
        workspace = torch.full((64 << 18,), fill, dtype=torch.int32, device="cuda").view(torch.uint8)
        ttq.ttq_paged_attention(q, b.k, b.v, b.dtable, b.q_start, b.kv_len, max_q, max_kv, out=out, lse=lse,
                                workspace=workspace)
        assert bool((out[b.total:] == 7.0).all()) and bool((lse[b.total:] == 7.0).all()), fill
        # each is off by 2 u A at most (the other tests' bound), A = sum p |v| < 1; other splits round otherwise
        assert torch.allclose(out[:b.total].float(), want.float(), atol=4 * U[F16], rtol=0)
    k, v = b.k.clone(), b.v.clone()
    new = torch.randn((more, kv_heads * dim), generator=b.gen).half().cuda()
    ttq.ttq_cache_write(new, new, k, v, b.dtable, b.q_start, b.kv_len)
    ttq.ttq_cache_write(new[:b.total], new[:b.total], b.k, b.v, b.dtable, b.q_start, b.kv_len)
    assert torch.equal(k.view(torch.int16), b.k.view(torch.int16))
    assert torch.equal(v.view(torch.int16), b.v.view(torch.int16))


@pytest.mark.parametrize("bounds", [(0, 0), (1, 1), (1, 1 << 20), (3, 100), (1 << 20, 1), (1 << 30, 0x7FFFFFFF)])
@pytest.mark.parametrize("lens,heads,kv_heads,dim", [([(40, 300), (1, 9), (1, 2000)], 4, 2, 64),
                                                    ([(130, 300), (5, 700)], 64, 32, 128), ([(1, 9000)], 2, 1, 256)])
def test_attention_bounds_on_either_side(lens, heads, kv_heads, dim, bounds):
    """Longest lengths that are too small or far too large choose other forms and splits, not other results."""
    check_attention(lens, heads, kv_heads, dim, 16, F16, bounds=bounds)


# -- log probabilities ----------------------------------------------------------
def best_ids(x, top):
    """Indices of the `top` best of each row by (value, lowest index), NaN below everything."""
    x = x.double().cpu()
    value = torch.where(torch.isnan(x), torch.full_like(x, -math.inf), x)
    by_value = torch.sort(value, dim=1, descending=True, stable=True).indices
    nan = torch.isnan(x).gather(1, by_value)
    return by_value.gather(1, torch.sort(nan.int(), dim=1, stable=True).indices)[:, :top]


@pytest.mark.parametrize("T,V", [(3, 9000), (3, 70), (3, 1), (2, 33), (3, 4097), (3, 120001), (2, 200003),
                                 (1100, 500)])  # whole rows, rows in chunks, a wave a row
@pytest.mark.parametrize("top", [1, 2, 5])
def test_alternatives_of_rows_with_few_numbers(T, V, top):
    """Rows of NaN but for a few logits, of a length that ends inside a group: every id is written, and right."""
    top = min(top, V)
    for numbers in ([], [V - 1], [V // 2], [0, V - 1], list(range(max(0, V - V % 32 - 1), V))[:top]):
        for value in (1.5, -math.inf):
            x = torch.full((T, V), math.nan)
            for i in numbers:
                x[:, i] = value - i * 1e-6 if math.isfinite(value) else value
            for dtype in (torch.float32, BF16):
                y = x.to(dtype).cuda()
                junk = torch.full((T * top,), 0x1234567812345678, dtype=torch.int64, device="cuda")
                del junk  # what the allocator hands out next
                _, _, ids, lp = ttq.ttq_token_logprobs(y, torch.zeros(T, dtype=torch.int64, device="cuda"), top=top)
                assert torch.equal(ids.cpu(), best_ids(y, top)), (numbers, value, dtype)
                if bool(torch.isnan(x).any()):
                    assert bool(torch.isnan(lp).all())


def check_scores(x, tokens, top):
    """Against 64 bits, for any finite logits.  Tolerance: the logits are exact; a log probability x - m - log s
    has two roundings of its own size, 2^-23, and log s of sums of V / 64 terms a thread in 32 bits, each of them
    exp2 of a rounded product of up to 24 where it counts (2^-19), V / 64 * 2^-24 relative; the entropy the same,
    its terms up to 24 times larger."""
    T, V = x.shape
    say(f"scores T={T} V={V} top={top} {x.dtype}")
    got = ttq.ttq_token_logprobs(x, tokens, top=top)
    lp = torch.log_softmax(x.double().cpu(), 1)
    p = lp.exp()
    entropy = torch.where(p > 0, -p * lp, torch.zeros_like(p)).sum(1)
    tol = V / 64 * 2.0 ** -24 + 2.0 ** -18
    lowest = torch.finfo(torch.float32).min

    def near(a, b, t):  # what 32 bits hold no more is -inf, or the lowest value
        a, b = a.cpu().double(), b
        inside = b >= lowest
        ok = torch.where(inside, (a - b).abs() <= t * (1 + b.abs()), a <= lowest)
        assert bool(ok.all()), (a, b)

    near(got[0], lp.gather(1, tokens.cpu()[:, None])[:, 0], tol)
    near(got[1], entropy, 24 * tol)
    if top:
        ids = best_ids(x, top)
        assert torch.equal(got[2].cpu(), ids)
        near(got[3], lp.gather(1, ids), tol)


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
def test_logits_of_any_finite_size(dtype):
    """Rows of equal logits, and of two far apart, up to the type's largest value."""
    g = torch.Generator().manual_seed(3)
    big = torch.finfo(dtype).max
    for V in (1000, 33000):
        x = torch.randn((6, V), generator=g)
        x[4] = -big
        for i, v in enumerate((1e9, 1e30, 3e38, big)):
            x[i] = v
        x[5, ::2], x[5, 1::2] = big, -big
        check_scores(x.to(dtype).cuda(), torch.tensor([5, 5, 5, 5, 5, 4]).cuda(), 4)
        check_scores(x.to(dtype).cuda(), torch.tensor([6, 6, 6, 6, 6, 5]).cuda(), 0)


def masks(dtype):
    values = [-1e4, -1e9, -1e30, -1e37, -1e38, -3e38, torch.finfo(dtype).min]
    return [v for v in values if v >= torch.finfo(dtype).min]


@pytest.mark.parametrize("dtype", [torch.float32, BF16, F16])
@pytest.mark.parametrize("T,V", [(4, 257), (4, 5003), (2, 60000), (3, 120001), (1030, 300)])
def test_logits_masked_by_finite_values(T, V, dtype):
    """Large negative numbers where a vocabulary is masked: for most of it, one token, all but one, all."""
    g = torch.Generator().manual_seed(V)
    base = torch.randn((T, V), generator=g)
    for mask in masks(dtype):
        few, one, single = base.clone(), base.clone(), torch.full((T, V), mask)
        few[:, V // 3:] = mask
        few[0, :V // 2], few[0, V // 2:] = mask, base[0, V // 2:]      # the masked part first
        one[:, 7] = mask
        single[:, V - 5] = 0.25
        for x in (few, one, single, torch.full((T, V), mask)):
            x = x.to(dtype).cuda()
            for tok in (7, V - 5):
                check_scores(x, torch.full((T,), tok, dtype=torch.int64, device="cuda"), 3)


def test_a_logit_far_above_the_others():
    """The type's largest value beside ordinary ones, in another thread's part and in another chunk."""
    g = torch.Generator().manual_seed(5)
    for V in (1000, 33000, 250001):
        for at in (0, 5, V // 2, V - 1):
            x = torch.randn((2, V), generator=g)
            x[:, at] = torch.finfo(torch.float32).max
            check_scores(x.cuda(), torch.tensor([at, (at + 1) % V]).cuda(), 4)


def test_largest_selections():
    """64 alternatives out of rows that one workgroup reads: most of the shared memory that a selection takes."""
    g = torch.Generator(device="cuda").manual_seed(4)
    for T, V, dtype in ((130, 262144, F16), (129, 170001, torch.float32), (257, 300000, BF16)):
        x = torch.randn((T, V), generator=g, device="cuda").to(dtype)
        say(f"largest selections {T} x {V} {dtype}")
        ids = ttq.ttq_token_logprobs(x, torch.zeros(T, dtype=torch.int64, device="cuda"), top=64)[2]
        want = torch.sort(x.float(), dim=1, descending=True, stable=True).indices[:, :64]
        assert torch.equal(ids, want)
