"""Attention over the 4-bit cache against plain numpy in 64 bits, every way a
call can be cut (asserted by its plan).

Tolerances.  With u the half step of the type that the keys, values and
probabilities are rounded to (2^-11 in fp16, which sequences of few rows are
worked on in; the rows' own type where pages are brought to 16 bits): a score is
off by at most dz = scale * u * max_j sum_c |q_c k_jc| (a cap makes that smaller,
and adds 3e-7 of itself), so a probability by 2 dz of itself, and the output by
sum_j p_j |v_j| * (2 dz + u [v] + u [p]) and its own rounding.  Sums and
exponentials in 32 bits add some 1e-6 of it.  Roundings being independent, the
whole output's norm is off by far less: three half steps are allowed (one each
for scores, for values and probabilities, and for the output)."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")
import packed_reference as ref  # noqa: E402
import test_activation_aware_amd as ttq  # noqa: E402
from test_activation_aware_amd import _capi  # noqa: E402

pytestmark = pytest.mark.gpu
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# Bounds that admit prompts with much to do: sequences of more rows than those of a few tokens then go by 16-bit pages.
PROMPTS = (1000, 1 << 20)


class Batch:
    def __init__(self, lens, heads=4, kv_heads=2, dim=128, page=16, dtype="f16", seed=0, spare=0, extra_pages=3,
                 columns=0, fused=False, q_scale=1.5, spread=1.0):
        rng = np.random.default_rng(seed)
        self.lens, self.heads, self.kvh, self.dim, self.page = lens, heads, kv_heads, dim, page
        self.dtype = TYPES[dtype]
        need = [-(-k // page) for _, k in lens]
        n = sum(need) + extra_pages
        order = rng.permutation(n).astype(np.int32)
        self.table = np.full((len(lens), max(need + [1]) + columns), -1, np.int32)
        at = 0
        for i, m in enumerate(need):
            self.table[i, :m] = order[at:at + m]
            at += m
        self.pools, self.values = [], []
        for keys in (True, False):
            pool = np.empty((n, kv_heads, page, dim * 5 // 8), np.uint8)
            self.values.append(ref.fill(pool, keys, rng, spread))
            self.pools.append(pool)
        self.rows = sum(q for q, _ in lens) + spare
        wide = (heads + 2 * kv_heads) * dim if fused else heads * dim
        q = torch.from_numpy((rng.standard_normal((self.rows, wide)) * q_scale).astype(np.float32)).to(self.dtype)
        self.q = q
        self.starts = np.cumsum([0] + [q for q, _ in lens]).astype(np.int32)
        self.kv = np.array([k for _, k in lens], np.int32)

    def on_gpu(self):
        dev = {"q": self.q.cuda()[:, :self.heads * self.dim], "k": torch.from_numpy(self.pools[0]).cuda(),
               "v": torch.from_numpy(self.pools[1]).cuda(), "table": torch.from_numpy(self.table).cuda(),
               "starts": torch.from_numpy(self.starts).cuda(), "kv": torch.from_numpy(self.kv).cuda()}
        self.dev = dev
        return dev

    def bounds(self):
        return max([q for q, _ in self.lens] + [0]), max([k for _, k in self.lens] + [0])

    def run(self, bounds=None, slopes=None, prefix=None, want_lse=True, **how):
        d = self.on_gpu()
        bounds = bounds or self.bounds()
        out = torch.full((self.rows, self.heads * self.dim), 77.0, dtype=self.dtype, device="cuda")
        lse = torch.full((self.rows, self.heads), 77.0, device="cuda") if want_lse else None
        got = ttq.ttq_packed_attention(
            d["q"], d["k"], d["v"], d["table"], d["starts"], d["kv"], bounds[0], bounds[1], out=out, lse=lse,
            slopes=None if slopes is None else torch.tensor(slopes, dtype=torch.float32, device="cuda"),
            prefix_len=None if prefix is None else torch.tensor(prefix, dtype=torch.int32, device="cuda"), **how)
        assert got is out
        torch.cuda.synchronize()
        return out.double().cpu().numpy(), None if lse is None else lse.double().cpu().numpy()

    def plan(self, bounds=None, window=0, prefix=None):
        bounds = bounds or self.bounds()
        c = _capi.ttq_packed_cache(1 << 20, 1 << 20, len(self.pools[0]), self.pools[0][0].size, self.kvh, self.page,
                                   self.dim, _capi.TTQ_F16)
        b = _capi.ttq_paged_batch(1 << 20, 1 << 20, 1 << 20, self.table.shape[1], self.table.shape[1], len(self.lens),
                                  self.rows, *bounds)
        a = _capi.ttq_attention(self.heads, 0.1, 0.0, window, None, None if prefix is None else 1 << 20)
        p = _capi.ttq_packed_plan()
        status = ttq.load().ttq_packed_attention_plan(ctypes.byref(c), ctypes.byref(b), ctypes.byref(a), ctypes.byref(p))
        assert status == 0, ttq.load().ttq_last_error()
        return p

    def want(self, scale=None, softcap=0.0, window=0, slopes=None, prefix=None, u=2.0 ** -11):
        """(outputs, lse, tolerance of each output, of each lse) of the batch's rows."""
        scale = self.dim ** -0.5 if scale is None else scale
        group, out, lses, tol, lse_tol = self.heads // self.kvh, [], [], [], []
        K, V = self.values
        for s, (ql, kl) in enumerate(self.lens):
            pages = self.table[s, :-(-kl // self.page)]
            x = self.q[self.starts[s]:self.starts[s + 1], :self.heads * self.dim].double().numpy().reshape(ql, self.heads, self.dim)
            o, t, ls, lt = np.zeros(x.shape), np.zeros(x.shape), np.full((ql, self.heads), -np.inf), np.zeros((ql, self.heads))
            i = np.arange(kl - ql, kl)[:, None]
            j = np.arange(kl)[None, :]
            seen = (j <= i) & ((i - j < window) if window else True)
            if prefix is not None:
                seen |= j < prefix[s]
            for h in range(self.heads):
                k, v = (c[pages][:, h // group].reshape(-1, self.dim)[:kl] for c in (K, V))
                z = scale * (x[:, h] @ k.T)
                dz = scale * u * (np.abs(x[:, h]) @ np.abs(k).T)
                if softcap:
                    z = softcap * np.tanh(z / softcap)
                    dz = dz + 3e-7 * softcap
                if slopes is not None:
                    z = z - slopes[h] * np.abs(i - j)
                    dz = dz + 2.0 ** -23 * slopes[h] * np.abs(i - j)
                z = np.where(seen, z, -np.inf)
                dz = np.where(seen, dz, 0).max(1, initial=0.0)[:, None]
                live = seen.any(1)
                if not live.any():
                    continue
                m = z[live].max(1, keepdims=True)
                e = np.exp(z[live] - m)
                p = e / e.sum(1, keepdims=True)
                o[live, h] = p @ v
                t[live, h] = (p @ np.abs(v)) * (2 * dz[live] + 2 * u + 4e-6)
                ls[live, h] = (m + np.log(e.sum(1, keepdims=True)))[:, 0]
                lt[:, h] = dz[:, 0]
            half = torch.finfo(self.dtype).eps / 2
            out.append(o.reshape(ql, self.heads * self.dim))
            tol.append((t + (np.abs(o) + t) * half + 1e-7).reshape(ql, self.heads * self.dim))
            lses.append(ls)
            lse_tol.append(lt)
        return tuple(np.concatenate(x) for x in (out, lses, tol, lse_tol))

    def check(self, bounds=None, u=None, **how):
        few = self.plan(bounds, how.get("window", 0), how.get("prefix")).expand_from == 0
        half = torch.finfo(self.dtype).eps / 2
        u = 2.0 ** -11 if few else half
        got, lse = self.run(bounds, **how)
        want, wl, tol, lse_tol = self.want(u=u, **{k: v for k, v in how.items() if k != "want_lse"})
        n = len(want)
        assert (got[n:] == 77).all() and (lse[n:] == 77).all()  # rows of no sequence
        off = np.abs(got[:n] - want)
        assert (off <= tol).all(), (np.argwhere(~(off <= tol))[:5], (off / tol).max())
        if np.linalg.norm(want):
            assert np.linalg.norm(off) <= 3 * half * np.linalg.norm(want), np.linalg.norm(off) / np.linalg.norm(want) / half
        assert np.array_equal(np.isinf(lse[:n]), np.isinf(wl))
        live = np.isfinite(wl)
        # log sum e^z moves by no more than the scores do (its derivatives are the probabilities, which add up to 1);
        # 32 bits of scores and of the sum of the maximum and a logarithm come on top, some units of 2^-23 of each
        assert (np.abs(lse[:n][live] - wl[live]) <= (lse_tol + 2e-6 * np.abs(wl) + 1e-5)[live]).all()


DECODE = ((1, 1), (1, 15), (1, 16), (1, 17), (1, 33), (0, 50), (1, 200), (1, 64))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads,kv_heads,dim,page", [(12, 12, 64, 16), (16, 2, 64, 32), (8, 1, 128, 16), (4, 2, 128, 64),
                                                     (16, 8, 128, 128), (6, 3, 256, 16), (8, 1, 256, 256), (24, 1, 128, 16)])
def test_decode(heads, kv_heads, dim, page, dtype):
    Batch(DECODE, heads, kv_heads, dim, page, dtype, spare=2, fused=True).check()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("q_len,rows", [(1, 16), (4, 16), (5, 32), (8, 32), (12, 32), (50, 32)])
def test_tiles_of_rows(dim, q_len, rows, dtype):
    """A few tokens of each sequence: 16 and 32 rows a tile (16 for heads of 256), one tile and more; whole contexts,
    and shares of them."""
    for longest, shares in ((100, False), (1200, True)):
        b = Batch([(q_len, k) for k in (q_len, q_len + 1, 80, longest)] + [(q_len - 1, 70), (0, 0)], 8, 2, dim, 16, dtype)
        p = b.plan()
        assert p.rows == (16 if dim == 256 else rows) and p.expand_from == 0 and (p.shares > 0) == shares
        b.check()


MODS = [dict(softcap=30.0), dict(softcap=5.0), dict(softcap=100.0), dict(window=7), dict(window=1), dict(window=50),
        dict(slopes=[0.5, 0.1, 0.02, 0.0]), dict(softcap=20.0, slopes=[0.3, 0.3, 0.01, 1.0], window=33),
        dict(softcap=80.0, slopes=[0.3, 0.3, 0.01, 1.0]), dict(prefix=[0, 5, 40, 100, 3]), dict(scale=0.5),
        dict(prefix=[16, 1, 20, 90, 0], window=4), dict(prefix=[1, 1, 39, 50, 64], slopes=[0.1, 0.2, 0.3, 0.4])]


@pytest.mark.parametrize("how", MODS, ids=[",".join(m) + str(i) for i, m in enumerate(MODS)])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("q_len", [1, 5, 20, 90])
@pytest.mark.parametrize("longest", [100, 1200])
def test_scores_and_masks(longest, q_len, dim, how):
    """Caps (both forms), bias, windows and prefixes over decode tokens and few rows; whole contexts, and shares of them."""
    lens = [(min(q_len, k), k) for k in (16, 30, 40, longest, 64)]
    Batch(lens, 4, 2, dim, 16, "f16" if dim != 128 else "bf16").check(**how)


@pytest.mark.parametrize("how", MODS, ids=[",".join(m) + str(i) for i, m in enumerate(MODS)])
def test_scores_and_masks_of_prompts(how):
    lens = [(16, 16), (1, 30), (40, 40), (700, 760), (0, 64)]
    b = Batch(lens, 4, 2, 64, 16)
    assert 0 < b.plan(PROMPTS).expand_from <= 6000
    b.check(PROMPTS, **how)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 16), (128, 64), (256, 32)])
@pytest.mark.parametrize("spread", [0, 200])
def test_prompts_beside_decode_tokens(dim, page, dtype, spread):
    """Sequences of many rows by 16-bit pages, the others as they are held; pages numbered by sequence and block, or
    (few blocks of many pages: `spread` more columns) as in the cache."""
    lens = ((100, 100), (1, 300), (0, 20), (33, 40), (400, 433), (1, 1), (16, 128), (65, 65), (290, 290))
    b = Batch(lens, 8, 2, dim, page, dtype, spare=3, columns=0 if spread == 0 else spread, extra_pages=3 + 1000 * (spread == 0))
    p = b.plan(PROMPTS)
    assert 4 * 33 < p.expand_from <= 4 * 290 and p.own_table == (spread == 0)
    b.check(PROMPTS)
    b.check(PROMPTS, window=50)
    b.check()


def test_much_to_do():
    """The same by the lengths themselves; the prompts' keys are not split."""
    b = Batch(((2400, 2500), (1, 900), (2500, 2500)), 16, 16, 64, 16)
    p = b.plan()
    assert p.expand_from > 1 and p.expand_splits == 1
    b.check()


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_one_prompt(dim):
    """A single sequence goes one way, whatever its rows are: also when there are few where the bounds admit many."""
    b = Batch(((300, 450),), 8, 2, dim, 16, spare=1)
    p = b.plan(PROMPTS)
    assert p.expand_from == 1 and p.rows == 0
    b.check(PROMPTS)
    b.check(PROMPTS, window=33, softcap=20.0)
    b = Batch(((1, 450),), 8, 2, dim, 16, spare=600)
    assert b.plan(PROMPTS).expand_from == 1
    b.check(PROMPTS)
    Batch(((0, 450),), 8, 2, dim, 16, spare=600).run(PROMPTS)


@pytest.mark.parametrize("dim,heads,kv_heads", [(128, 8, 1), (64, 4, 4), (256, 6, 3), (128, 24, 1)])
def test_shares(dim, heads, kv_heads):
    """Equal shares of the work that begin and end inside sequences: long ones in many, short ones several in one."""
    b = Batch(((1, 5000), (1, 700), (1, 3), (0, 9), (2, 1500), (1, 1)), heads, kv_heads, dim, 64)
    assert b.plan().shares > 0
    b.check()
    b.check(softcap=30.0, window=600)
    b.check(prefix=[700, 0, 3, 9, 64, 1], window=100)


def test_shares_of_many_sequences():
    """More than 64 sequences, of which a share has several."""
    rng = np.random.default_rng(0)
    lens = [(int(rng.integers(0, 4)), int(rng.integers(3, 60))) for _ in range(300)]
    lens[70] = (3, 1000)
    lens[200] = (2, 3000)
    b = Batch(lens, 4, 2, 64, 16, spare=2)
    assert b.plan().shares > 0
    b.check()


def test_splits_beside_shares():
    """A prompt whose keys are split beside decode tokens that are shared."""
    b = Batch(((1, 3000), (70, 3000), (0, 0), (1, 64)), 8, 1, 64, 64, "bf16")
    p = b.plan(PROMPTS)
    assert p.expand_from > 0 and p.expand_splits > 1 and p.shares > 0
    b.check(PROMPTS)


@pytest.mark.parametrize("bounds", [(1, 1), (1, 100000), (1000, 10), PROMPTS, (60, 3000), (0, 0)])
def test_bounds_cost_speed_only(bounds):
    for lens in (((3, 300), (1, 40), (0, 9)), ((150, 200), (1, 1500), (300, 300))):
        Batch(lens, 8, 2, 128, 16, spare=1).check(bounds=bounds)


def test_one_wave_workgroups():
    """Many short contexts: a wave each."""
    b = Batch([(1, 1 + i % 40) for i in range(300)], 8, 8, 64, 16)
    assert b.plan().waves == 1
    b.check()


@pytest.mark.parametrize("q_len", [1, 40, 300])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_what_lies_behind_the_last_key(dim, q_len):
    """Places past a sequence's end hold anything, scales of NaN and infinity among it."""
    b = Batch(((min(q_len, 41), 41), (q_len, q_len), (1, 17)), 4, 2, dim, 32)
    bounds = PROMPTS if q_len == 300 else None
    clean, _ = b.run(bounds)
    for pool, keys in zip(b.pools, (True, False)):
        for s, (_, kl) in enumerate(b.lens):
            for p in range(kl, -(-kl // b.page) * b.page):
                words, scales, apart = ref.places(dim, p % b.page, keys)
                for h in range(b.kvh):
                    flat = pool[b.table[s, p // b.page], h].reshape(-1)
                    for at in scales:
                        flat[at:at + 2] = np.array([0x7E00 if p % 2 else 0x7C00], np.uint16).view(np.uint8)
                        flat[at + apart:at + apart + 2] = np.array([0xFC00], np.uint16).view(np.uint8)
    dirty, _ = b.run(bounds)
    assert np.isfinite(dirty).all() and np.array_equal(clean, dirty)
    b.check(bounds)


def test_rows_that_see_nothing():
    """Positions before 0 (more new tokens than the cache holds): zeros, and a sum of nothing."""
    b = Batch(((5, 2), (1, 0), (40, 3), (70, 0), (200, 4)), 4, 2, 64, 16, spare=1)
    for bounds in (None, PROMPTS):
        got, lse = b.run(bounds)
        seen = [3, 4, 43, 44, 45, 312, 313, 314, 315]
        for row in range(316):
            if row in seen:
                assert np.isfinite(got[row]).all() and np.isfinite(lse[row]).all() and np.abs(got[row]).max() > 0
            else:
                assert (got[row] == 0).all() and np.isneginf(lse[row]).all()


@pytest.mark.parametrize("q_len", [1, 40, 300])
def test_pages_outside_the_cache(q_len):
    """They are read as zeros: as if these positions held zeros."""
    b = Batch(((q_len, q_len + 20), (q_len, q_len + 40)), 4, 2, 128, 16)
    page = b.table[0, 1]
    b.table[0, 1] = 1 << 20
    b.table[1, 2] = -7
    bounds = PROMPTS if q_len == 300 else None
    got, _ = b.run(bounds)
    assert np.isfinite(got).all()
    for i, s in ((page, 0),):
        for v in b.values:
            v[i] = 0
    b.table[0, 1] = page
    b.pools = [p.copy() for p in b.pools]
    for p in b.pools:
        p[page] = 0
    want, _ = b.run(bounds)
    rows = slice(0, q_len)
    assert np.array_equal(got[rows], want[rows])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_large_and_small_queries(dtype):
    """bf16 queries go into fp16 by a power of two of their row: far outside fp16's range, and rows of zeros."""
    b = Batch(((1, 100), (1, 100), (1, 100), (1, 100)), 4, 2, 128, 16, dtype)
    size = [1e30, 1e-30, 0.0, 1.0] if dtype == "bf16" else [1e3, 1e-4, 0.0, 1.0]
    q = b.q.float()
    for i, x in enumerate(size):
        q[i] = q[i] * x
    b.q = q.to(b.dtype)
    got, _ = b.run(scale=1e-3)
    assert np.isfinite(got).all()
    want, _, tol, _ = b.want(scale=1e-3)
    rows = [1, 2, 3] if dtype == "bf16" else [0, 1, 2, 3]
    assert (np.abs(got[rows] - want[rows]) <= tol[rows]).all()
    if dtype == "bf16":  # scores of 1e27: one key takes all, if no two are alike
        assert (np.abs(got[0] - want[0]) <= 2.0 ** -8 * np.abs(want[0]) + 1e-6).all()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("how", [dict(scale=1e-3), dict(scale=1e-3, softcap=30.0), dict(scale=1e-3, slopes=[0.5, 0.25, 0.01, 1.0])])
def test_large_and_small_queries_of_prompts(dim, how):
    """The same where the cache is brought to fp16 for a prompt: each row by its own power of two, 2^-64 the least."""
    b = Batch(((300, 400), (1, 40)), 4, 2, dim, 16, "bf16")
    q = b.q.float()
    size = torch.tensor([1.0, 1e-38, 2.0 ** -70, 1e-8, 0.0, 1e3, 1.5])
    q = q * size.to(q.device)[torch.arange(q.shape[0], device=q.device) % 7, None]
    b.q = q.to(b.dtype)
    assert 0 < b.plan(PROMPTS).expand_from <= 600
    got, _ = b.run(PROMPTS, **how)
    want, _, tol, _ = b.want(**how)
    assert (np.abs(got - want) <= tol).all()


def test_no_row_depends_on_another():
    """A query's output is the same bits whatever else is in the batch, tile or wave."""
    lens = ((1, 77), (3, 90), (1, 500), (2, 10))
    whole = Batch(lens, 8, 2, 128, 16)
    plan = whole.plan()
    got, _ = whole.run()
    for s, (ql, kl) in enumerate(lens):
        one = Batch(lens, 8, 2, 128, 16)
        one.lens = (lens[s],)
        one.table = whole.table[s:s + 1].copy()
        one.q = whole.q[whole.starts[s]:whole.starts[s + 1]].clone()
        one.rows, one.starts, one.kv = ql, np.array([0, ql], np.int32), whole.kv[s:s + 1]
        assert plan.shares == one.plan(whole.bounds()).shares == 0 and plan.waves == one.plan(whole.bounds()).waves
        alone, _ = one.run(bounds=whole.bounds())
        assert np.array_equal(alone, got[whole.starts[s]:whole.starts[s + 1]])


@pytest.mark.parametrize("lens", [((1, 3000), (1, 20)), ((100, 200), (1, 900), (0, 3)), ((200, 300),)])
def test_streams_workspaces_and_graphs(lens):
    b = Batch(lens, 8, 1, 128, 16, "bf16", spare=1)
    mq, mk = PROMPTS if max(q for q, _ in lens) >= 100 else b.bounds()
    want, _ = b.run((mq, mk))
    d = b.dev

    def call(out, ws=None):
        return ttq.ttq_packed_attention(d["q"], d["k"], d["v"], d["table"], d["starts"], d["kv"], mq, mk, out=out, workspace=ws)

    c = _capi.ttq_packed_cache(1 << 20, 1 << 20, len(b.pools[0]), b.pools[0][0].size, b.kvh, b.page, b.dim, _capi.TTQ_BF16)
    bb = _capi.ttq_paged_batch(1 << 20, 1 << 20, 1 << 20, b.table.shape[1], b.table.shape[1], len(lens), b.rows, mq, mk)
    a = _capi.ttq_attention(b.heads, 0.1, 0.0, 0, None, None)
    need = ttq.load().ttq_packed_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(bb), ctypes.byref(a))
    assert need > 0
    stream = torch.cuda.Stream()
    out = torch.full((b.rows, 8 * 128), 77.0, dtype=b.dtype, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        call(out)
    stream.synchronize()
    assert np.array_equal(out.double().cpu().numpy(), want)
    # a workspace full of anything, one that is too small, and a graph replayed among other work
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    out.fill_(77.0)
    call(out, ws)
    assert np.array_equal(out.double().cpu().numpy(), want)
    with pytest.raises(ttq.TTQError):
        call(out, ws[:need - 1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out, ws)
    for i in range(3):
        out.fill_(77.0)
        ws.fill_(i)
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(out.double().cpu().numpy(), want)


def test_pages_far_into_a_pool():
    """Offsets pass 32 bits, in the pages and in the workspace's."""
    pages, stride = 70, 1 << 26
    b = Batch(((1, 40), (400, 400)), 4, 2, 128, 16, extra_pages=0)
    assert b.plan(PROMPTS).expand_from > 0
    want, _ = b.run(PROMPTS)
    pools = [torch.zeros(pages * stride, dtype=torch.uint8, device="cuda") for _ in range(2)]
    far = [p.as_strided((pages, 2, 16, 80), (stride, 16 * 80, 80, 1)) for p in pools]
    n = len(b.pools[0])
    for f, p in zip(far, b.pools):
        f[pages - n:] = torch.from_numpy(p).cuda()
    d = b.on_gpu()
    table = torch.where(d["table"] >= 0, d["table"] + (pages - n), d["table"])
    got = ttq.ttq_packed_attention(d["q"], far[0], far[1], table, d["starts"], d["kv"], *PROMPTS)
    assert np.array_equal(got.double().cpu().numpy(), want)


def test_cache_of_a_model():
    """PagedCache(bits=4): rotated appends in chunks, forked, then attention as over what was appended."""
    torch.manual_seed(0)
    cache = ttq.PagedCache(1, 64, 2, 64, page_size=16, bits=4)
    table = ttq.rotation_table(200, 64)
    rows = torch.randn((90, (8 + 4) * 64), device="cuda").half()
    q, k, v = rows.split([512, 128, 128], 1)
    out = []
    for at, n in ((0, 50), (50, 37), (87, 1)):
        cache.extend("a", n)
        b = cache.batch(["a"], [n])
        x = cache.append(0, q[at:at + n], k[at:at + n], v[at:at + n], b, table)
        out.append(cache.attend(0, x, b))
    cache.fork("a", ["b", "c"])
    cache.extend("b", 1)
    cache.extend("c", 1)
    b = cache.batch(["b", "c"], [1, 1])
    x = cache.append(0, q[88:], k[88:], v[88:], b, table)
    out.append(cache.attend(0, x, b))
    out = torch.cat(out).double().cpu().numpy().reshape(90, 8, 64)
    # the same in 64 bits
    t = table.cpu().numpy()
    pos = np.array(list(range(88)) + [88, 88])
    rot = [ref.rotated(x.float().cpu().numpy().reshape(90, -1, 64), t, pos, False) for x in (q, k)]
    Q = torch.from_numpy(rot[0]).half().double().numpy()
    K, V = ref.held(rot[1]), ref.held(v.float().cpu().numpy().reshape(90, 2, 64))
    want = np.empty_like(out)
    for i in range(90):
        seen = list(range(i + 1)) if i < 88 else list(range(88)) + [i]
        for h in range(8):
            z = K[seen, h // 4] @ Q[i, h] / 8
            p = np.exp(z - z.max())
            want[i, h] = p @ V[seen, h // 4] / p.sum()
    assert np.linalg.norm(out - want) <= 3 * 2.0 ** -11 * np.linalg.norm(want)


def test_refused_tensors():
    b = Batch(((1, 20),), 4, 2, 128, 16)
    d = b.on_gpu()

    def call(**kw):
        a = dict(Q=d["q"], kcache=d["k"], vcache=d["v"], block_table=d["table"], q_start=d["starts"], kv_len=d["kv"],
                 max_q_len=1, max_kv_len=20)
        a.update(kw)
        return ttq.ttq_packed_attention(**a)

    call()
    for bad, kind in ((dict(Q=d["q"].float()), TypeError), (dict(kcache=d["k"].char()), TypeError),
                      (dict(kcache=d["k"][..., :75], vcache=d["v"][..., :75]), ValueError), (dict(vcache=d["v"][:1]), ValueError),
                      (dict(Q=d["q"][:, :400]), ValueError), (dict(Q=d["q"][:, :128]), ttq.TTQError),
                      (dict(scale=-1.0), ttq.TTQError), (dict(window=-1), ttq.TTQError), (dict(out=d["q"].bfloat16()), TypeError),
                      (dict(lse=torch.empty((1, 3), device="cuda")), ValueError), (dict(max_q_len=-1), ttq.TTQError)):
        with pytest.raises(kind):
            call(**bad)
