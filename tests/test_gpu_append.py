"""Rotated appends into the 16-bit and the 4-bit cache, against plain numpy.

The rotation is defined by single roundings in fp32, so that every bit of what
the kernels leave can be told: rotated queries, 16-bit pages and the bytes of
4-bit pages are compared for equality, and everything that no token owns for
being as it was.  The formula itself, in 64 bits, is checked apart from that."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
import packed_reference as ref  # noqa: E402
import test_activation_aware_amd as ttq  # noqa: E402

pytestmark = pytest.mark.gpu
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


class Case:
    """A ragged batch, q_len new tokens of kv_len positions each, pages in random order."""

    def __init__(self, dim=128, heads=4, kv_heads=2, page=16, dtype="f16", lens=((1, 1), (3, 20), (0, 7), (40, 40)),
                 rotated=None, spare=0, packed=True, seed=0, positions=32768, base=10000.0):
        self.dim, self.heads, self.kvh, self.page, self.packed = dim, heads, kv_heads, page, packed
        self.dtype = TYPES[dtype]
        g = torch.Generator().manual_seed(seed)
        self.lens = lens
        need = [-(-k // page) for _, k in lens]
        pages = sum(need) + 2
        order = torch.randperm(pages, generator=g).int()
        self.table = torch.full((len(lens), max(need + [1])), -1, dtype=torch.int32)
        at = 0
        for i, n in enumerate(need):
            self.table[i, :n] = order[at:at + n]
            at += n
        self.rows = sum(q for q, _ in lens) + spare
        starts = np.cumsum([0] + [q for q, _ in lens])
        self.q_start = torch.tensor(starts, dtype=torch.int32)
        self.kv_len = torch.tensor([k for _, k in lens], dtype=torch.int32)
        # queries, keys and values as they lie in the output of one projection
        qkv = torch.randn((self.rows, (heads + 2 * kv_heads) * dim), generator=g).to(self.dtype)
        self.qkv = qkv
        if packed:
            self.k, self.v = (torch.randint(0, 256, (pages, kv_heads, page, dim * 5 // 8), generator=g,
                                            dtype=torch.uint8) for _ in range(2))
        else:
            self.k, self.v = (torch.randn((pages, kv_heads, page, dim), generator=g).to(self.dtype) for _ in range(2))
        r = dim if rotated is None else rotated
        self.rotation = ttq.rotation_table(positions, r, base=base, device="cpu") if r else None
        self.token_seq = [i for i, (q, _) in enumerate(lens) for _ in range(q)]
        self.token_pos = [k - q + j for q, k in lens for j in range(q)]

    def split(self, x):
        return x.split([self.heads * self.dim, self.kvh * self.dim, self.kvh * self.dim], 1)

    def run(self, positions=None, interleaved=False, queries=True, out=None, device="cuda"):
        d = {n: getattr(self, n).to(device) for n in ("qkv", "k", "v", "table", "q_start", "kv_len")}
        rot = None if self.rotation is None else self.rotation.to(device)
        pos = None if positions is None else torch.tensor(positions, dtype=torch.int32, device=device)
        q, k, v = self.split(d["qkv"])
        f = ttq.ttq_packed_append if self.packed else ttq.ttq_cache_append
        if out is not None:
            out = out.to(device)
        got = f(q if queries else None, k, v, d["k"], d["v"], d["table"], d["q_start"], d["kv_len"], rot, pos,
                interleaved, out)
        torch.cuda.synchronize()
        return got, d["k"].cpu(), d["v"].cpu(), d

    def want(self, positions=None, interleaved=False, place=lambda i, p: True):
        """(rotated Q, k pages, v pages); rows of Q that no token owns are left out."""
        n = len(self.token_pos)
        q, k, v = (x[:n].float().numpy().reshape(n, -1, self.dim) for x in self.split(self.qkv))
        table = None if self.rotation is None else self.rotation.numpy()
        pos = np.array(self.token_pos if positions is None else positions[:n])
        live = np.ones(n, bool) if table is None else (pos >= 0) & (pos < len(table))
        if table is not None:
            q, k = (ref.rotated(x, table, np.where(live, pos, 0), interleaved) for x in (q, k))
        kp, vp = self.k.clone(), self.v.clone()
        for i in range(n):
            s, p = self.token_seq[i], self.token_pos[i]
            if not live[i] or not place(s, p):
                continue
            page = int(self.table[s, p // self.page])
            for h in range(self.kvh):
                if self.packed:
                    ref.put(kp[page, h].numpy().reshape(-1), p % self.page, k[i, h], True)
                    ref.put(vp[page, h].numpy().reshape(-1), p % self.page, v[i, h], False)
                else:
                    kp[page, h, p % self.page] = torch.from_numpy(k[i, h]).to(self.dtype)
                    vp[page, h, p % self.page] = torch.from_numpy(v[i, h]).to(self.dtype)
        return torch.from_numpy(q.reshape(n, -1)).to(self.dtype), live, kp, vp

    def check(self, place=lambda i, p: True, **how):
        wide = {k: v for k, v in how.items() if k in ("positions", "interleaved")}
        got, k, v, _ = self.run(**how)
        q, live, kp, vp = self.want(place=place, **wide)
        if how.get("queries", True):
            assert same(got.cpu()[:len(q)][live], q[live])
        assert same(k, kp)
        assert same(v, vp)


def same(a, b):
    """Bit for bit, but for the sign and payload of NaN."""
    if a.dtype == torch.uint8:
        return torch.equal(a, b)
    return bool(((a == b) | (a.isnan() & b.isnan())).all())


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dim,heads,kv_heads,page,rotated,interleaved", [
    (64, 3, 1, 16, 64, False), (64, 12, 12, 32, 32, False), (64, 2, 2, 16, 16, True),
    (128, 4, 2, 16, 128, False), (128, 64, 8, 64, 128, False), (128, 20, 4, 32, 48, False), (128, 1, 1, 128, 128, True),
    (256, 16, 8, 16, 256, False), (256, 2, 1, 256, 64, True), (256, 1, 1, 16, 208, False),
    (128, 5, 2, 16, 0, False),
])
def test_every_layout(packed, dtype, dim, heads, kv_heads, page, rotated, interleaved):
    Case(dim, heads, kv_heads, page, dtype, rotated=rotated, packed=packed, spare=3).check(interleaved=interleaved)


@pytest.mark.parametrize("packed", [False, True])
def test_many_tokens_one_workgroup_each(packed):
    """More than 1024 tokens: all rounds of heads in one workgroup."""
    c = Case(64, 20, 20, 16, "bf16", ((700, 900), (400, 400)), packed=packed)
    assert (len(c.token_pos) * 2 > 1024)
    c.check()


@pytest.mark.parametrize("packed", [False, True])
def test_many_sequences(packed):
    lens = [(i % 3, i % 3 + i % 50) for i in range(200)]
    Case(128, 2, 1, 16, "f16", lens, packed=packed).check()


@pytest.mark.parametrize("packed", [False, True])
def test_given_positions(packed):
    c = Case(packed=packed, positions=50)
    n = len(c.token_pos)
    rows = [(7 * i) % 50 for i in range(n)]
    rows[2], rows[5], rows[n - 1] = -1, 50, 1 << 30  # rows that the table does not have: skipped whole
    c.check(positions=rows)


@pytest.mark.parametrize("packed", [False, True])
def test_positions_past_the_table_are_skipped(packed):
    Case(packed=packed, positions=19).check()


@pytest.mark.parametrize("packed", [False, True])
def test_without_queries_and_in_place(packed):
    c = Case(packed=packed)
    c.check(queries=False)
    q, live, kp, vp = c.want()
    d = {n: getattr(c, n).cuda() for n in ("qkv", "k", "v", "table", "q_start", "kv_len")}
    rot = c.rotation.cuda()
    x, k, v = c.split(d["qkv"])
    f = ttq.ttq_packed_append if packed else ttq.ttq_cache_append
    got = f(x, k, v, d["k"], d["v"], d["table"], d["q_start"], d["kv_len"], rot, out=x)
    assert got is x
    assert same(x.cpu(), q) and same(d["k"].cpu(), kp)
    assert torch.equal(k.cpu(), c.split(c.qkv)[1])  # keys and values beside them are as they were


@pytest.mark.parametrize("packed", [False, True])
def test_rows_of_no_sequence_stay(packed):
    c = Case(packed=packed, spare=5)
    out = torch.full((c.rows, c.heads * c.dim + 8), 7.0, dtype=c.dtype)
    d = out.cuda()
    c.run(out=None)
    q, k, v = c.split(c.qkv.cuda())
    f = ttq.ttq_packed_append if packed else ttq.ttq_cache_append
    f(q, k, v, c.k.cuda(), c.v.cuda(), c.table.cuda(), c.q_start.cuda(), c.kv_len.cuda(), c.rotation.cuda(),
      out=d[:, :-8])
    d = d.cpu()
    assert bool((d[-5:] == 7).all()) and bool((d[:, -8:] == 7).all())
    assert same(d[:-5, :-8], c.want()[0])


@pytest.mark.parametrize("packed", [False, True])
def test_places_that_do_not_exist(packed):
    """Pages outside the cache, more positions than the table has columns, positions before 0: queries are rotated
    where the rotation has a row, nothing is written."""
    c = Case(packed=packed, lens=((4, 20), (3, 33), (5, 2)), positions=100)
    c.table[0, 1] = 1 << 20       # positions 16 to 19 of sequence 0
    c.table = c.table[:, :2].contiguous()  # position 32 of sequence 1
    c.check(place=lambda s, p: p >= 0 and not (s == 0 and p >= 16) and p < 32)


SPECIAL = [0.0, -0.0, 1e-8, 6e-8, 65504.0, -65504.0, float("inf"), float("-inf"), float("nan"), 32768.0, 1.0]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_values_at_the_ends(dtype):
    """Groups that are constant, tiny, huge, or hold infinities and NaN: finite, and by the definition."""
    c = Case(128, 1, 1, 16, dtype, ((16, 16),), rotated=0)
    x = c.qkv.clone()
    for i in range(16):
        x[i, :] = SPECIAL[i % len(SPECIAL)]
    x[11, ::3] = float("nan")
    x[12, ::5] = float("inf")
    x[13, ::2] = -65504.0 if dtype == "f16" else -3e38
    x[13, 1::2] = 65504.0 if dtype == "f16" else 3e38
    x[14] = torch.linspace(1.0, 1.01, x.shape[1]).to(c.dtype)
    c.qkv = x
    got, k, v, d = c.run()
    _, _, kp, vp = c.want()
    assert same(k, kp) and same(v, vp)
    kr, vr = ttq.ttq_packed_read(d["k"], d["v"], d["table"], d["q_start"], d["kv_len"], c.rows)
    assert bool(kr.isfinite().all()) and bool(vr.isfinite().all())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_read_back(dim, dtype):
    """What ttq_packed_read gives is the formula's value rounded once, and near what went in."""
    c = Case(dim, 2, 2, 32, dtype, ((1, 70), (30, 31), (0, 5), (3, 3)), spare=2)
    _, _, _, d = c.run()
    kr, vr = ttq.ttq_packed_read(d["k"], d["v"], d["table"], d["q_start"], d["kv_len"], c.rows, dtype=c.dtype)
    n = len(c.token_pos)
    kq, vq = (x[:n].float().numpy().reshape(n, -1, dim) for x in c.split(c.qkv)[1:])
    kq = ref.rotated(kq, c.rotation.numpy(), np.array(c.token_pos), False)
    half_step = torch.finfo(c.dtype).eps / 2
    for got, x in ((kr, kq), (vr, vq)):
        want = ref.held(x)
        got = got[:n].double().cpu().numpy().reshape(want.shape)
        # one rounding to the type, and one to 32 bits before it (the sum scale * code + lo)
        assert (np.abs(got - want) <= np.abs(want) * half_step * 1.001 + 1e-7).all()
        g = x.reshape(*x.shape[:-1], -1, 32)
        step = (g.max(-1) - g.min(-1)) / 15
        # half a step; the scale's own rounding over 15 steps and lo's, 2^-11 of each
        room = step * (0.5 + 15 * 2.0 ** -11) + np.abs(g).max(-1) * 2.0 ** -11 + 1e-6
        assert (np.abs(want.reshape(g.shape) - g) <= room[..., None]).all()


def test_the_formula_in_64_bits():
    """Rotated queries against the formula at far positions: the error of two products and a sum in fp32 (each half a
    step of 2^-23, relative to |a c| + |b s|), of the table's entries (the same), and of the rounding to the type."""
    c = Case(128, 8, 1, 16, "f16", ((64, 131072),), rotated=128, positions=131072)
    got = c.run()[0].double().cpu().numpy().reshape(64, 8, 128)
    x = c.split(c.qkv)[0].double().numpy().reshape(64, 8, 128)
    half = 64
    angle = np.array(c.token_pos)[:, None] * 10000.0 ** (-np.arange(half) / half)
    table = np.concatenate([np.cos(angle), np.sin(angle)], 1)
    want = ref.rotated(x, table, np.arange(64), False)
    size = np.abs(x[..., :64]) + np.abs(x[..., 64:])
    room = np.concatenate([size, size], -1) * 2.0 ** -24 * 5 + np.abs(want) * 2.0 ** -11 * 1.001 + 2.0 ** -25
    assert (np.abs(got - want) <= room).all()


@pytest.mark.parametrize("packed", [False, True])
def test_another_stream_and_a_graph(packed):
    c = Case(packed=packed)
    q, live, kp, vp = c.want()
    d = {n: getattr(c, n).cuda() for n in ("qkv", "k", "v", "table", "q_start", "kv_len")}
    rot = c.rotation.cuda()
    x, k, v = c.split(d["qkv"])
    f = ttq.ttq_packed_append if packed else ttq.ttq_cache_append
    fresh = {n: d[n].clone() for n in ("k", "v")}
    out = torch.empty((c.rows, c.heads * c.dim), dtype=c.dtype, device="cuda")
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        f(x, k, v, d["k"], d["v"], d["table"], d["q_start"], d["kv_len"], rot, out=out)
    stream.synchronize()
    assert same(out.cpu(), q) and same(d["k"].cpu(), kp) and same(d["v"].cpu(), vp)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f(x, k, v, d["k"], d["v"], d["table"], d["q_start"], d["kv_len"], rot, out=out)
    for _ in range(3):
        d["k"].copy_(fresh["k"])
        d["v"].copy_(fresh["v"])
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same(out.cpu(), q) and same(d["k"].cpu(), kp) and same(d["v"].cpu(), vp)


def test_pages_beyond_four_gigabytes():
    """Pages far apart and far into a pool: offsets pass 32 bits."""
    pages, stride = 70, 1 << 26
    c = Case(128, 2, 2, 16, "f16", ((2, 18), (16, 16)))
    size = 2 * 16 * 80
    pools = [torch.zeros(pages * stride, dtype=torch.uint8, device="cuda") for _ in range(2)]
    k, v = (p.as_strided((pages, 2, 16, 80), (stride, 16 * 80, 80, 1)) for p in pools)
    c.table[0, :2] = torch.tensor([69, 66], dtype=torch.int32)
    c.table[1, 0] = 68
    c.k, c.v = (torch.zeros((pages, 2, 16, 80), dtype=torch.uint8) for _ in range(2))
    _, _, kp, vp = c.want()
    x, kk, vv = c.split(c.qkv.cuda())
    ttq.ttq_packed_append(x, kk, vv, k, v, c.table.cuda(), c.q_start.cuda(), c.kv_len.cuda(), c.rotation.cuda())
    assert torch.equal(k.cpu(), kp) and torch.equal(v.cpu(), vp)
    assert int(pools[0].view(pages, stride)[:, size:].max()) == 0
    kr, _ = ttq.ttq_packed_read(k, v, c.table.cuda(), c.q_start.cuda(), c.kv_len.cuda(), c.rows)
    assert float(kr.abs().max()) > 1


def test_copies_of_packed_pages():
    """Fork and compaction of a 4-bit PagedCache keep what attention would read."""
    cache = ttq.PagedCache(2, 40, 2, 64, page_size=16, bits=4)
    g = torch.Generator().manual_seed(0)
    cache.extend("a", 37)
    b = cache.batch(["a"], [37])
    rows = [torch.randn((37, 128), generator=g).half().cuda() for _ in range(4)]
    for layer in range(2):
        cache.write(layer, rows[2 * layer], rows[2 * layer + 1], b)

    def read(seq, layer):
        b = cache.batch([seq], [cache.length(seq)])
        return ttq.ttq_packed_read(cache.k[layer], cache.v[layer], b["block_table"], b["q_start"], b["kv_len"], 37)

    want = [read("a", layer) for layer in range(2)]
    cache.fork("a", ["b", "c"])
    cache.free("a")
    cache.extend("b", 0)
    for seq in ("b", "c"):
        for layer in range(2):
            assert all(torch.equal(x, y) for x, y in zip(read(seq, layer), want[layer]))
    cache.free("b")
    assert cache.compact() > 0
    for layer in range(2):
        assert all(torch.equal(x, y) for x, y in zip(read("c", layer), want[layer]))


def test_refused_tensors():
    c = Case()
    d = {n: getattr(c, n).cuda() for n in ("qkv", "k", "v", "table", "q_start", "kv_len")}
    x, k, v = c.split(d["qkv"])
    rot = c.rotation.cuda()

    def call(**kw):
        a = dict(Q=x, K=k, V=v, kcache=d["k"], vcache=d["v"], block_table=d["table"], q_start=d["q_start"],
                 kv_len=d["kv_len"], rotation=rot)
        a.update(kw)
        return ttq.ttq_packed_append(**a)

    for bad, kind in ((dict(K=k.float()), TypeError), (dict(kcache=d["k"].char()), TypeError),
                      (dict(kcache=d["k"][..., :72]), ValueError), (dict(Q=x[:, :100]), ValueError),
                      (dict(Q=x[:-1]), ValueError), (dict(V=v.cpu()), ValueError), (dict(rotation=rot.double()), TypeError),
                      (dict(rotation=rot[:, :24]), ValueError), (dict(positions=d["kv_len"].long()), TypeError),
                      (dict(rotation=rot[:, :24].contiguous()), ttq.TTQError),
                      (dict(rotation=torch.ones((9, 144), device="cuda")), ttq.TTQError),
                      (dict(out=x[:, :128]), ValueError), (dict(Q=None, out=x), ValueError)):
        with pytest.raises(kind):
            call(**bad)
    with pytest.raises(TypeError):
        ttq.ttq_cache_append(x, k, v, d["k"], d["v"], d["table"], d["q_start"], d["kv_len"])
    with pytest.raises(TypeError):
        ttq.ttq_packed_read(d["k"], d["v"], d["table"], d["q_start"], d["kv_len"], c.rows, dtype=torch.float32)
