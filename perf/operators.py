"""The serving operators next to the quantised projections, as cases to run.

Four operators take a layer's projected queries, keys and values to an answer:

  write      new keys and values go to their places in a paged cache
  attention  a ragged batch of new tokens (prompt chunks and single decode
             tokens) attends over the paged cache, with capped scores, a bias
             by distance, a window and a prefix mask where the model has them
  copy       pages are copied inside the cache of several layers (fork of a
             sequence, compaction) and the block table is rewritten
  logprobs   log probabilities of given tokens under the logits, the entropy
             of each row, and its most likely alternatives

Each case is run in one of two ways, chosen by `own`: the plain form in
elementary torch operations in 32 bits, or the framework's own entry points.
`exact` computes the same in 64 bits, written apart from the plain form.

Sequence lengths belong to a case (they are drawn from its "lens" number), the
values, the order of the pages and the tokens to the seed.
"""
import math
import random

import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------
def _attention_case(seqs, q_lo, q_hi, kv_lo, kv_hi, heads, kv_heads, dim, page, dtype, lens, softcap=0.0,
                    window=0, slopes=False, prefix=0, fused=False):
    return {"op": "attention", "seqs": seqs, "q_lo": q_lo, "q_hi": q_hi, "kv_lo": kv_lo, "kv_hi": kv_hi,
            "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page, "dtype": dtype, "lens": lens,
            "softcap": softcap, "window": window, "slopes": slopes, "prefix": prefix, "fused": fused}


def _write_case(seqs, q_lo, q_hi, kv_lo, kv_hi, kv_heads, dim, page, dtype, lens):
    return {"op": "write", "seqs": seqs, "q_lo": q_lo, "q_hi": q_hi, "kv_lo": kv_lo, "kv_hi": kv_hi,
            "kv_heads": kv_heads, "dim": dim, "page": page, "dtype": dtype, "lens": lens}


def _copy_case(layers, pages, pairs, kv_heads, dim, page, dtype, remap):
    return {"op": "copy", "layers": layers, "pages": pages, "pairs": pairs, "kv_heads": kv_heads, "dim": dim,
            "page": page, "dtype": dtype, "remap": remap}


def _logprobs_case(rows, vocab, top, dtype):
    return {"op": "logprobs", "rows": rows, "vocab": vocab, "top": top, "dtype": dtype}


def listed():
    cases = {
        # one user's next token in a small model (12 heads of 64), a short context: latency is all
        "attention_decode_one": _attention_case(1, 1, 1, 333, 333, 12, 12, 64, 16, "f16", 1),
        # a decode step of a busy server: 64 users, contexts from a few tokens to 8192, 64 heads over 8
        "attention_decode_batch": _attention_case(64, 1, 1, 1, 8192, 64, 8, 128, 64, "f16", 2),
        # few users with very long documents: the work has to be split along the context
        "attention_decode_long": _attention_case(3, 1, 1, 65536, 131072, 32, 8, 128, 128, "bf16", 3),
        # a chunk of 4096 prompt tokens over a context that is 10000 tokens with it: bound by arithmetic;
        # the queries are a slice of the fused projection's output
        "attention_prompt_chunk": _attention_case(1, 4096, 4096, 10000, 10000, 64, 8, 128, 64, "f16", 4, fused=True),
        # prompts in chunks beside decoding users, heads of 256 with capped scores and a window
        "attention_mixed_capped": _attention_case(24, 1, 512, 1, 4096, 16, 8, 256, 32, "bf16", 5, softcap=50.0,
                                                  window=1024),
        # whole prompts of odd lengths whose prefix is seen from everywhere, bias by distance, a head each
        "attention_prefix_bias": _attention_case(5, 100, 1500, 0, 0, 16, 16, 64, 16, "f16", 6, slopes=True,
                                                 prefix=200),
        # the new keys and values of a decode step
        "write_step": _write_case(64, 1, 1, 1, 1024, 8, 128, 64, "f16", 7),
        # the keys and values of long prompts
        "write_prompt": _write_case(3, 2000, 9000, 2000, 16384, 8, 128, 64, "bf16", 8),
        # a sequence forked into 16 answers: its last, partly filled page for each of them, in every layer
        "copy_fork": _copy_case(16, 64, 16, 8, 128, 16, "f16", False),
        # a cache compacted: a third of its pages move, the tables follow
        "copy_compact": _copy_case(4, 2048, 700, 8, 128, 64, "bf16", True),
        # the sampled tokens of a decode step with a few alternatives, logits in 32 bits, an odd vocabulary
        "logprobs_step": _logprobs_case(7, 50257, 5, "f32"),
        # a prompt scored: each of its tokens, with entropy and alternatives
        "logprobs_prompt": _logprobs_case(2048, 151936, 20, "bf16"),
    }
    return [dict(c, name=n) for n, c in cases.items()]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "write", "copy", "logprobs", "logprobs"])
    lens = rng.randrange(1 << 30)
    if op == "attention":
        heads, kv_heads, dim = rng.choice([(12, 12, 64), (16, 16, 64), (16, 8, 128), (32, 8, 128), (64, 8, 128),
                                           (20, 4, 128), (16, 8, 256), (8, 1, 256)])
        page, dtype = rng.choice([16, 32, 64, 128, 256]), rng.choice(["f16", "bf16"])
        mods = dict(softcap=rng.choice([0.0, 0.0, 30.0, 50.0]), slopes=rng.random() < 0.25,
                    window=rng.choice([0, 0, _log(rng, 50, 4096)]), fused=rng.random() < 0.5)
        if rng.random() < 0.5:  # decoding
            seqs = _log(rng, 1, 128)
            most = max(64, min(131072, 300_000 // seqs))
            kv_hi = _log(rng, 16, most)
            return _attention_case(seqs, 1, 1, rng.choice([1, max(1, kv_hi // 2), kv_hi]), kv_hi, heads, kv_heads,
                                   dim, page, dtype, lens, **mods)
        q_hi = _log(rng, 2, 4096)
        seqs = _log(rng, 1, max(1, min(32, 6000 // q_hi)))
        kv_hi = q_hi + _log(rng, 1, 6000) if rng.random() < 0.7 else 0
        prefix = _log(rng, 1, q_hi) if rng.random() < 0.25 else 0
        return _attention_case(seqs, rng.choice([1, max(1, q_hi // 2), q_hi]), q_hi, kv_hi // 2, kv_hi, heads,
                               kv_heads, dim, page, dtype, lens, prefix=prefix, **mods)
    if op == "write":
        kv_heads, dim = rng.choice([(12, 64), (16, 64), (8, 128), (4, 128), (8, 256), (1, 256)])
        q_hi = rng.choice([1, _log(rng, 2, 8192)])
        seqs = _log(rng, 1, max(1, min(256, 16000 // q_hi)))
        return _write_case(seqs, rng.choice([1, max(1, q_hi // 2)]), q_hi, q_hi, q_hi + _log(rng, 1, 1024), kv_heads,
                           dim, rng.choice([16, 32, 64, 128, 256]), rng.choice(["f16", "bf16"]), lens)
    if op == "copy":
        kv_heads, dim = rng.choice([(12, 64), (8, 128), (4, 128), (1, 256)])
        layers, pages = _log(rng, 1, 12), _log(rng, 8, 2048)
        return _copy_case(layers, pages, _log(rng, 1, max(1, min(pages // 3, 2800 // layers))), kv_heads, dim,
                          rng.choice([16, 32, 64]), rng.choice(["f16", "bf16"]), rng.random() < 0.5)
    vocab = _log(rng, 500, 262144)
    dtype = rng.choice(["f16", "bf16", "f32"])
    rows = _log(rng, 1, max(1, min(16384, 150_000_000 // vocab)))
    return _logprobs_case(rows, vocab, rng.choice([0, 1, 5, 10, 20]), dtype)


def _lens(case):
    """(query lengths, key lengths, prefix lengths) of the case's sequences."""
    rng = random.Random(case["lens"])
    ql, kl, pl = [], [], []
    for _ in range(case["seqs"]):
        q = rng.randint(case["q_lo"], case["q_hi"])
        if case["q_hi"] > 1 and case["q_lo"] == 1 and rng.random() < 0.5:
            q = 1  # a decoding user in a batch with prompt chunks
        k = max(q, rng.randint(case["kv_lo"], case["kv_hi"]))
        ql.append(q)
        kl.append(k)
        pl.append(min(k, rng.randint(0, case.get("prefix", 0))))
    return ql, kl, pl


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _tables(case, kl, gen):
    """A block table [seqs][blocks] of pages in random order, -1 where a sequence has none, and the page count."""
    page = case["page"]
    need = [-(-k // page) for k in kl]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=gen).to(torch.int32)
    table = torch.full((len(kl), max(need)), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    return table, pages


def _starts(ql):
    out = [0]
    for q in ql:
        out.append(out[-1] + q)
    return out


def prepare(case, seed):
    gen = torch.Generator().manual_seed(seed)
    dev = torch.Generator("cuda").manual_seed(seed)
    dt = TYPES[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(shape, generator=dev, device="cuda", dtype=torch.float32) * scale).to(dtype)

    def cache(*shape):  # keys, values: filled in slices, so that no 32-bit copy of all of it is needed
        out = torch.empty(shape, dtype=dt, device="cuda")
        flat = out.view(-1)
        for i in range(0, flat.numel(), 1 << 26):
            flat[i:i + (1 << 26)] = normal(min(1 << 26, flat.numel() - i))
        return out

    s = {"case": dict(case)}
    if case["op"] in ("attention", "write"):
        ql, kl, pl = _lens(case)
        table, pages = _tables(case, kl, gen)
        kvh, dim, rows = case["kv_heads"], case["dim"], sum(ql)
        s.update(table=table.cuda(), q_start=torch.tensor(_starts(ql), dtype=torch.int32).cuda(),
                 kv_len=torch.tensor(kl, dtype=torch.int32).cuda(), max_q=max(ql), max_kv=max(kl),
                 kcache=cache(pages, kvh, case["page"], dim), vcache=cache(pages, kvh, case["page"], dim))
    if case["op"] == "attention":
        heads = case["heads"]
        if case["fused"]:  # the queries as they lie in the output of one projection to q, k and v
            s["q"] = normal(rows, (heads + 2 * kvh) * dim, scale=1.5)[:, :heads * dim]
        else:
            s["q"] = normal(rows, heads * dim, scale=1.5)
        s["slopes"] = None
        if case["slopes"]:  # a geometric row of slopes, one a head
            s["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / heads) for h in range(heads)],
                                       dtype=torch.float32).cuda()
        s["prefix"] = torch.tensor(pl, dtype=torch.int32).cuda() if case["prefix"] else None
        s["scale"] = dim ** -0.5
    elif case["op"] == "write":
        qkv = normal(rows, 2 * kvh * dim)  # keys and values as the projection leaves them
        s["k"], s["v"] = qkv[:, :kvh * dim], qkv[:, kvh * dim:]
    elif case["op"] == "copy":
        shape = (case["layers"], case["pages"], case["kv_heads"], case["page"], case["dim"])
        s["kcache"], s["vcache"] = cache(*shape), cache(*shape)
        order = torch.randperm(case["pages"], generator=gen).to(torch.int32)
        n = case["pairs"]
        s["src"], s["dst"] = order[:n].cuda(), order[n:2 * n].cuda()
        used = torch.cat([order[:n], order[2 * n:]])  # pages that the tables name, those that move among them
        pick = torch.randint(0, used.numel(), (32, max(1, case["pages"] // 32)), generator=gen)
        table = used[pick]
        table[torch.rand(table.shape, generator=gen) < 0.1] = -1
        s["table"] = table.cuda() if case["remap"] else None
    elif case["op"] == "logprobs":
        rows, vocab = case["rows"], case["vocab"]
        logits = torch.empty((rows, vocab), dtype=dt, device="cuda")
        step = max(1, (1 << 26) // vocab)
        for i in range(0, rows, step):
            n = min(step, rows - i)
            x = normal(n, vocab, scale=2.0, dtype=torch.float32)
            # a few tokens stand out of each row, as they do in a trained model
            hot = torch.randint(0, vocab, (n, 8), generator=dev, device="cuda")
            x.scatter_add_(1, hot, normal(n, 8, scale=6.0, dtype=torch.float32).abs())
            logits[i:i + n] = x.to(dt)
        s["logits"] = logits
        s["tokens"] = torch.randint(0, vocab, (rows,), generator=dev, device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    return RUN[s["case"]["op"]][bool(own)](s)


def _own_attention(s):
    import test_activation_aware_amd as ttq
    c = s["case"]
    return ttq.ttq_paged_attention(s["q"], s["kcache"], s["vcache"], s["table"], s["q_start"], s["kv_len"],
                                   max_q_len=s["max_q"], max_kv_len=s["max_kv"], scale=s["scale"],
                                   softcap=c["softcap"], window=c["window"], slopes=s["slopes"],
                                   prefix_len=s["prefix"])


def _own_write(s):
    import test_activation_aware_amd as ttq
    ttq.ttq_cache_write(s["k"], s["v"], s["kcache"], s["vcache"], s["table"], s["q_start"], s["kv_len"])
    return s["kcache"], s["vcache"]


def _own_copy(s):
    import test_activation_aware_amd as ttq
    ttq.ttq_cache_copy_pages(s["kcache"], s["vcache"], s["src"], s["dst"], table=s["table"])
    return s["kcache"], s["vcache"], s["table"]


def _own_logprobs(s):
    import test_activation_aware_amd as ttq
    return ttq.ttq_token_logprobs(s["logits"], s["tokens"], top=s["case"]["top"])


def _rows(s, n):
    """Sequence of each of the n new tokens, its place in the chunk, and its position in the sequence."""
    starts, row = s["q_start"].long(), torch.arange(n, device="cuda")
    seq = torch.searchsorted(starts, row, right=True) - 1
    inside = row - starts[seq]
    return seq, inside, s["kv_len"].long()[seq] - (starts[seq + 1] - starts[seq]) + inside


def _plain_attention(s):
    c, q = s["case"], s["q"]
    heads, kvh, dim, most = c["heads"], c["kv_heads"], c["dim"], s["max_q"]
    group, seqs = heads // kvh, c["seqs"]

    def gathered(pool):  # [seqs][kv heads][positions][dim], 32 bits
        x = pool[s["table"].clamp(min=0).long()].transpose(1, 2)
        return x.reshape(seqs, kvh, -1, dim)[:, :, :s["max_kv"]].float()

    keys, values = gathered(s["kcache"]), gathered(s["vcache"])
    starts, kv = s["q_start"].long(), s["kv_len"].long()
    at = (starts[:seqs, None] + torch.arange(most, device="cuda")).clamp(max=q.shape[0] - 1)
    x = q[at].float().reshape(seqs, most, kvh, group, dim).permute(0, 2, 3, 1, 4).reshape(seqs, kvh, -1, dim)
    scores = torch.matmul(x, keys.transpose(2, 3)).mul_(s["scale"])
    if c["softcap"]:
        scores.div_(c["softcap"]).tanh_().mul_(c["softcap"])
    scores = scores.reshape(seqs, kvh, group, most, -1)
    i = (kv - (starts[1:] - starts[:seqs]))[:, None] + torch.arange(most, device="cuda")  # position of each query
    i, j = i[:, :, None], torch.arange(scores.shape[-1], device="cuda")
    seen = j <= i
    if c["window"]:
        seen = seen & (i - j < c["window"])
    if s["prefix"] is not None:
        seen = seen | (j < s["prefix"][:, None, None])
    seen = (seen & (j < kv[:, None, None]))[:, None, None]
    if s["slopes"] is not None:
        scores = scores - s["slopes"].reshape(kvh, group, 1, 1) * (i - j).abs().float()[:, None, None]
    scores = scores.masked_fill_(~seen, -math.inf)
    scores = scores.sub_(scores.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    total = scores.sum(-1, keepdim=True)
    out = torch.matmul(scores.reshape(seqs, kvh, group * most, -1), values)
    out = out.reshape(seqs, kvh, group, most, dim) / total.clamp(min=1e-30)
    seq, inside, _ = _rows(s, q.shape[0])
    return out.permute(0, 3, 1, 2, 4)[seq, inside].reshape(q.shape[0], heads * dim).to(q.dtype)


def _plain_write(s):
    c, k, v = s["case"], s["k"], s["v"]
    seq, _, pos = _rows(s, k.shape[0])
    page, slot = s["table"].long()[seq, pos // c["page"]], pos % c["page"]
    s["kcache"][page, :, slot] = k.reshape(-1, c["kv_heads"], c["dim"])
    s["vcache"][page, :, slot] = v.reshape(-1, c["kv_heads"], c["dim"])
    return s["kcache"], s["vcache"]


def _plain_copy(s):
    src, dst, table = s["src"].long(), s["dst"].long(), s["table"]
    s["kcache"][:, dst] = s["kcache"][:, src]
    s["vcache"][:, dst] = s["vcache"][:, src]
    if table is not None:
        to = torch.arange(s["case"]["pages"], device="cuda", dtype=torch.int32)
        to[src] = s["dst"]
        table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()], table))
    return s["kcache"], s["vcache"], table


def _plain_logprobs(s):
    x, top = s["logits"].float(), s["case"]["top"]
    most = x.amax(-1, keepdim=True)
    e = (x - most).exp()
    total = e.sum(-1, keepdim=True)
    lse = most + total.log()
    logprob = (x.gather(1, s["tokens"][:, None]) - lse)[:, 0]
    # sum p (lse - x) over the row; e = 0 where x is -inf
    entropy = torch.where(e > 0, (lse - x) * e, 0.0).sum(-1) / total[:, 0]
    if not top:
        return logprob, entropy
    # order by value, then by index: the value's bits as a whole number that grows with it, over the index
    bits = (x + 0.0).view(torch.int32)
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
    key = (order << 32) + (0xFFFFFFFF - torch.arange(x.shape[1], device="cuda"))
    ids = 0xFFFFFFFF - (key.topk(top, dim=1).values & 0xFFFFFFFF)
    return logprob, entropy, ids, x.gather(1, ids) - lse


RUN = {"attention": (_plain_attention, _own_attention), "write": (_plain_write, _own_write),
       "copy": (_plain_copy, _own_copy), "logprobs": (_plain_logprobs, _own_logprobs)}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def _size(case):
    return 4 if case["dtype"] == "f32" else 2


def work(case):
    b = _size(case)
    if case["op"] == "attention":
        ql, kl, pl = _lens(case)
        pairs = keys = 0
        for q, k, p in zip(ql, kl, pl):
            w, first = case["window"] or k, k - q
            lo = max(0, first - w + 1)  # keys that some query sees: the prefix, and from the first window on
            keys += max(0, k - max(lo, p)) + p
            for i in range(first, k):
                low = max(0, i - w + 1)
                pairs += p + max(0, i + 1 - max(low, p))
        token = case["kv_heads"] * case["dim"]
        return {"bytes": b * (2 * keys * token + 2 * sum(ql) * case["heads"] * case["dim"]),
                "flops": 4 * pairs * case["heads"] * case["dim"]}
    if case["op"] == "write":
        return {"bytes": 4 * b * sum(_lens(case)[0]) * case["kv_heads"] * case["dim"], "flops": 0}
    if case["op"] == "copy":
        return {"bytes": 4 * b * case["layers"] * case["pairs"] * case["kv_heads"] * case["page"] * case["dim"],
                "flops": 0}
    n = case["rows"] * case["vocab"]
    return {"bytes": n * b + case["rows"] * (16 + 12 * case["top"]), "flops": 5 * n}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "attention":
        return _exact_attention(case, prepare(case, seed))
    if case["op"] == "logprobs":
        return _exact_logprobs(case, prepare(case, seed))
    return None  # what is moved is not computed


def _exact_attention(case, s):
    ql, kl, pl = _lens(case)
    heads, kvh, dim = case["heads"], case["kv_heads"], case["dim"]
    group = heads // kvh
    out = torch.zeros((sum(ql), heads, dim), dtype=torch.float64, device="cuda")
    begin = 0
    for n, (q_len, k_len, prefix) in enumerate(zip(ql, kl, pl)):
        page = s["table"][n, :-(-k_len // case["page"])].long()
        key_pos = torch.arange(k_len, device="cuda")
        for h in range(kvh):
            K = s["kcache"][page, h].reshape(-1, dim)[:k_len].double()
            V = s["vcache"][page, h].reshape(-1, dim)[:k_len].double()
            for r in range(0, q_len, 1024):  # by blocks of queries: the scores of a block fit
                m = min(1024, q_len - r)
                rows = slice(begin + r, begin + r + m)
                pos = torch.arange(k_len - q_len + r, k_len - q_len + r + m, device="cuda")
                far = pos[:, None] - key_pos[None, :]
                hidden = far < 0
                if case["window"]:
                    hidden |= far >= case["window"]
                hidden &= (key_pos >= prefix)[None, :]
                for g in range(group):
                    head = h * group + g
                    Q = s["q"][rows, head * dim:(head + 1) * dim].double()
                    z = (Q @ K.T) / math.sqrt(dim)
                    if case["softcap"]:
                        z = case["softcap"] * torch.tanh(z / case["softcap"])
                    if case["slopes"]:
                        z = z - 2.0 ** (-8.0 * (head + 1) / heads) * far.abs()
                    z[hidden] = -math.inf
                    out[rows, head] = torch.softmax(z, dim=1) @ V
        begin += q_len
    return out.reshape(sum(ql), heads * dim)


def _exact_logprobs(case, s):
    top, got = case["top"], []
    step = max(1, (1 << 25) // case["vocab"])
    for r in range(0, case["rows"], step):
        x = s["logits"][r:r + step].double()
        logp = torch.log_softmax(x, dim=1)
        entropy = torch.special.entr(logp.exp()).sum(1)
        part = [logp.gather(1, s["tokens"][r:r + step, None])[:, 0], entropy]
        if top:
            ids = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :top]
            part += [ids, logp.gather(1, ids)]
        got.append(part)
    return tuple(torch.cat(p) for p in zip(*got))
