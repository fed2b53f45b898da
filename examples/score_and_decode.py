"""A prompt scored and continued by a small model with quantised projections.

One attention layer between an embedding and a head, random weights.  Its
projections are TTQLinear layers: the prompt quantises them, the decode steps
reuse that quantisation.  Between them stand the serving operators:

  1. the prompt's keys and values go to a PagedCache in chunks, each chunk
     attends over what is there (ttq_cache_write, ttq_paged_attention);
  2. the prompt is scored: the log probability of each next token, the mean
     entropy, the perplexity beside that of the same weights unquantised
     (ttq_token_logprobs);
  3. the sequence is forked into answers that start with the most likely
     alternatives and continue greedily, one token a step for all of them;
  4. all but the two best are freed, the cache is compacted, and these two
     continue.

    python examples/score_and_decode.py [--tokens 600] [--answers 4] [--steps 12]
"""
import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import test_activation_aware_amd as ttq  # noqa: E402


class Model:
    def __init__(self, dim=512, heads=8, kv_heads=2, head_dim=64, vocab=2048, max_tokens=4096, seed=0, q=4):
        g = torch.Generator().manual_seed(seed)

        def weight(n, m, scale):
            return (torch.randn((n, m), generator=g) * scale).half().cuda()

        self.q_cols, self.kv_cols = heads * head_dim, kv_heads * head_dim
        self.embed = weight(vocab, dim, 1.0)
        self.w = {"qkv": weight(self.q_cols + 2 * self.kv_cols, dim, dim ** -0.5),
                  "out": weight(dim, self.q_cols, self.q_cols ** -0.5), "head": weight(vocab, dim, 2.0 * dim ** -0.5)}
        self.proj = {n: ttq.TTQLinear(w, q=q, g=32, T_max=max_tokens) for n, w in self.w.items()}
        self.cache = ttq.PagedCache(1, max_tokens // 16, kv_heads, head_dim, page_size=16)
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim

    def split(self, qkv):
        return qkv[:, :self.q_cols], qkv[:, self.q_cols:self.q_cols + self.kv_cols], qkv[:, self.q_cols + self.kv_cols:]

    def attend(self, qkv, seqs, new):
        """The new tokens of seqs into the cache and over it."""
        for s, n in zip(seqs, new):
            self.cache.extend(s, n)
        batch = self.cache.batch(seqs, new)
        q, k, v = self.split(qkv)
        self.cache.write(0, k, v, batch)
        return self.cache.attend(0, q, batch)

    def prompt(self, seq, tokens, chunk=256):
        """Logits [T][vocab] of a prompt; quantises the projections for it."""
        x = self.embed[tokens]
        qkv = self.proj["qkv"].prefill(x)
        att = torch.cat([self.attend(qkv[i:i + chunk], [seq], [min(chunk, len(qkv) - i)])
                         for i in range(0, len(qkv), chunk)])
        return self.proj["head"].prefill(x + self.proj["out"].prefill(att))

    def step(self, seqs, tokens):
        """Logits of one more token of each sequence, with the prompt's quantisation."""
        x = self.embed[tokens]
        att = self.attend(self.proj["qkv"].linear(x), seqs, [1] * len(seqs))
        return self.proj["head"].linear(x + self.proj["out"].linear(att))

    def dense(self, tokens):
        """The same weights unquantised, in plain 32-bit torch: logits of a prompt."""
        x = self.embed[tokens].float()
        q, k, v = (t.unflatten(1, (-1, self.head_dim)).transpose(0, 1) for t in self.split(x @ self.w["qkv"].float().T))
        group = self.heads // self.kv_heads
        k, v = k.repeat_interleave(group, 0), v.repeat_interleave(group, 0)
        z = torch.matmul(q, k.transpose(1, 2).contiguous()) * self.head_dim ** -0.5
        z = z.masked_fill(torch.ones_like(z[0], dtype=torch.bool).triu(1), float("-inf"))
        att = torch.matmul(torch.softmax(z, -1), v.contiguous()).transpose(0, 1).flatten(1)
        return (x + att @ self.w["out"].float().T) @ self.w["head"].float().T


def run(tokens=600, answers=4, steps=12, seed=0, show=print):
    model = Model(seed=seed)
    g = torch.Generator().manual_seed(seed + 1)
    text = torch.randint(0, model.embed.shape[0], (tokens,), generator=g).cuda()

    logits = model.prompt("prompt", text)
    logprob, entropy = ttq.ttq_token_logprobs(logits[:-1], text[1:])
    dense_logprob, _ = ttq.ttq_token_logprobs(model.dense(text)[:-1], text[1:])
    perplexity, dense_perplexity = (float(torch.exp(-x.mean())) for x in (logprob, dense_logprob))
    show(f"prompt of {tokens} tokens: perplexity {perplexity:.1f} (unquantised {dense_perplexity:.1f}), "
         f"mean entropy {float(entropy.mean()):.2f}")

    _, _, ids, first = ttq.ttq_token_logprobs(logits[-1:], text[-1:], top=answers)
    names = [f"answer {i}" for i in range(answers)]
    model.cache.fork("prompt", names)
    model.cache.free("prompt")
    said = {n: [int(t)] for n, t in zip(names, ids[0])}
    score = {n: float(p) for n, p in zip(names, first[0])}

    def decode(names, count):
        for _ in range(count):
            now = torch.tensor([said[n][-1] for n in names], device="cuda")
            _, _, best, logp = ttq.ttq_token_logprobs(model.step(names, now), now, top=1)
            for n, t, p in zip(names, best[:, 0].tolist(), logp[:, 0].tolist()):
                said[n].append(t)
                score[n] += p

    decode(names, steps)
    kept = sorted(names, key=score.get, reverse=True)[:2]
    for n in names:
        if n not in kept:
            model.cache.free(n)
    moved = model.cache.compact()
    decode(kept, steps)
    for n in kept:
        show(f"{n}: log probability {score[n]:.2f}, tokens {said[n][:6]} ...")
    show(f"{moved} pages moved, {model.cache.free_pages} of {model.cache.pages} free")
    return {"perplexity": perplexity, "dense_perplexity": dense_perplexity, "said": said, "score": score, "kept": kept,
            "moved": moved, "text": text, "model": model}


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=600)
    ap.add_argument("--answers", type=int, default=4)
    ap.add_argument("--steps", type=int, default=12)
    a = ap.parse_args()
    run(a.tokens, a.answers, a.steps)
