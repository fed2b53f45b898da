"""A prompt continued by beams over a cache held in 4 bits.

The small model of score_and_decode.py with rotated queries and keys: the
projections quantise themselves on the prompt, and between them

  1. the prompt's chunks are rotated on their way into a PagedCache of 4 bits
     and attend over it (ttq_packed_append, ttq_packed_attention);
  2. the last token's logits give the first beams, each step the best
     continuations of all of them, with their histories (ttq_beam_select);
  3. the beams' pages follow their parents: full ones are shared, the last one is
     copied where several go on from one beam (PagedCache.reorder).

    python examples/beam_search.py [--tokens 300] [--beams 4] [--steps 24] [--bits 4]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

from score_and_decode import Model, ttq  # noqa: E402


class RotatedModel(Model):
    def __init__(self, bits=4, max_tokens=4096, **how):
        super().__init__(max_tokens=max_tokens, **how)
        self.cache = ttq.PagedCache(1, max_tokens // 16, self.kv_heads, self.head_dim, page_size=16, bits=bits)
        self.rotation = ttq.rotation_table(max_tokens, self.head_dim)

    def attend(self, qkv, seqs, new):
        """The new tokens of seqs, rotated by their positions, into the cache and over it."""
        for s, n in zip(seqs, new):
            self.cache.extend(s, n)
        batch = self.cache.batch(seqs, new)
        q = self.cache.append(0, *self.split(qkv), batch, self.rotation)
        return self.cache.attend(0, q, batch)


def run(tokens=300, beams=4, steps=24, bits=4, seed=0, show=print):
    model = RotatedModel(bits=bits, seed=seed)
    g = torch.Generator().manual_seed(seed + 1)
    text = torch.randint(0, model.embed.shape[0], (tokens,), generator=g).cuda()
    first = model.prompt("prompt", text)[-1:]
    held = 2 * model.cache.k[0, 0].numel() * model.cache.k.element_size() / 16
    show(f"prompt of {tokens} tokens, {held:.0f} bytes of keys and values a token")

    names = [f"beam {i}" for i in range(beams)]
    # one beam, the prompt, before the first token
    scores, parents, now, history = ttq.ttq_beam_select(
        first, torch.zeros((1, 1), device="cuda"), beams, torch.empty((1, 0), dtype=torch.int64, device="cuda"))
    model.cache.fork("prompt", ["kept"])
    model.cache.reorder(["prompt"], parents[0].tolist(), names=names)
    for _ in range(steps - 1):
        logits = model.step(names, now[0])
        scores, parents, now, history = ttq.ttq_beam_select(logits, scores, beams, history)
        model.cache.reorder(names, parents[0].tolist())
    for n, s, h in zip(names, scores[0].tolist(), history.tolist()):
        show(f"{n}: log probability {s:.2f}, tokens {h[:8]} ...")
    shared = sum(len(model.cache.pages_of(n)) for n in names) - len({p for n in names for p in model.cache.pages_of(n)})
    show(f"{model.cache.pages - model.cache.free_pages} pages in use, {shared} times shared")
    return {"model": model, "first": first, "scores": scores[0], "history": history, "names": names, "shared": shared}


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=300)
    ap.add_argument("--beams", type=int, default=4)
    ap.add_argument("--steps", type=int, default=24)
    ap.add_argument("--bits", type=int, default=4)
    a = ap.parse_args()
    run(a.tokens, a.beams, a.steps, a.bits)
