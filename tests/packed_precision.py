"""How far attention over the 4-bit cache may be off as a whole: from its roundings alone.

A rounding to a type whose neighbouring numbers lie eps apart (relative to the
power of two below the value) is off by a uniform error of at most half of that,
eps / sqrt(12) of the value or less in the mean square.  Keys, values and
probabilities are rounded to fp16 whatever the type of the rows, and outputs to
their own type.  Independent errors of the values and of the probabilities reach
the output as its own would (sum_j p_j v_j with independent factors of 1 +
error); those of the keys move a score by eps / sqrt(12) times n, n^2 = sum_c
(scale q_c k_c)^2, and a probability by as much of itself, less the mean of that
over the keys, which is another such error.  In all, of the output's norm,
  sqrt(r(own)^2 + r(fp16)^2 (2 + 2 n^2)),  r(t) = eps(t) / sqrt(12),
with n^2 averaged by the probabilities.  5 % are added: a mean square of 10^4
errors is within 1 % of what it is expected to be, and one in 32 bits adds
nothing that could be seen."""
import numpy as np
import torch


def rounded(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x)).to(dtype).double().numpy()


def attend(b, low=None, scale=None, softcap=0.0, window=0, slopes=None, prefix=None):
    """(outputs, n^2) of a Batch in 64 bits; with `low` its keys, values and probabilities are rounded to that type."""
    scale = b.dim ** -0.5 if scale is None else scale
    cut = (lambda x: x) if low is None else (lambda x: rounded(x, low))
    group, outs, noise, rows = b.heads // b.kvh, [], 0.0, 0
    for s, (ql, kl) in enumerate(b.lens):
        pages = b.table[s, :-(-kl // b.page)]
        x = b.q[b.starts[s]:b.starts[s + 1], :b.heads * b.dim].double().numpy().reshape(ql, b.heads, b.dim)
        out = np.zeros(x.shape)
        i, j = np.arange(kl - ql, kl)[:, None], np.arange(kl)[None, :]
        seen = (j <= i) & ((i - j < window) if window else True)
        if prefix is not None:
            seen |= j < prefix[s]
        live = seen.any(1)
        for h in range(b.heads):
            if not live.any():
                continue
            k, v = (cut(c[pages][:, h // group].reshape(-1, b.dim)[:kl]) for c in b.values)
            z = scale * (x[live, h] @ k.T)
            if softcap:
                z = softcap * np.tanh(z / softcap)
            if slopes is not None:
                z = z - slopes[h] * np.abs(i - j)[live]
            z = np.where(seen[live], z, -np.inf)
            e = np.exp(z - z.max(1, keepdims=True))
            total = e.sum(1, keepdims=True)
            out[live, h] = cut(e) @ v / total
            noise += float((e / total * (scale ** 2 * (x[live, h] ** 2 @ (k ** 2).T))).sum())
            rows += int(live.sum())
        outs.append(out.reshape(ql, b.heads * b.dim))
    return np.concatenate(outs), noise / max(rows, 1)


def bound(dtype, noise):
    r = {t: torch.finfo(t).eps / 12 ** 0.5 for t in (torch.float16, torch.bfloat16)}
    return 1.05 * (r[dtype] ** 2 + r[torch.float16] ** 2 * (2 + 2 * noise)) ** 0.5


def off(got, want):
    return np.linalg.norm(got - want) / np.linalg.norm(want)
