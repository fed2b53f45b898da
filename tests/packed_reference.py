"""The 4-bit cache and the rotation, plainly: numpy on the CPU, one value after
the other where that says it best.  What the tests hold the kernels to."""
import numpy as np

ORDER = (0, 2, 4, 6, 1, 3, 5, 7)  # channel of each slot of a word
GROUP = 32


def codes_of(x):
    """x [..., 32 n] fp32 -> codes, scale, lo, as the definition has them in 32 bits."""
    with np.errstate(all="ignore"):
        x = np.where(np.isnan(x), np.float32(0), np.clip(x, np.float32(-32768), np.float32(32768))).astype(np.float32)
        g = x.reshape(*x.shape[:-1], -1, GROUP)
        least, most = g.min(-1), g.max(-1)
        lo = least.astype(np.float16)
        scale = ((most - least) / np.float32(15)).astype(np.float16)
        q = (g - lo.astype(np.float32)[..., None]) / scale.astype(np.float32)[..., None]
        q = np.where(scale[..., None] > 0, q, np.float32(0))
        codes = np.clip(np.rint(q), 0, 15).astype(np.uint32)
    return codes, scale, lo


def held(x):
    """What the cache holds for x, in 64 bits."""
    codes, scale, lo = codes_of(np.asarray(x, np.float32))
    return (codes * scale.astype(np.float64)[..., None] + lo.astype(np.float64)[..., None]).reshape(x.shape)


def places(dim, t, keys):
    """(byte of each 8-channel word, byte of each group's scale, bytes from a scale to its lo) of token t in a head's page."""
    c = min(dim, 128)
    words, scales = [], []
    for v in range(dim // 8):
        base = (t // 16 * (dim // c) + v // (c // 8)) * 10 * c
        u, w = t % 16, v % (c // 8)
        at = u * (c // 8) + w % 4 * (c // 32) + w // 4 if keys else (u // 4 * (c // 8) + w) * 4 + u % 4
        words.append(base + 4 * at)
        if v % 4 == 0:
            scales.append(base + 8 * c + ((u * (c // 32) + w // 4) * 4 if keys else
                                          (u // 4 * (c // 32) + w // 4) * 16 + u % 4 * 2))
    return words, scales, 2 if keys else 8


def put(page, t, x, keys):
    """Row x [dim] fp32 as token t of one head's page (bytes, flat), in place."""
    codes, scale, lo = codes_of(np.asarray(x, np.float32))
    codes = codes.reshape(-1, 8)
    words, scales, apart = places(len(x), t, keys)
    for c, at in zip(codes, words):
        w = 0
        for slot, channel in enumerate(ORDER):
            w |= int(c[channel]) << (4 * slot)
        page[at:at + 4] = np.array([w], np.uint32).view(np.uint8)
    for s, l, at in zip(scale.reshape(-1), lo.reshape(-1), scales):
        page[at:at + 2] = np.array([s]).view(np.uint8)
        page[at + apart:at + apart + 2] = np.array([l]).view(np.uint8)


def get(page, t, dim, keys):
    """Token t of one head's page (bytes, flat), in 64 bits."""
    words, scales, apart = places(dim, t, keys)
    out = np.empty(dim)
    for v, at in enumerate(words):
        w = int(page[at:at + 4].copy().view(np.uint32)[0])
        s = scales[v // 4]
        scale, lo = (float(page[i:i + 2].copy().view(np.float16)[0]) for i in (s, s + apart))
        for slot, channel in enumerate(ORDER):
            out[8 * v + channel] = scale * (w >> (4 * slot) & 15) + lo
    return out


def fill(pages, keys, rng, spread=1.0):
    """Random rows in every place of pages [n][kv heads][page size][5/8 dim] (uint8), quickly; returns their values, 64 bits."""
    n, kvh, size, row = pages.shape
    dim = row * 8 // 5
    x = (rng.standard_normal((n, kvh, size, dim)) * spread).astype(np.float32)
    codes, scale, lo = codes_of(x)
    words = np.zeros((n, kvh, size, dim // 8), np.uint32)
    c8 = codes.reshape(n, kvh, size, dim // 8, 8)
    for slot, channel in enumerate(ORDER):
        words |= c8[..., channel] << np.uint32(4 * slot)
    flat = pages.reshape(n, kvh, size * row)
    for t in range(size):
        at, scales, apart = places(dim, t, keys)
        for v, i in enumerate(at):
            flat[:, :, i:i + 4] = np.ascontiguousarray(words[:, :, t, v]).view(np.uint8).reshape(n, kvh, 4)
        for g, i in enumerate(scales):
            flat[:, :, i:i + 2] = np.ascontiguousarray(scale[:, :, t, g]).view(np.uint8).reshape(n, kvh, 2)
            flat[:, :, i + apart:i + apart + 2] = np.ascontiguousarray(lo[:, :, t, g]).view(np.uint8).reshape(n, kvh, 2)
    return (codes * scale.astype(np.float64)[..., None] + lo.astype(np.float64)[..., None]).reshape(x.shape)


def rotated(x, table, positions, interleaved):
    """x [tokens][heads][dim] turned by rows `positions` of the table, every product and sum rounded by itself in
    table.dtype (fp32: the kernels' bits; fp64: the formula)."""
    half = table.shape[1] // 2
    x = x.astype(table.dtype).copy()
    c, s = table[positions][:, None, :half], table[positions][:, None, half:]
    first = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    second = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    with np.errstate(all="ignore"):
        a, b = x[..., first].copy(), x[..., second].copy()
        x[..., first] = a * c - b * s
        x[..., second] = b * c + a * s
    return x
