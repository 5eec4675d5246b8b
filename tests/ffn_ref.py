"""Plain 64-bit forms of the 8-bit operators of the feed-forward sublayer and the head, written from their definitions, with the
bounds that the tests hold the kernels to.

Bounds. U = 2^-24 is half a step of fp32. A rounding to bf16 is off by at most 2^-8 of the value, one to e4m3 by at most 2^-4 of it or
half a subnormal step, 2^-10.
  product: the products of codes are exact in fp32. The tensor cores add up 128 of them in fp32: each addition is taken to be off by
    at most a whole step of the largest sum met, 2 U sum |x w|. The product of two scales (1 U), its FMA (1 U) and the additions of
    blocks and of a cluster's parts (one U each, of the sums' magnitude) follow.
  norm: d squares are added up in any order (d U relative at most, half of it in the root), a few roundings beside.
  softmax sums: a thread adds up at most vocab / 256 + 64 terms one after the other; the joins add a few."""

import numpy as np

U = 2.0 ** -24
BF16 = 2.0 ** -8
BLOCK = 128


def e4m3_values():
    """The values of the 256 codes."""
    out = np.zeros(256)
    for c in range(256):
        e, m = c >> 3 & 15, c & 7
        v = m / 512 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[c] = np.nan if e == 15 and m == 7 else v
    out[128:] = -out[128:]
    return out


def blocks(n):
    return -(-n // BLOCK)


def half_step(q):
    """How far a rounding to e4m3 takes q."""
    return np.maximum(np.abs(q) * 2.0 ** -4, 2.0 ** -10)


def block_max(y):
    return np.stack([np.abs(y[:, i:i + BLOCK]).max(1) for i in range(0, y.shape[1], BLOCK)], 1)


def spread(scales, cols, rows=None):
    """A block's scale at each place: of a row's blocks, or with `rows` of 128 x 128 blocks."""
    out = np.repeat(scales, BLOCK, 1)[:, :cols]
    return out if rows is None else np.repeat(out, BLOCK, 0)[:rows]


def quantised(y):
    """(y / scale, scale) of rows in 64 bits: what the codes round."""
    s = np.maximum(block_max(y), 2.0 ** -64) / 448
    return y / spread(s, y.shape[1]), s


def norm(s, w, eps):
    return s / np.sqrt((s * s).mean(1, keepdims=True) + eps) * (1.0 if w is None else w)


def product(x, xs, w, ws):
    """(values, bound) of the product of rows of values-of-codes x with scales xs and weights w with scales ws."""
    k = x.shape[1]
    a, b = x * spread(xs, k), w * spread(ws, k, w.shape[0])
    out, mag = a @ b.T, np.abs(a) @ np.abs(b).T
    return out, (2 * BLOCK + blocks(k) + 16) * U * mag


def act(g, kind):
    if kind == "silu":
        return g / (1 + np.exp(-g))
    return g / 2 * (1 + np.tanh(np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)))


def gated(x, xs, wg, gs, wu, us, kind):
    """(values, bound). Both activations have slopes below 1.14; their fp32 forms are off by a few U of the result, and by 2 U
    of the exponent's argument."""
    g, eg = product(x, xs, wg, gs)
    u, eu = product(x, xs, wu, us)
    with np.errstate(over="ignore"):
        a = act(g, kind)
    ea = 1.14 * eg + (32 + 8 * np.minimum(np.abs(g) + np.abs(g) ** 3, 100)) * U * np.abs(a)
    return a * u, np.abs(u) * ea + np.abs(a) * eu + ea * eu + 2 * U * np.abs(a * u)


def logprobs(x, tokens, scale, top):
    """(logprob, entropy, top_logprob, top_token, bound of log probabilities, bound of the entropy); 64 bits, NaN-free rows."""
    z = x * scale
    m = z.max(1, keepdims=True)
    m = np.where(np.isneginf(m), 0.0, m)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.exp(z - m)
        total = e.sum(1, keepdims=True)
        lp = z - m - np.log(total)
        p = e / np.where(total > 0, total, 1)
        t = np.where(p > 0, z - m, 0.0)
        h = (np.log(total) - (p * t).sum(1, keepdims=True))[:, 0]
    none = total[:, 0] == 0
    lp[none], h[none] = -np.inf, 0.0
    which = np.argsort(-x, axis=1, kind="stable")[:, :top]
    given = np.where((tokens >= 0) & (tokens < x.shape[1]), np.take_along_axis(lp, np.clip(tokens, 0, x.shape[1] - 1)[:, None], 1)[:, 0], 0.0)
    adds = (x.shape[1] / 256 + 128) * U
    spread_t = np.abs(p * t).sum(1)
    return given, h, np.take_along_axis(lp, which, 1), which, adds, adds * (2 + 2 * spread_t)
