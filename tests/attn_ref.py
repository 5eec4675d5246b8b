"""Plain 64-bit implementations of the attention sublayer's operators, written from the formulas in
include/hc.h: the norms and the rotation, the 4-bit cache (values and byte layout) and the attention.
numpy only; arrays of bf16 come in as float64 values that bf16 holds exactly."""

import math

import numpy as np

BF16_HALF_STEP = 2.0 ** -8    # torch.finfo(bfloat16).eps / 2, relative
F16_HALF_STEP = 2.0 ** -11
U = 2.0 ** -24

CODES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
SCALES = np.array([m / 512.0 for m in range(8)]
                  + [(1 + m / 8.0) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1])  # bytes 0..126


def bf16(x):
    """x rounded to bf16 (nearest even), as float64; x holds float32 values."""
    a = np.asarray(x, np.float32)
    b = a.view(np.uint32)
    r = ((b >> 16) & 1) + 0x7FFF
    out = np.where(np.isfinite(a), (b + r) & 0xFFFF0000, b & 0xFFFF0000).astype(np.uint32)
    return out.view(np.float32).astype(np.float64)


# ---- norms and rotation --------------------------------------------------------------------------

def norm_rope(x, w, positions, inv_freq, axis, start, pairs, eps):
    """x [n, heads, dim]; w [heads, dim]; positions [axes, n] (python ints or int64) -> exact result, and the
    sum of the magnitudes of its two terms."""
    n, _, dim = x.shape
    r = 1.0 / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
    u = x * r * w[None]
    out, mag = u.copy(), np.abs(u)
    half = len(inv_freq)
    for j in range(half):
        a, b = (start + 2 * j, start + 2 * j + 1) if pairs else (start + j, start + half + j)
        turns = float(inv_freq[j]) / (2 * math.pi)
        for t in range(n):
            phi = math.fmod(int(positions[axis[j]][t]) * turns, 1.0) * 2 * math.pi
            c, s = math.cos(phi), math.sin(phi)
            out[t, :, a] = u[t, :, a] * c - u[t, :, b] * s
            out[t, :, b] = u[t, :, b] * c + u[t, :, a] * s
            mag[t, :, a] = mag[t, :, b] = np.abs(u[t, :, a]) + np.abs(u[t, :, b])
    return out, mag


# ---- the 4-bit cache ------------------------------------------------------------------------------

def nearest(x, levels):
    """Index of the level nearest to each x >= 0; of two as near, the even index."""
    mid = (levels[1:] + levels[:-1]) / 2
    lo, hi = np.searchsorted(mid, x, side="left"), np.searchsorted(mid, x, side="right")
    return np.where(lo % 2 == 0, lo, hi)


def quantise(x, unit):
    """x [..., dim] -> codes [..., dim] (0..15), scale bytes [..., dim / 16]."""
    g = np.asarray(x, np.float64).reshape(x.shape[:-1] + (x.shape[-1] // 16, 16)) / unit
    amax = np.abs(g).max(-1)
    bad = ~np.isfinite(amax)
    byte = nearest(np.where(bad, 0, amax) / 6.0, SCALES)
    s = SCALES[byte][..., None]
    safe = np.where(np.isfinite(g), g, 0.0)
    code = nearest(np.where(s > 0, np.abs(safe) / np.where(s > 0, s, 1.0), 0.0), CODES) + 8 * np.signbit(safe)
    return code.reshape(x.shape), np.where(bad, 127, byte)


def values(code, byte, unit):
    s = np.append(SCALES, np.nan)[byte]
    return (CODES[code % 8] * np.where(code >= 8, -1.0, 1.0)) * np.repeat(s, 16, axis=-1) * unit


def key_code_byte(t, i, dim):
    k = i % (dim // 4)
    return k // 16 * 512 + t % 8 * 64 + i // (dim // 4) * 16 + k // 4 % 4 * 4 + t // 8 * 2 + k // 2 % 2


def key_scale_byte(t, i, dim):
    return 8 * dim + t % 8 * (dim // 8) + i // (dim // 4) * (dim // 32) + t // 8 * (dim // 64) + i % (dim // 4) // 16


def value_code_byte(t, i, dim):
    v = i % (dim // 8)
    return 9 * dim + v // 8 * 512 + i // (dim // 8) * 64 + t % 8 // 2 * 16 + v // 2 % 4 * 4 + t // 8 * 2 + t % 2


def value_scale_byte(t, i, dim):
    return 17 * dim + i // 16 * 16 + t % 8 // 2 * 4 + t // 8 * 2 + t % 2


class Cache:
    """The cache as numpy bytes, written and read token by token."""

    def __init__(self, pages, page_size, heads, dim, k_unit=1.0, v_unit=1.0, fill=0):
        self.pages, self.size, self.heads, self.dim = pages, page_size, heads, dim
        self.units = (k_unit, v_unit)
        self.bytes = np.full((pages, heads, page_size // 16, 18 * dim), fill, np.uint8)
        t, i = np.arange(16)[:, None], np.arange(dim)[None]
        self.code_at = (key_code_byte(t, i, dim), value_code_byte(t, i, dim))
        i = np.arange(0, dim, 16)[None]
        self.scale_at = (key_scale_byte(t, i, dim), value_scale_byte(t, i, dim))

    def write(self, k, v, slots):
        """k, v [n, heads, dim] float64."""
        for part, x in ((0, k), (1, v)):
            code, byte = quantise(x, self.units[part])
            pair = code[..., 0::2] + 16 * code[..., 1::2]
            for j, s in enumerate(slots):
                if 0 <= s < self.pages * self.size:
                    block = self.bytes[s // self.size, :, s % self.size // 16]
                    block[:, self.code_at[part][s % 16, 0::2]] = pair[j]
                    block[:, self.scale_at[part][s % 16]] = byte[j]

    def read(self, slots):
        """(k, v) [n, heads, dim] float64; zeros for a slot outside."""
        out = np.zeros((2, len(slots), self.heads, self.dim))
        for part in (0, 1):
            for j, s in enumerate(slots):
                if 0 <= s < self.pages * self.size:
                    block = self.bytes[s // self.size, :, s % self.size // 16]
                    pair = block[:, self.code_at[part][s % 16, 0::2]].astype(np.int64)
                    code = np.stack((pair % 16, pair // 16), -1).reshape(self.heads, self.dim)
                    out[part, j] = values(code, block[:, self.scale_at[part][s % 16]].astype(np.int64), self.units[part])
        return out[0], out[1]


# ---- attention --------------------------------------------------------------------------------------

def attention(q, q_start, kv_len, table, cache: Cache, scale, causal=True, window=0):
    """Exact (out, lse) of every row that a sequence has (NaN elsewhere), and bounds on what an evaluation as
    include/hc.h describes it may be off by: the products in fp32, weights rounded to fp16, out rounded to bf16."""
    n, hq, dim = q.shape
    group = hq // cache.heads
    out, lse = np.full((n, hq, dim), np.nan), np.full((n, hq), np.nan)
    out_tol, lse_tol = np.zeros((n, hq, dim)), np.zeros((n, hq))
    for b, kvl in enumerate(kv_len):
        kvl = int(kvl)
        slots = []
        for p in range(kvl):
            page = int(table[b][p // cache.size])
            slots.append(page * cache.size + p % cache.size if 0 <= page < cache.pages else -1)
        K, V = cache.read(slots) if kvl else (np.zeros((0, cache.heads, dim)),) * 2
        there = np.array(slots, np.int64) >= 0
        ql = int(q_start[b + 1] - q_start[b])
        for i in range(ql):
            row = int(q_start[b]) + i
            pos = kvl - ql + i
            p = np.arange(kvl)
            seen = there & ((p <= pos) if causal else True) & ((p > pos - window) if window else True)
            for h in range(hq):
                k, v = K[seen, h // group], V[seen, h // group]
                if len(k) == 0:
                    out[row, h], lse[row, h] = 0.0, -np.inf
                    continue
                z = scale * (k @ q[row, h])
                m = z.max()
                w = np.exp(z - m)
                total = w.sum()
                out[row, h] = (w @ v) / total
                lse[row, h] = m + math.log(total)
                # z: a sum of dim products in fp32 and two roundings of its factor; exp2: 2^-22; the weights' sum: pairwise
                # per lane, at most len / 32 + 64 terms in a row
                dz = (dim + 16) * 2 * U * scale * (np.abs(k) @ np.abs(q[row, h])).max() + 4 * U * np.abs(z).max()
                # queries below 2^-22 of the row's largest may lose bits in fp16: 2^-25 of 2^-14 of the scaled row, a part in 2^33 of its
                # largest, per column
                dz += scale * np.abs(k).sum(-1).max() * np.abs(q[row, h]).max() * 2.0 ** -32
                rel = 2 * dz + 2.0 ** -21 + (len(k) / 32 + 64) * U
                wv = (w @ np.abs(v)) / total
                fine = len(k) * 2.0 ** -25 * np.abs(v).max() / total  # weights below fp16's normal range
                off = wv * (F16_HALF_STEP + 2 * rel) + fine
                out_tol[row, h] = off + BF16_HALF_STEP * (np.abs(out[row, h]) + off) + 2.0 ** -134
                lse_tol[row, h] = rel + 4 * U * abs(lse[row, h]) + 4 * U * abs(m)
    return out, lse, out_tol, lse_tol
