"""The attention sublayer's operators on the GPU against their plain 64-bit forms (attn_ref): norms with the
rotation, the 4-bit cache (byte for byte), the attention over it, their behaviour at the edges (no key, no
token, padding, indices out of range, NaN where nothing is seen, other streams, captured graphs), and a run of
them together inside a Hyper-Connection sublayer.

Tolerances, derived before any run:
  norm and rotation: the sum of squares has dim terms, r and the products a few roundings more, sine and cosine
    are off by less than 2^-22: an fp32 evaluation of a cos - b sin is off by at most (dim + 32) 2^-24 (|a| + |b|),
    and the result is rounded to bf16 once (2^-8 of the value: attn_ref.BF16_HALF_STEP).
  cache: none; the bytes are equal and the values read back are equal.
  attention: attn_ref.attention gives the bound with each row (fp32 products, weights rounded to fp16, one
    rounding to bf16)."""

import numpy as np
import pytest
import torch

import hyper_connection_residual_hc_gb300 as hc

import attn_ref as ar
import gpu_util as gu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    hc.load()
    gu.device_error_clear()
    yield
    gu.device_error_clear()


def bf(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16).cuda()


def f64(t):
    return t.double().cpu().numpy()


def ints(x, dtype):
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


def same(a, b):
    return np.array_equal(a, b, equal_nan=True)


# ---- norms and rotation ---------------------------------------------------------------------------

def _rope_case(n, hq, hk, dim, rot, start, pairs, axes, positions, rng, gain="shared"):
    x = ar.bf16(rng.standard_normal((n, hq + 2 * hk, dim)) * np.exp(rng.standard_normal((n, 1, 1))))
    w = {"none": np.ones((hq + hk, dim)), "shared": np.repeat(1 + 0.2 * rng.standard_normal((2, dim)), [hq, hk], 0),
         "head": 1 + 0.2 * rng.standard_normal((hq + hk, dim))}[gain].astype(np.float32).astype(np.float64)
    freq = [10000.0 ** (-2.0 * j / rot) for j in range(rot // 2)]
    axis = [int(a) for a in rng.integers(0, axes, rot // 2)]
    ref, mag = ar.norm_rope(x[:, :hq + hk], w, positions, freq, axis, start, pairs, 1e-6)
    table = None
    if rot:
        table = torch.empty(hc.hc_rope_table_size(rot), dtype=torch.uint8, device="cuda")
        hc.hc_prepare_rope(freq, axis if axes > 1 else None if not any(axis) else axis, rot, axes, table)
    return x, w, ref, mag, table


def _check_rope(got, ref, mag, dim):
    e = (dim + 32) * ar.U * mag
    tol = e + ar.BF16_HALF_STEP * (np.abs(ref) + e)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (int(bad.sum()), np.abs(got - ref)[bad].max(), np.argwhere(bad)[:4])


@pytest.mark.parametrize("gain", ["none", "shared", "head"])
@pytest.mark.parametrize("n,hq,hk,dim,rot,start,pairs,axes", [
    (1, 1, 1, 128, 128, 0, False, 1), (5, 40, 8, 128, 128, 0, False, 1), (3, 33, 3, 128, 64, 64, True, 1),
    (7, 4, 0, 64, 32, 16, False, 2), (2, 70, 70, 64, 64, 0, True, 3), (4, 5, 5, 80, 80, 0, False, 3),
    (3, 6, 2, 96, 48, 48, False, 4), (3, 9, 3, 192, 64, 128, True, 1), (5, 16, 4, 256, 256, 0, False, 1),
    (4, 3, 1, 256, 32, 104, True, 2), (2, 11, 2, 16, 16, 0, False, 1), (6, 3, 3, 8, 0, 0, False, 1), (3, 2, 1, 40, 32, 8, True, 1),
    (2, 4, 4, 128, 0, 0, False, 1),
])
def test_norm_rope(n, hq, hk, dim, rot, start, pairs, axes, gain):
    rng = np.random.default_rng(n * 1000 + dim)
    positions = rng.integers(-(1 << 20), 1 << 20, (axes, n))
    positions[0, 0] = 0
    x, w, ref, mag, table = _rope_case(n, hq, hk, dim, rot, start, pairs, axes, positions, rng, gain)
    X = bf(x).reshape(n, -1)  # one buffer: q, k and v columns side by side
    stride = X.stride(0)
    q, k = X[:, :hq * dim], X[:, hq * dim:]
    wt = {"none": (None, None), "shared": (gu.dev_f32(w[0]), gu.dev_f32(w[hq] if hk else w[0])),
          "head": (gu.dev_f32(w[:hq]), gu.dev_f32(w[hq:]) if hk else None)}[gain]
    pos = ints(positions, torch.int64)
    r = hc.rope(table, rot, start, axes, hc.HC_ROPE_PAIRS if pairs else hc.HC_ROPE_HALF)
    s = hc.heads(hq, hk, dim, 1e-6, gain == "head")
    qo, ko = gu.guarded((n, hq, dim)), gu.guarded((n, max(hk, 1), dim))
    before = X.clone()
    hc.hc_qk_norm_rope(q, stride, k if hk else None, stride, wt[0], wt[1], pos if rot else None, r, n, s, qo, hq * dim,
                       ko if hk else None, hk * dim)
    assert torch.equal(X, before)
    _check_rope(f64(qo), ref[:, :hq], mag[:, :hq], dim)
    if hk:
        _check_rope(f64(ko)[:, :hk], ref[:, hq:], mag[:, hq:], dim)
    # in place on the columns of the buffer: the same values, the v columns untouched
    hc.hc_qk_norm_rope(q, stride, k if hk else None, stride, wt[0], wt[1], pos if rot else None, r, n, s, q, stride,
                       k if hk else None, stride)
    got = X.reshape(n, hq + 2 * hk, dim)
    assert torch.equal(got[:, :hq], qo) and torch.equal(got[:, hq + hk:], before.reshape(n, -1, dim)[:, hq + hk:])
    assert hk == 0 or torch.equal(got[:, hq:hq + hk], ko)


def test_norm_rope_of_far_positions():
    """2^40 positions on: the angle modulo a turn is still the frequency's (whose 2^-52 relative error is then 2^-12 turns for
    the fastest, so the check takes frequencies that are whole fractions of a turn, exact in the table)."""
    rng = np.random.default_rng(5)
    n, h, dim = 9, 2, 64
    x = ar.bf16(rng.standard_normal((n, h, dim)))
    k = rng.integers(1, 1 << 20, dim // 2)
    positions = rng.integers(-(1 << 40), 1 << 40, (1, n))
    table = torch.empty(hc.hc_rope_table_size(dim), dtype=torch.uint8, device="cuda")
    hc.hc_prepare_rope([2 * np.pi * int(v) / 2.0 ** 20 for v in k], None, dim, 1, table)
    qo = gu.guarded((n, h, dim))
    hc.hc_qk_norm_rope(bf(x), h * dim, None, 0, None, None, ints(positions, torch.int64), hc.rope(table, dim), n, hc.heads(h, 0, dim, 0.0),
                       qo, h * dim, None, 0)
    u = x / np.sqrt((x ** 2).mean(-1, keepdims=True))
    # 2 pi k / 2^20 is off by 2^-53 relative in fp64, and its quotient by 2 pi as much again: 2^-52 * 2^40 turns at most
    slack = 2 * np.pi * 2.0 ** -12
    turns = np.array([[int(p) * int(v) % (1 << 20) / 2.0 ** 20 for v in k] for p in positions[0]])[:, None]
    a, b, c, s = u[..., :32], u[..., 32:], np.cos(2 * np.pi * turns), np.sin(2 * np.pi * turns)
    ref = np.concatenate((a * c - b * s, b * c + a * s), -1)
    mag = np.concatenate((np.abs(a) + np.abs(b),) * 2, -1)
    e = ((dim + 32) * ar.U + slack) * mag
    assert (np.abs(f64(qo) - ref) <= e + ar.BF16_HALF_STEP * (np.abs(ref) + e)).all()


def test_norm_rope_specials_stay_in_their_head():
    rng = np.random.default_rng(6)
    n, hq, hk, dim = 2, 3, 1, 128
    positions = np.array([[5, 9]])
    x, w, ref, mag, table = _rope_case(n, hq, hk, dim, 64, 0, False, 1, positions, rng, "none")
    x[0, 1, 7], x[1, 3, 100] = np.nan, np.inf  # a query head, the key head
    x[0, 2] = 0.0
    X = bf(x[:, :hq + hk])
    qo, ko = gu.guarded((n, hq, dim)), gu.guarded((n, hk, dim))
    st = (hq + hk) * dim
    hc.hc_qk_norm_rope(X, st, X[:, hq:], st, None, None, ints(positions, torch.int64), hc.rope(table, 64), n, hc.heads(hq, hk, dim),
                       qo, hq * dim, ko, hk * dim)
    q, k = f64(qo), f64(ko)
    assert np.isnan(q[0, 1]).all() and (q[0, 2] == 0).all()
    # r = 0 for the infinite row: its finite columns are 0, the infinite one NaN
    assert np.isnan(k[1, 0, 100]) and (np.delete(k[1, 0], 100) == 0).all()
    for t, h in ((0, 0), (1, 0), (1, 1), (1, 2)):
        _check_rope(q[t, h], ref[t, h], mag[t, h], dim)


# ---- the cache --------------------------------------------------------------------------------------

def _kv(rng, n, heads, dim):
    """Values of many magnitudes, groups with exact ties, zeros, one value among zeros."""
    x = rng.standard_normal((2, n, heads, dim)) * np.exp(2 * rng.standard_normal((2, n, heads, 1)))
    grid = rng.integers(-24, 25, x.shape) / 4.0  # multiples of 1/4 of a scale of 1: ties between codes
    pick = rng.random((2, n, heads, 1))
    x = np.where(pick < 0.3, grid * 2.0 ** rng.integers(-6, 6, x.shape[:-1] + (1,)), x)
    x = np.where(pick > 0.95, 0.0, x)
    x[:, :, :, 3] = np.where(pick[..., 0] > 0.9, -2.0 ** rng.integers(-14, 14, pick.shape[:-1]), x[:, :, :, 3])
    return ar.bf16(x)


def _device_cache(c):
    return torch.from_numpy(c.bytes.copy()).cuda()


def _shape(c):
    return hc.kv_shape(c.pages, c.size, c.heads, c.dim, *c.units)


def _write(c, dev, k, v, slots):
    heads, dim, n = c.heads, c.dim, len(slots)
    both = torch.cat((bf(k).reshape(n, -1), bf(v).reshape(n, -1)), 1)  # a token's keys, then its values
    st = both.stride(0)
    hc.hc_kv_write(both, st, both[:, heads * dim:], st, ints(slots, torch.int64), n, _shape(c), dev)


def _slots(kind, n, cap, rng):
    if kind == "run":          # from the start of a block on
        return np.arange(n) + 32
    if kind == "odd":          # from the middle of a block on: ragged ends
        return np.arange(n) + 21
    if kind == "runs":         # several sequences, each with a ragged start and end
        out, at = [], 0
        while len(out) < n:
            at += int(rng.integers(1, 40))
            m = min(int(rng.integers(1, 70)), n - len(out))
            out += list(range(at, at + m))
            at += m
        return np.array(out)
    out = rng.permutation(cap)[:n]  # anywhere
    if kind == "padded":
        out = np.where(rng.random(n) < 0.3, -1 - rng.integers(0, 99, n), out)
    return out


@pytest.mark.parametrize("kind", ["run", "odd", "runs", "scattered", "padded"])
@pytest.mark.parametrize("heads,dim,size,units,n", [
    (1, 64, 16, (1.0, 1.0), 97), (3, 128, 64, (0.25, 1024.0), 150), (8, 128, 32, (1.0, 1.0), 31), (2, 256, 128, (2.0 ** -20, 2.0 ** 9), 83),
    (9, 64, 1024, (1.0, 0.5), 16), (1, 128, 16, (1.0, 1.0), 1),
])
def test_cache_bytes_and_values(kind, heads, dim, size, units, n):
    rng = np.random.default_rng(heads * 100 + n)
    pages = -(-(3 * n + 150) // size)
    c = ar.Cache(pages, size, heads, dim, *units, fill=0x5A)
    dev = _device_cache(c)
    slots = _slots(kind, n, pages * size, rng)
    k, v = _kv(rng, n, heads, dim)
    _write(c, dev, k, v, slots)
    c.write(k, v, slots)
    assert same(dev.cpu().numpy(), c.bytes)  # every byte, those of other tokens too
    # read back in the same order, with strides, and once more in another order with repeats
    for order in (slots, rng.permutation(np.concatenate((slots, slots[: n // 2], [-1, -7])))):
        m = len(order)
        ko, vo = gu.guarded((m, heads * dim + 24)), gu.guarded((m, heads, dim))
        ko.zero_()
        hc.hc_kv_read(dev, ints(order, torch.int64), m, _shape(c), ko, heads * dim + 24, vo, heads * dim)
        rk, rv = c.read(order)
        assert same(f64(ko)[:, :heads * dim].reshape(m, heads, dim), rk) and same(f64(vo), rv)
        assert (ko[:, heads * dim:] == 0).all()
        one = gu.guarded((m, heads, dim))
        hc.hc_kv_read(dev, ints(order, torch.int64), m, _shape(c), None, 0, one, heads * dim)
        assert same(f64(one), rv)
    gu.device_error_clear()


def test_cache_bytes_do_not_depend_on_grouping():
    """A prompt written at once, in two calls cut anywhere, or token by token: the same bytes."""
    rng = np.random.default_rng(8)
    heads, dim, n = 2, 128, 70
    k, v = _kv(rng, n, heads, dim)
    slots = np.arange(n) + 16
    ref = None
    for cuts in ([0, n], [0, 7, n], [0, 33, 34, n], list(range(n + 1))):
        c = ar.Cache(4, 64, heads, dim)
        dev = _device_cache(c)
        for a, b in zip(cuts[:-1], cuts[1:]):
            _write(c, dev, k[a:b], v[a:b], slots[a:b])
        ref = dev if ref is None else ref
        assert torch.equal(dev, ref)


def test_cache_specials_and_bad_slots():
    rng = np.random.default_rng(9)
    heads, dim, n = 2, 64, 40
    c = ar.Cache(4, 16, heads, dim, fill=0x33)
    k, v = _kv(rng, n, heads, dim)
    k[3, 0, 5], k[20, 1, 63], v[3, 1, 0], v[39, 0, 17] = np.nan, -np.inf, np.inf, np.nan
    k[4, 0, :16] = 3e38  # saturates: the largest scale and code
    k[4, 0, 3] = -3e38
    slots = np.arange(n) + 8
    dev = _device_cache(c)
    _write(c, dev, k, v, slots)
    c.write(k, v, slots)
    # the codes of a group with the scale NaN are not specified
    ko, vo = gu.guarded((n, heads, dim)), gu.guarded((n, heads, dim))
    hc.hc_kv_read(dev, ints(slots, torch.int64), n, _shape(c), ko, heads * dim, vo, heads * dim)
    rk, rv = c.read(slots)
    assert same(f64(ko), rk) and same(f64(vo), rv)
    assert np.isnan(rk[3, 0, :16]).all() and not np.isnan(rk[3, 0, 16:]).any() and rk[4, 0, 0] == 2688 and rk[4, 0, 3] == -2688
    gu.device_error_clear()
    # past the end: left out, the bit set, nothing else touched
    before = dev.clone()
    bad = np.array([64, 1 << 40, -1])
    _write(c, dev, k[:3], v[:3], bad)
    assert torch.equal(dev, before)
    assert hc.hc_device_error(clear=True) == 1 << 20
    hc.hc_kv_read(dev, ints(bad, torch.int64), 3, _shape(c), ko, heads * dim, vo, heads * dim)
    assert (ko[:3] == 0).all() and (vo[:3] == 0).all()
    assert hc.hc_device_error(clear=True) == 1 << 20 and hc.hc_device_error(clear=True) == 0


# ---- attention ----------------------------------------------------------------------------------------

class Problem:
    """Sequences on shuffled pages: `lens` = [(queries, keys)]; pages no sequence has are full of NaN scales, as are the
    tokens behind each sequence's last key."""

    def __init__(self, lens, hq, hk, dim, size, seed=0, units=(1.0, 1.0), spare=3, extra_rows=0):
        rng = np.random.default_rng(seed)
        self.lens, self.hq = lens, hq
        need = [-(-kv // size) for _, kv in lens]
        self.max_pages = max(need + [1]) + 1
        self.cache = c = ar.Cache(sum(need) + spare, size, hk, dim, *units, fill=0xFF)
        order = rng.permutation(c.pages)
        self.table = np.full((len(lens), self.max_pages), -1, np.int32)
        at = 0
        for b, m in enumerate(need):
            self.table[b, :m] = order[at:at + m]
            at += m
        for b, (_, kv) in enumerate(lens):
            k = ar.bf16(rng.standard_normal((kv, hk, dim)) * units[0])
            v = ar.bf16(rng.standard_normal((kv, hk, dim)) * units[1])
            c.write(k, v, [int(self.table[b, p // size]) * size + p % size for p in range(kv)])
        self.q_start = np.concatenate(([0], np.cumsum([q for q, _ in lens]))).astype(np.int32)
        self.n = int(self.q_start[-1]) + extra_rows
        self.q = ar.bf16(rng.standard_normal((self.n, hq, dim)))
        self.kv_len = np.array([kv for _, kv in lens], np.int32)
        self.scale = dim ** -0.5 / units[0]

    def to_device(self):
        self.d = dict(q=bf(self.q), q_start=ints(self.q_start, torch.int32), kv_len=ints(self.kv_len, torch.int32),
                      table=ints(self.table, torch.int32), cache=_device_cache(self.cache))
        return self

    def run(self, causal=True, window=0, max_q_len=None, with_lse=True, ws=None, fill=7.0, scale=None, stream=None):
        d, dim = self.d, self.cache.dim
        a = hc.attention(self.n, len(self.lens), max(q for q, _ in self.lens) if max_q_len is None else max_q_len, self.max_pages,
                         self.hq, self.scale if scale is None else scale, causal, window)
        out, lse = gu.guarded((self.n, self.hq, dim)), gu.guarded((self.n, self.hq), torch.float32)
        out.fill_(fill)
        lse.fill_(fill)
        hc.hc_kv_attention(d["q"], self.hq * dim, d["q_start"], d["kv_len"], d["table"], d["cache"], a, _shape(self.cache), out,
                           self.hq * dim, lse if with_lse else None, workspace() if ws is None else ws, stream)
        return out, lse

    def check(self, out, lse, causal=True, window=0, scale=None):
        ref, rlse, tol, ltol = ar.attention(self.q, self.q_start, self.kv_len, self.table, self.cache,
                                            self.scale if scale is None else scale, causal, window)
        m = int(self.q_start[-1])
        got, glse = f64(out), f64(lse)
        bad = ~(np.abs(got[:m] - ref[:m]) <= tol[:m])
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4], got[:m][bad][:4], ref[:m][bad][:4], tol[:m][bad][:4])
        inf = np.isneginf(rlse[:m])
        assert (np.isneginf(glse[:m]) == inf).all()
        bad = ~(np.abs(glse[:m][~inf] - rlse[:m][~inf]) <= ltol[:m][~inf])
        assert not bad.any(), (int(bad.sum()), glse[:m][~inf][bad][:4], rlse[:m][~inf][bad][:4], ltol[:m][~inf][bad][:4])


_WS = None


def workspace():
    global _WS
    if _WS is None:
        _WS = hc.new_kv_workspace()
    return _WS


@pytest.mark.parametrize("lens", [
    [(1, 1)], [(1, 17), (1, 300), (1, 0), (1, 64)], [(3, 40), (1, 5), (0, 100), (4, 200)], [(2, 1), (5, 3), (1, 16)],
    [(70, 70), (1, 129)], [(33, 257)],
], ids=["one", "decode", "drafts", "fewer_keys_than_queries", "prefill", "chunk"])
@pytest.mark.parametrize("hq,hk,dim,size", [(1, 1, 64, 16), (5, 1, 128, 64), (8, 2, 128, 16), (6, 6, 64, 32), (16, 1, 256, 128), (12, 4, 256, 16),
                                            (40, 2, 64, 64), (34, 2, 128, 32)])
def test_attention(lens, hq, hk, dim, size):
    p = Problem(lens, hq, hk, dim, size, seed=hq * dim + len(lens), extra_rows=2).to_device()
    out, lse = p.run()
    p.check(out, lse)
    m = int(p.q_start[-1])
    assert (out[m:] == 7).all() and (lse[m:] == 7).all()  # rows behind the last sequence
    gu.device_error_clear()
    again, lagain = p.run()
    assert torch.equal(out, again) and torch.equal(lse, lagain)
    gu.device_error_clear()


@pytest.mark.parametrize("lens,window", [([(1, 300), (1, 40)], 64), ([(1, 500), (3, 77), (1, 1)], 1), ([(40, 200), (7, 7)], 33), ([(130, 130)], 17),
                                         ([(1, 90)], 1000)])
@pytest.mark.parametrize("hq,hk,dim,size", [(5, 1, 128, 16), (8, 2, 64, 64), (4, 4, 256, 32)])
def test_attention_window(lens, window, hq, hk, dim, size):
    p = Problem(lens, hq, hk, dim, size, seed=window).to_device()
    # pages that no query sees any more are given back: their entries hold nothing valid
    for b, (q, kv) in enumerate(lens):
        gone = max(0, kv - q - window + 1) // size
        p.table[b, :gone] = [-1, 10 ** 6][b % 2]
    p.d["table"] = ints(p.table, torch.int32)
    out, lse = p.run(window=window)
    p.check(out, lse, window=window)
    gu.device_error_clear()


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 5])
@pytest.mark.parametrize("hq,hk,dim", [(5, 1, 128), (4, 2, 64), (2, 1, 256)])
def test_attention_widest_window_with_fewer_keys_than_queries(hq, hk, dim, window):
    for lens in ([(5, 3), (1, 20), (3, 0)], [(70, 40), (5, 3)]):
        p = Problem(lens, hq, hk, dim, 32, seed=5).to_device()
        out, lse = p.run(window=window)
        p.check(out, lse)


@pytest.mark.parametrize("hq,hk,dim", [(5, 1, 128), (4, 2, 64), (2, 1, 256)])
def test_attention_without_causal_mask(hq, hk, dim):
    p = Problem([(4, 50), (20, 133), (3, 0), (150, 64)], hq, hk, dim, 32, seed=3).to_device()
    out, lse = p.run(causal=False)
    p.check(out, lse, causal=False)


def test_attention_strides_units_scale_and_no_lse():
    p = Problem([(2, 70), (1, 200)], 6, 2, 128, 64, seed=11, units=(0.125, 8.0)).to_device()
    ref, _ = p.run(scale=0.5)
    p.check(ref, p.run(scale=0.5)[1], scale=0.5)
    n, w = p.n, 6 * 128
    wide = torch.full((n, w + 40), 3.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 8:8 + w] = p.d["q"].reshape(n, w)
    out = gu.guarded((n, w + 16))
    out.fill_(5.0)
    a = hc.attention(n, 2, 2, p.max_pages, 6, 0.5)
    hc.hc_kv_attention(wide[:, 8:], w + 40, p.d["q_start"], p.d["kv_len"], p.d["table"], p.d["cache"], a, _shape(p.cache), out[:, 16:],
                       w + 16, None, workspace())
    assert torch.equal(out[:, 16:].reshape(n, 6, 128), ref) and (out[:, :16] == 5).all()
    zero, lse = p.run(scale=0.0)  # equal weights
    p.check(zero, lse, scale=0.0)


@pytest.mark.parametrize("hint", [0, 1, 3, 1000])
def test_attention_right_for_any_longest_query_hint(hint):
    p = Problem([(9, 120), (1, 33), (200, 260)], 5, 1, 128, 32, seed=12).to_device()
    out, lse = p.run(max_q_len=hint)
    p.check(out, lse)


@pytest.mark.parametrize("window", [0, 100])
@pytest.mark.parametrize("hq,hk,dim", [(1, 1, 64), (5, 1, 128), (16, 2, 64), (32, 1, 128), (34, 1, 128), (2, 1, 256)])
def test_attention_chunks_among_single_tokens(hq, hk, dim, window):
    """Sequences on either side of every border between few queries and many, in one batch; then a batch too small for
    its own hint."""
    p = Problem([(1, 70), (300, 400), (1, 0), (0, 5), (2, 33), (8, 50), (9, 60), (1, 513), (40, 40)], hq, hk, dim, 32, seed=hq).to_device()
    out, lse = p.run(window=window)
    p.check(out, lse, window=window)
    again, lagain = p.run(window=window)
    assert torch.equal(out, again) and torch.equal(lse, lagain)
    gu.device_error_clear()
    p = Problem([(1, 70), (0, 3), (2, 90)], hq, hk, dim, 32, seed=hq).to_device()
    out, lse = p.run(window=window, max_q_len=500)
    p.check(out, lse, window=window)
    gu.device_error_clear()


@pytest.mark.parametrize("hq,hk,dim", [(5, 1, 128), (16, 2, 64)])
def test_attention_chunk_among_single_tokens_replayed(hq, hk, dim):
    """Both kernels of such a call cut their keys, and so use the workspace; calls follow each other in one graph."""
    p = Problem([(1, 6000), (40, 5000), (1, 4100)], hq, hk, dim, 64, seed=21).to_device()
    out, lse = p.run()
    p.check(out, lse)
    ws = hc.new_kv_workspace()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        results = [p.run(ws=ws, fill=float(i)) for i in range(3)]
    for _ in range(3):
        for o, l in results:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        for o, l in results:
            assert torch.equal(o, out) and torch.equal(l, lse)
    assert (ws[:2048] == 0).all()  # the counters
    gu.device_error_clear()


@pytest.mark.parametrize("scale", [1.0, 30.0])
def test_attention_with_large_and_growing_scores(scale):
    """Scores of hundreds whose maximum comes late: a running maximum that rises at every step."""
    p = Problem([(1, 900), (6, 400)], 4, 1, 128, 64, seed=13).to_device()
    c = p.cache
    for b, (_, kv) in enumerate(p.lens):
        slots = [int(p.table[b, t // c.size]) * c.size + t % c.size for t in range(kv)]
        k, v = c.read(slots)
        c.write(ar.bf16(k * (1 + np.arange(kv) / 100.0)[:, None, None]), v, slots)
    p.to_device()
    out, lse = p.run(scale=scale * p.scale)
    p.check(out, lse, scale=scale * p.scale)


def test_attention_keeps_small_queries_beside_large_ones():
    """A query row of many magnitudes and one of tiny ones: the fp16 products lose nothing of them."""
    p = Problem([(3, 150)], 4, 2, 64, 16, seed=14)
    rng = np.random.default_rng(2)
    p.q[0] *= 2.0 ** rng.integers(-12, 12, p.q[0].shape)
    p.q[1] *= 2.0 ** -60
    p.q[2] *= 2.0 ** 20
    p.to_device()
    for scale in (1.0, 2.0 ** 50):
        if scale > 1:
            p.q[0], p.q[2] = p.q[0] * 2.0 ** -60, p.q[2] * 2.0 ** -70
            p.to_device()
        out, lse = p.run(scale=scale)
        p.check(out, lse, scale=scale)


def test_attention_specials():
    """NaN and infinities reach the rows that see them and no other."""
    p = Problem([(6, 70)], 4, 2, 128, 16, seed=15)
    c = p.cache
    slots = [int(p.table[0, t // 16]) * 16 + t % 16 for t in range(70)]
    k, v = c.read(slots)
    k[67, 0, 3] = np.nan  # position 67: seen by queries 3, 4, 5 (positions 67, 68, 69); kv head 0
    v[68, 1, 40] = np.inf  # seen by queries 4, 5; kv head 1, columns 32..47
    c.write(k, v, slots)
    p.q[1, 2, 9] = np.nan
    p.to_device()
    out, lse = p.run()
    got, glse = f64(out), f64(lse)
    assert np.isnan(got[3:, :2]).all() and np.isnan(glse[3:, :2]).all()
    assert np.isnan(got[1, 2]).all()
    assert np.isnan(got[4:, 2:, 32:48]).all()
    clean = Problem([(6, 70)], 4, 2, 128, 16, seed=15)
    ref, rlse, tol, ltol = ar.attention(clean.q, clean.q_start, clean.kv_len, clean.table, clean.cache, clean.scale)
    for i in range(6):
        for h in range(4):
            if (h < 2 and i >= 3) or (i, h) == (1, 2):
                continue
            cols = np.r_[0:32, 48:128] if h >= 2 and i >= 4 else np.arange(128)
            assert (np.abs(got[i, h, cols] - ref[i, h, cols]) <= tol[i, h, cols]).all(), (i, h)
            assert abs(glse[i, h] - rlse[i, h]) <= ltol[i, h]


@pytest.mark.parametrize("lens", [[(1, 150), (3, 90)], [(120, 150), (140, 300)]], ids=["few", "many"])
def test_attention_bad_pages_and_bounds(lens):
    """A page out of range is left out and told of; so are lengths past the table; row bounds are clamped."""
    p = Problem(lens, 5, 1, 128, 32, seed=16).to_device()
    p.table[0, 1] = -3
    p.table[1, 0] = p.cache.pages
    p.d["table"] = ints(p.table, torch.int32)
    out, lse = p.run()
    p.check(out, lse)
    assert hc.hc_device_error(clear=True) == 1 << 20
    p = Problem(lens, 5, 1, 128, 32, seed=17).to_device()
    p.d["kv_len"] = ints([lens[0][1], -4], torch.int32)
    out, lse = p.run()
    assert hc.hc_device_error(clear=True) & ~(1 << 20) == 1 << 21
    p.kv_len[1] = 0
    p.check(out, lse)
    p.d["kv_len"] = ints([10 ** 9, lens[1][1]], torch.int32)  # past the table: the last page's entry is -1
    out, lse = p.run(causal=False)
    assert hc.hc_device_error(clear=True) == 3 << 20
    p = Problem(lens, 5, 1, 128, 32, seed=18).to_device()
    p.d["q_start"] = ints([0, lens[0][0], p.n + 5], torch.int32)  # the second sequence is said to have five rows more than there are
    out, _ = p.run()
    assert hc.hc_device_error(clear=True) & ~(1 << 20) == 1 << 21
    p.d["q_start"] = ints([-2, lens[0][0], p.n], torch.int32)
    out, _ = p.run()
    assert hc.hc_device_error(clear=True) & ~(1 << 20) == 1 << 21


def test_attention_long_context():
    """70,001 keys of one sequence: spread over the GPU and joined; offsets past 2^31 in the cache."""
    rng = np.random.default_rng(20)
    hq, hk, dim, size, kv = 5, 1, 128, 128, 70001
    pages = 1 + (1 << 32) // (18 * dim * size // 16)  # past 2^32 bytes
    shape = hc.kv_shape(pages, size, hk, dim)
    nbytes = hc.hc_kv_cache_size(shape)
    assert nbytes > 1 << 32
    cache = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    need = -(-kv // size)
    table = np.concatenate((np.arange(need // 2), pages - 1 - np.arange(need - need // 2)))
    slots = torch.from_numpy(table[np.arange(kv) // size] * size + np.arange(kv) % size).cuda()
    k = torch.randn((kv, hk, dim), device="cuda", dtype=torch.bfloat16)
    v = torch.randn((kv, hk, dim), device="cuda", dtype=torch.bfloat16)
    hc.hc_kv_write(k, dim, v, dim, slots, kv, shape, cache)
    kq, vq = torch.empty_like(k), torch.empty_like(v)
    hc.hc_kv_read(cache, slots, kv, shape, kq, dim, vq, dim)
    q = bf(ar.bf16(rng.standard_normal((1, hq, dim))))
    out, lse = gu.guarded((1, hq, dim)), gu.guarded((1, hq), torch.float32)
    a = hc.attention(1, 1, 1, need, hq, dim ** -0.5)
    hc.hc_kv_attention(q, hq * dim, ints([0, 1], torch.int32), ints([kv], torch.int32), ints(table[None], torch.int32), cache, a, shape, out,
                       hq * dim, lse, workspace())
    K, V, Q = f64(kq)[:, 0], f64(vq)[:, 0], f64(q)[0]
    z = Q @ K.T * dim ** -0.5
    m = z.max(-1, keepdims=True)
    w = np.exp(z - m)
    ref, rl = (w @ V) / w.sum(-1, keepdims=True), (m + np.log(w.sum(-1, keepdims=True)))[:, 0]
    # as in attn_ref.attention: z off by dz, each weight by 2 dz + 2^-21 + 2^-11, weights below fp16's normal range by 2^-25
    dz = (dim + 16) * 2 * ar.U * dim ** -0.5 * (np.abs(Q) @ np.abs(K).T).max() + 4 * ar.U * np.abs(z).max()
    rel = 2 * dz + 2.0 ** -21 + (kv / 32 + 64) * ar.U
    off = (w @ np.abs(V)) / w.sum(-1, keepdims=True) * (ar.F16_HALF_STEP + 2 * rel) + kv * 2.0 ** -25 * np.abs(V).max() / w.sum(-1, keepdims=True)
    assert (np.abs(f64(out)[0] - ref) <= off + ar.BF16_HALF_STEP * (np.abs(ref) + off)).all()
    assert (np.abs(f64(lse)[0] - rl) <= rel + 8 * ar.U * np.abs(rl)).all()
    gu.device_error_clear()


@pytest.mark.parametrize("window", [0, 700])
@pytest.mark.parametrize("hq,hk,dim,size", [(5, 1, 128, 64), (8, 2, 64, 16)])
def test_attention_chunk_behind_a_long_context(hq, hk, dim, size, window):
    """A few row tiles over many keys: the keys of a tile in slices, joined in their order; one page is not there."""
    p = Problem([(40, 3000), (33, 1201)], hq, hk, dim, size, seed=hq).to_device()
    if window == 0:
        p.table[0, 3] = -1
        p.d["table"] = ints(p.table, torch.int32)
    w = hc.new_kv_workspace()
    out, lse = p.run(window=window, ws=w)
    p.check(out, lse, window=window)
    assert hc.hc_device_error(clear=True) == (1 << 20 if window == 0 else 0)
    for _ in range(3):
        again, lagain = p.run(window=window, ws=w)
        assert torch.equal(out, again) and torch.equal(lse, lagain)
    assert (w[:2048] == 0).all()
    hc.hc_device_error(clear=True)


@pytest.mark.parametrize("seqs", [300, 1000])
def test_attention_many_sequences(seqs):
    rng = np.random.default_rng(seqs)
    lens = [(int(rng.integers(0, 3)), int(kv)) for kv in rng.integers(0, 40, seqs)]
    p = Problem(lens, 2, 1, 64, 16, seed=seqs).to_device()
    out, lse = p.run()
    p.check(out, lse)
    gu.device_error_clear()


@pytest.mark.parametrize("seqs", [32, 33, 500, 900])
def test_attention_many_sequences_of_many_queries(seqs):
    rng = np.random.default_rng(seqs)
    lens = [(int(q), int(kv)) for q, kv in zip(rng.choice([0, 1, 4, 5, 9, 20, 40], seqs), rng.integers(0, 40, seqs))]
    p = Problem(lens, 8, 1, 64, 16, seed=seqs).to_device()
    out, lse = p.run()
    p.check(out, lse)
    gu.device_error_clear()


def test_attention_on_two_streams_at_once():
    """Two calls that overlap, each with a workspace of its own, on streams other than the tensors'."""
    ps = [Problem([(1, 3000), (1, 1000)], 5, 1, 128, 64, seed=21 + i).to_device() for i in range(2)]
    alone = [p.run() for p in ps]
    ws = [hc.new_kv_workspace() for _ in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for p, w, s in zip(ps, ws, streams):
            with torch.cuda.stream(s):
                got.append(p.run(ws=w))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert torch.equal(g[0], alone[i % 2][0]) and torch.equal(g[1], alone[i % 2][1])
    for p, (o, l) in zip(ps, alone):
        p.check(o, l)


@pytest.mark.parametrize("dim", [64, 128])
def test_attention_of_many_queries_beside_other_calls(dim):
    """A prefill on one stream, decode and another prefill on two others, each with a workspace of its own."""
    ps = [Problem(lens, 8, 2, dim, 32, seed=31 + i).to_device()
          for i, lens in enumerate([[(300, 700), (40, 1500)], [(1, 3000), (1, 1000)], [(1, 900), (200, 200), (64, 2500)]])]
    alone = [p.run() for p in ps]
    ws = [hc.new_kv_workspace() for _ in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for p, w, s in zip(ps, ws, streams):
            with torch.cuda.stream(s):
                got.append(p.run(ws=w))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert torch.equal(g[0], alone[i % 3][0]) and torch.equal(g[1], alone[i % 3][1])
    for p, (o, l) in zip(ps, alone):
        p.check(o, l)
    gu.device_error_clear()


def test_attention_replayed_as_the_context_grows():
    """One captured call, replayed with longer and shorter contexts, as a decode loop does; the workspace's counters are left
    at zero each time."""
    p = Problem([(1, 2500), (1, 700), (1, 64)], 5, 1, 128, 64, seed=23).to_device()
    w = hc.new_kv_workspace()
    p.run(ws=w)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = p.run(ws=w)
    for lens in ([2500, 700, 64], [1, 0, 33], [1999, 700, 50], [2500, 16, 64]):
        p.kv_len = np.array(lens, np.int32)
        p.d["kv_len"].copy_(ints(lens, torch.int32))
        g.replay()
        torch.cuda.synchronize()
        p.check(out, lse)
        assert (w[:2048] == 0).all()
    gu.device_error_clear()


# ---- together -----------------------------------------------------------------------------------------

class Sublayer:
    """An attention sublayer between two Hyper-Connection calls: y -> q, k, v -> norms and rotation -> cache -> attention ->
    output projection -> Delta. Static buffers, so that a decode step can be captured."""

    def __init__(self, seqs, size, pages, seed=0, d=512, hq=4, hk=1, dim=128):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.d, self.hq, self.hk, self.dim, self.seqs = d, hq, hk, dim, seqs
        self.w = torch.randn(((hq + 2 * hk) * dim, d), generator=g, device="cuda", dtype=torch.bfloat16) * d ** -0.5
        self.o = torch.randn((d, hq * dim), generator=g, device="cuda", dtype=torch.bfloat16) * (hq * dim) ** -0.5
        self.qw = 1 + 0.1 * torch.randn(dim, generator=g, device="cuda")
        self.kw = 1 + 0.1 * torch.randn(dim, generator=g, device="cuda")
        self.freq = [10000.0 ** (-2.0 * j / dim) for j in range(dim // 2)]
        self.table = torch.empty(hc.hc_rope_table_size(dim), dtype=torch.uint8, device="cuda")
        hc.hc_prepare_rope(self.freq, None, dim, 1, self.table)
        self.shape = hc.kv_shape(seqs * pages, size, hk, dim)
        self.cache = torch.zeros(hc.hc_kv_cache_size(self.shape), dtype=torch.uint8, device="cuda")
        self.pages = torch.randperm(seqs * pages, generator=g, device="cuda").int().reshape(seqs, pages)
        self.size, self.ws = size, hc.new_kv_workspace()

    def slots(self, positions):
        """[seqs, tokens] positions -> slots, flattened."""
        page = torch.gather(self.pages.long(), 1, positions // self.size)
        return (page * self.size + positions % self.size).reshape(-1)

    def __call__(self, y, positions, slots, q_start, kv_len, longest):
        n, hq, hk, dim = len(y), self.hq, self.hk, self.dim
        qkv = y @ self.w.T
        st = qkv.stride(0)
        k, v = qkv[:, hq * dim:], qkv[:, (hq + hk) * dim:]
        hc.hc_qk_norm_rope(qkv, st, k, st, self.qw, self.kw, positions, hc.rope(self.table, dim), n, hc.heads(hq, hk, dim), qkv, st, k, st)
        hc.hc_kv_write(k, st, v, st, slots, n, self.shape, self.cache)
        a = hc.attention(n, self.seqs, longest, self.pages.shape[1], hq, dim ** -0.5)
        out = torch.empty((n, hq * dim), dtype=torch.bfloat16, device="cuda")
        hc.hc_kv_attention(qkv, st, q_start, kv_len, self.pages, self.cache, a, self.shape, out, hq * dim, None, self.ws)
        return out @ self.o.T, out


def _hc_sublayer_params(d, seed):
    from hyper_connection_residual_hc_gb300 import synth
    w = synth.small("step_b1_t64", 1, 8, d, seed=seed)
    return gu.DevParams(synth.params(w, 0), d), gu.shape_of(w)


def test_run_together_prefill_then_captured_decode():
    """hc_expand_pre_step, the attention sublayer, hc_post_then_pre: a prefill of 37 tokens for 3 sequences, then 12 decode
    steps replayed from one captured graph. The whole, run eagerly in one piece with all 49 tokens at once, is the same up to
    the order of sums; each step's attention is held to its bound against the 64-bit form on the cache that the GPU holds."""
    seqs, pre, steps, d = 3, 37, 12, 512
    sub = Sublayer(seqs, 16, 4, seed=3, d=d)
    P0, s = _hc_sublayer_params(d, 31)
    P1, _ = _hc_sublayer_params(d, 32)
    total = pre + steps
    h = torch.randn((seqs, total, d), generator=torch.Generator(device="cuda").manual_seed(4), device="cuda", dtype=torch.bfloat16)
    hws = hc.new_workspace()

    class Buffers:
        def __init__(self, n):
            e = lambda *sh, t=torch.float32: torch.empty(sh, dtype=t, device="cuda")  # noqa: E731
            b = torch.bfloat16
            self.n, self.h = n, e(n, d, t=b)
            self.X, self.X2, self.y, self.y2 = e(n, 4, d, t=b), e(n, 4, d, t=b), e(n, d, t=b), e(n, d, t=b)
            self.c = [e(n, 4), e(n, 4), e(n, 4, 4)]
            self.c2 = [e(n, 4), e(n, 4), e(n, 4, 4)]
            self.pos, self.slots = e(1, n, t=torch.int64), e(n, t=torch.int64)
            self.kv_len = e(seqs, t=torch.int32)
            self.q_start = torch.arange(0, n + 1, n // seqs, dtype=torch.int32, device="cuda")

        def set(self, a, b):
            self.h.copy_(h[:, a:b].reshape(-1, d))
            p = torch.arange(a, b, device="cuda").expand(seqs, -1).contiguous()
            self.pos.copy_(p.reshape(1, -1))
            self.slots.copy_(sub.slots(p))
            self.kv_len.fill_(b)

        def run(self):
            n = self.n
            hc.hc_expand_pre_step(self.h, P0.c, n, s, self.X, self.y, *self.c, hws)
            self.delta, self.att = sub(self.y, self.pos, self.slots, self.q_start, self.kv_len, n // seqs)
            hc.hc_post_then_pre(self.delta, self.X, self.c[1], self.c[2], self.c[0], P1.c, n, s, self.X2, self.y2, *self.c2, hws)

    pf = Buffers(seqs * pre)
    pf.set(0, pre)
    pf.run()
    dec = Buffers(seqs)
    dec.set(pre, pre + 1)
    dec.run()  # warm
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dec.run()
    ref_cache = ar.Cache(seqs * 4, 16, sub.hk, sub.dim)
    atts = []
    for t in range(pre, total):
        dec.set(t, t + 1)
        g.replay()
        torch.cuda.synchronize()
        atts.append(dec.att.clone())
        # the attention of this step in 64 bits, on the GPU's own queries and cache
        qkv = dec.y @ sub.w.T
        q = gu.guarded((seqs, sub.hq, sub.dim))
        hc.hc_qk_norm_rope(qkv, qkv.stride(0), None, 0, sub.qw, None, dec.pos, hc.rope(sub.table, sub.dim), seqs, hc.heads(sub.hq, 0, sub.dim), q,
                           sub.hq * sub.dim, None, 0)
        ref_cache.bytes = sub.cache.cpu().numpy().reshape(ref_cache.bytes.shape)
        ref, _, tol, _ = ar.attention(f64(q), np.arange(seqs + 1), [t + 1] * seqs, sub.pages.cpu().numpy(), ref_cache, sub.dim ** -0.5)
        assert (np.abs(f64(dec.att).reshape(ref.shape) - ref) <= tol).all(), t
    y_decode, cache_decode = dec.y2.clone(), sub.cache.clone()
    whole = Buffers(seqs * total)
    whole.set(0, total)
    whole.run()
    # A key or value that rounds the other way may take another code, half a step of 4 bits off; few do, and a query averages over 49.
    att = whole.att.reshape(seqs, total, -1)
    for i, a in enumerate(atts):
        b = att[:, pre + i].float()
        assert float((a.float() - b).norm() / b.norm()) < 0.05
    assert float((sub.cache != cache_decode).float().mean()) < 0.02
    last = whole.y2.reshape(seqs, total, d)[:, -1].float()
    assert float((y_decode.float() - last).norm() / last.norm()) < 0.05
    gu.device_error_clear()
