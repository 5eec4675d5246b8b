"""The attention sublayer's operators where no GPU is needed: argument checks (fake device addresses that
are never dereferenced: each call returns from its checks, or is a no-op), sizes, and the 64-bit reference
itself (byte layout and quantisation) against hand-worked values."""

import ctypes

import numpy as np
import pytest

import hyper_connection_residual_hc_gb300 as hc
from hyper_connection_residual_hc_gb300 import build as hcbuild

import attn_ref as ar

A = [0x7F0000000000 + i * (1 << 36) for i in range(16)]


@pytest.fixture(scope="module", autouse=True)
def lib():
    hcbuild.build()
    return hc.load()


def _expect(status, fn, *args):
    with pytest.raises(hc.HCError) as e:
        fn(*args)
    assert e.value.status == status, (e.value.status, status)


def _with(args, **changes):
    out = list(args)
    for k, v in changes.items():
        out[int(k[1:])] = v
    return out


# ---- sizes ------------------------------------------------------------------------------------------

def test_sizes():
    assert hc.hc_rope_table_size(128) == 64 * 16 and hc.hc_rope_table_size(0) == 0
    for rot in (-16, 8, 272):
        _expect(hc.HC_ERR_SHAPE, hc.hc_rope_table_size, rot)
    assert hc.hc_kv_cache_size(hc.kv_shape(3, 64, 8, 128)) == 3 * 64 * 8 * 128 * 9 // 8
    # past 2^32 bytes
    assert hc.hc_kv_cache_size(hc.kv_shape(100000, 128, 8, 128)) == 100000 * 128 * 8 * 128 * 9 // 8
    assert hc.hc_kv_workspace_size() == 512 * 4 + 256 * 256 * 130 * 4 == 34080768


@pytest.mark.parametrize("bad,status", [
    (dict(pages=0), hc.HC_ERR_SHAPE), (dict(page_size=48), hc.HC_ERR_SHAPE), (dict(page_size=8), hc.HC_ERR_SHAPE),
    (dict(page_size=2048), hc.HC_ERR_SHAPE), (dict(heads=0), hc.HC_ERR_SHAPE), (dict(heads=1025), hc.HC_ERR_SHAPE),
    (dict(dim=0), hc.HC_ERR_SHAPE), (dict(dim=96), hc.HC_ERR_UNSUPPORTED), (dict(k_scale=3.0), hc.HC_ERR_ARG),
    (dict(k_scale=0.0), hc.HC_ERR_ARG), (dict(v_scale=-1.0), hc.HC_ERR_ARG), (dict(v_scale=float("nan")), hc.HC_ERR_ARG),
    (dict(v_scale=float("inf")), hc.HC_ERR_ARG), (dict(k_scale=2.0 ** 41), hc.HC_ERR_ARG),
])
def test_cache_shape_refusals(bad, status):
    s = hc.kv_shape(**{**dict(pages=4, page_size=64, heads=8, dim=128), **bad})
    _expect(status, hc.hc_kv_cache_size, s)
    _expect(status, hc.hc_kv_write, A[0], 1024, A[1], 1024, A[2], 4, s, A[3], 0)
    _expect(status, hc.hc_kv_read, A[3], A[2], 4, s, A[0], 1024, A[1], 1024, 0)
    a = hc.attention(4, 1, 4, 2, 8, 1.0)
    _expect(status, hc.hc_kv_attention, A[0], 1024, A[1], A[2], A[3], A[4], a, s, A[5], 1024, None, A[6], 0)


# ---- refusals -----------------------------------------------------------------------------------------

def test_prepare_rope_refusals():
    f = [1.0] * 8
    _expect(hc.HC_ERR_NULL, hc.hc_prepare_rope, None, None, 16, 1, A[0], 0)
    _expect(hc.HC_ERR_NULL, hc.hc_prepare_rope, f, None, 16, 1, None, 0)
    _expect(hc.HC_ERR_SHAPE, hc.hc_prepare_rope, [], None, 0, 1, A[0], 0)
    _expect(hc.HC_ERR_SHAPE, hc.hc_prepare_rope, f + f[:4], None, 24, 1, A[0], 0)
    _expect(hc.HC_ERR_SHAPE, hc.hc_prepare_rope, f, None, 16, 5, A[0], 0)
    _expect(hc.HC_ERR_ALIGN, hc.hc_prepare_rope, f, None, 16, 1, A[0] + 8, 0)
    _expect(hc.HC_ERR_ARG, hc.hc_prepare_rope, f, [0] * 7 + [2], 16, 2, A[0], 0)
    _expect(hc.HC_ERR_ARG, hc.hc_prepare_rope, f, [-1] + [0] * 7, 16, 2, A[0], 0)
    _expect(hc.HC_ERR_ARG, hc.hc_prepare_rope, f[:7] + [float("inf")], None, 16, 1, A[0], 0)
    with pytest.raises(ValueError):
        hc.hc_prepare_rope(f[:7], None, 16, 1, A[0], 0)


def test_norm_rope_refusals():
    hq, hk, d = 4, 2, 64
    r, s = hc.rope(A[7], 64), hc.heads(hq, hk, d)
    ok = [A[0], 256, A[1], 128, A[2], A[3], A[4], r, 8, s, A[5], 256, A[6], 128, 0]
    f = hc.hc_qk_norm_rope
    f(*_with(ok, _8=0))  # no rows: a no-op
    for i in (0, 2, 6, 10, 12):
        _expect(hc.HC_ERR_NULL, f, *_with(ok, **{"_%d" % i: None}))
    _expect(hc.HC_ERR_NULL, f, *_with(ok, _7=hc.rope(None, 64)))
    f(*_with(ok, _8=0, _4=None, _5=None, _6=None, _7=hc.rope(None, 0)))               # no gains, no rotation
    f(*_with(ok, _8=0, _2=None, _12=None, _3=0, _13=0, _9=hc.heads(hq, 0, d)))        # queries only
    _expect(hc.HC_ERR_SHAPE, f, *_with(ok, _8=-1))
    for i in (1, 3, 11, 13):
        _expect(hc.HC_ERR_SHAPE, f, *_with(ok, **{"_%d" % i: ok[i] - 8}))   # narrower than a row
        _expect(hc.HC_ERR_SHAPE, f, *_with(ok, **{"_%d" % i: ok[i] + 4}))   # rows off 16 bytes
    for h in (hc.heads(0, hk, d), hc.heads(hq, -1, d), hc.heads(hq, hk, 60), hc.heads(hq, hk, 0)):
        _expect(hc.HC_ERR_SHAPE, f, *_with(ok, _9=h))
    _expect(hc.HC_ERR_UNSUPPORTED, f, *_with(ok, _9=hc.heads(hq, hk, 264), _1=2048, _3=2048, _11=2048, _13=2048))
    for rr in (hc.rope(A[7], 72), hc.rope(A[7], -16), hc.rope(A[7], 80), hc.rope(A[7], 48, 24), hc.rope(A[7], 32, 4),
               hc.rope(A[7], 32, -8), hc.rope(A[7], 64, 0, 0), hc.rope(A[7], 64, 0, 5)):
        _expect(hc.HC_ERR_SHAPE, f, *_with(ok, _7=rr))
    _expect(hc.HC_ERR_ARG, f, *_with(ok, _7=hc.rope(A[7], 64, style=2)))
    _expect(hc.HC_ERR_ARG, f, *_with(ok, _9=hc.heads(hq, hk, d, float("nan"))))
    for i in (0, 2, 4, 5, 10, 12):
        _expect(hc.HC_ERR_ALIGN, f, *_with(ok, **{"_%d" % i: ok[i] + 8}))
    _expect(hc.HC_ERR_ALIGN, f, *_with(ok, _6=A[4] + 4))
    # in place is allowed, shifted or with another stride it is not; nor are outputs on other arguments
    f(*_with(ok, _8=0, _10=A[0], _12=A[1]))
    _expect(hc.HC_ERR_ALIAS, f, *_with(ok, _10=A[0] + 16))
    _expect(hc.HC_ERR_ALIAS, f, *_with(ok, _10=A[0], _11=264))
    _expect(hc.HC_ERR_ALIAS, f, *_with(ok, _10=A[1]))
    _expect(hc.HC_ERR_ALIAS, f, *_with(ok, _12=A[5] + 64))
    _expect(hc.HC_ERR_ALIAS, f, *_with(ok, _10=A[4] - 64))
    _expect(hc.HC_ERR_ALIAS, f, *_with(ok, _12=A[7]))
    _expect(hc.HC_ERR_ALIAS, f, *_with(ok, _12=A[3] - 1024))
    # q and k in place as columns of one buffer lie side by side; one column further they meet
    fused = _with(ok, _1=512, _2=A[0] + 512, _3=512, _10=A[0], _11=512, _12=A[0] + 512, _13=512)
    f(*_with(fused, _8=0))
    _expect(hc.HC_ERR_ALIAS, f, *_with(fused, _2=A[0] + 496, _12=A[0] + 496))


def test_kv_move_refusals():
    s = hc.kv_shape(4, 64, 8, 128)
    ok = [A[0], 1024, A[1], 1024, A[2], 4, s, A[3], 0]
    w = hc.hc_kv_write
    w(*_with(ok, _5=0))
    for i in (0, 2, 4, 7):
        _expect(hc.HC_ERR_NULL, w, *_with(ok, **{"_%d" % i: None}))
    _expect(hc.HC_ERR_SHAPE, w, *_with(ok, _5=-1))
    _expect(hc.HC_ERR_SHAPE, w, *_with(ok, _5=1 << 31))
    _expect(hc.HC_ERR_SHAPE, w, *_with(ok, _1=1016))
    _expect(hc.HC_ERR_SHAPE, w, *_with(ok, _3=1028))
    for i in (0, 2, 7):
        _expect(hc.HC_ERR_ALIGN, w, *_with(ok, **{"_%d" % i: ok[i] + 8}))
    _expect(hc.HC_ERR_ALIGN, w, *_with(ok, _4=A[2] + 4))
    for i in (0, 2, 4):
        _expect(hc.HC_ERR_ALIAS, w, *_with(ok, **{"_%d" % i: A[3] + 32}))
    ok = [A[3], A[2], 4, s, A[0], 1024, A[1], 1024, 0]
    r = hc.hc_kv_read
    r(*_with(ok, _2=0))
    r(*_with(ok, _2=0, _4=None, _5=0))
    _expect(hc.HC_ERR_NULL, r, *_with(ok, _4=None, _6=None))
    _expect(hc.HC_ERR_NULL, r, *_with(ok, _0=None))
    _expect(hc.HC_ERR_NULL, r, *_with(ok, _1=None))
    _expect(hc.HC_ERR_SHAPE, r, *_with(ok, _2=-1))
    _expect(hc.HC_ERR_SHAPE, r, *_with(ok, _5=1000))
    _expect(hc.HC_ERR_SHAPE, r, *_with(ok, _7=0))
    _expect(hc.HC_ERR_ALIGN, r, *_with(ok, _4=A[0] + 2))
    _expect(hc.HC_ERR_ALIAS, r, *_with(ok, _4=A[3]))
    _expect(hc.HC_ERR_ALIAS, r, *_with(ok, _6=A[2] - 1024))
    _expect(hc.HC_ERR_ALIAS, r, *_with(ok, _6=A[0] + 2048))
    r(*_with(ok, _2=0, _5=2048, _7=2048, _6=A[0] + 2048))  # two column ranges of one buffer


def test_attention_refusals():
    s, n = hc.kv_shape(4, 64, 8, 128), 4
    a = dict(n=n, seqs=2, max_q_len=2, max_pages=2, q_heads=40, scale=0.1)
    mk = lambda **k: hc.attention(**{**a, **k})  # noqa: E731
    ok = [A[0], 5120, A[1], A[2], A[3], A[4], mk(), s, A[5], 5120, A[6], A[7], 0]
    f = hc.hc_kv_attention
    f(*_with(ok, _6=mk(n=0)))
    f(*_with(ok, _6=mk(seqs=0)))
    for i in (0, 2, 3, 4, 5, 8, 11):
        _expect(hc.HC_ERR_NULL, f, *_with(ok, **{"_%d" % i: None}))
    for k in (dict(n=-1), dict(n=1 << 31), dict(seqs=-1), dict(max_q_len=-1), dict(max_pages=0), dict(q_heads=0), dict(q_heads=41),
              dict(q_heads=8 * 129), dict(max_pages=1 << 25), dict(max_pages=(1 << 24) + 1), dict(seqs=(1 << 24) + 1)):
        _expect(hc.HC_ERR_SHAPE, f, *_with(ok, _6=mk(**k), _1=1 << 18, _9=1 << 18))
    _expect(hc.HC_ERR_SHAPE, f, *_with(ok, _1=5112))
    _expect(hc.HC_ERR_SHAPE, f, *_with(ok, _9=5124))
    for k in (dict(scale=float("nan")), dict(scale=-1.0), dict(window=-1), dict(window=5, causal=False)):
        _expect(hc.HC_ERR_ARG, f, *_with(ok, _6=mk(**k)))
    for i in (0, 5, 8, 11):
        _expect(hc.HC_ERR_ALIGN, f, *_with(ok, **{"_%d" % i: ok[i] + 8}))
    for i in (2, 3, 4, 10):
        _expect(hc.HC_ERR_ALIGN, f, *_with(ok, **{"_%d" % i: ok[i] + 2}))
    for i in (0, 1, 2, 3, 4, 6, 7):  # out on each other argument in turn
        j = {0: 0, 1: 2, 2: 3, 3: 4, 4: 5, 6: 10, 7: 11}[i]
        _expect(hc.HC_ERR_ALIAS, f, *_with(ok, _8=ok[j]))
    _expect(hc.HC_ERR_ALIAS, f, *_with(ok, _10=A[4] + 64))
    _expect(hc.HC_ERR_ALIAS, f, *_with(ok, _10=A[0] + 64))
    _expect(hc.HC_ERR_ALIAS, f, *_with(ok, _11=A[4] - 1024))
    _expect(hc.HC_ERR_ALIAS, f, *_with(ok, _11=A[3] - 1024))


# ---- the reference itself -----------------------------------------------------------------------------

@pytest.mark.parametrize("dim", [64, 128, 256])
def test_layout_places_are_a_permutation(dim):
    """Every byte of a block has exactly one place: codes two columns a byte, scales 16 columns a byte."""
    t, i = np.arange(16)[:, None], np.arange(0, dim, 2)[None]
    s = np.arange(0, dim, 16)[None]
    at = np.concatenate([ar.key_code_byte(t, i, dim).ravel(), ar.key_scale_byte(t, s, dim).ravel(),
                         ar.value_code_byte(t, i, dim).ravel(), ar.value_scale_byte(t, s, dim).ravel()])
    assert sorted(at) == list(range(18 * dim))
    assert (ar.key_code_byte(t, i, dim) == ar.key_code_byte(t, i + 1, dim)).all()
    assert (ar.value_code_byte(t, i, dim) == ar.value_code_byte(t, i + 1, dim)).all()
    assert len({int(ar.key_scale_byte(3, x, dim)) for x in range(16, 32)}) == 1


def test_quantise_by_hand():
    x = np.zeros(32)
    # scale 6 / 6 = 1: each value is its own quotient; ties go to the even code
    x[:16] = [6, -6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, 0.26, 4.9, 5.1, 0, -0.0]
    code, byte = ar.quantise(x, 1.0)
    assert byte.tolist() == [56, 0]  # 1.0 in e4m3; a group of zeros
    assert code[:16].tolist() == [7, 15, 0, 2, 2, 4, 4, 6, 6, 8, 10, 1, 6, 7, 0, 8]
    assert code[16:].tolist() == [0] * 16
    # scales: 448 is the largest; a tie between two scales goes to the even one (17 / 16 lies between 1 and 1.125)
    assert ar.quantise(np.full(16, 1e6), 1.0)[1][0] == 126
    assert ar.quantise(np.full(16, 6 * 17 / 16), 1.0)[1][0] == 56
    assert ar.quantise(np.full(16, 6 * 19 / 16), 1.0)[1][0] == 58
    assert ar.quantise(np.full(16, 6 * 2.0 ** -10), 1.0)[1][0] == 0 and ar.quantise(np.full(16, 6 * 2.0 ** -9), 1.0)[1][0] == 1
    assert ar.quantise(np.full(16, 12.0), 2.0)[1][0] == 56
    assert ar.quantise(np.array([np.inf] + [1.0] * 15), 1.0)[1][0] == 127
    v = ar.values(code, byte, 1.0)
    assert v[:9].tolist() == [6, -6, 0, 1, 1, 2, 2, 4, 4] and np.isnan(ar.values(code, np.array([127, 0]), 1.0)[:16]).all()


def test_reference_attention_of_one_key_and_none():
    c = ar.Cache(2, 16, 1, 64)
    rng = np.random.default_rng(1)
    k, v = ar.bf16(rng.standard_normal((3, 1, 64))), ar.bf16(rng.standard_normal((3, 1, 64)))
    c.write(k, v, [16, 17, 18])
    q = ar.bf16(rng.standard_normal((3, 2, 64)))
    out, lse, _, _ = ar.attention(q, [0, 3], [2], [[1]], c, 0.125)
    K, V = c.read([16, 17])
    assert (out[0] == 0).all() and np.isneginf(lse[0]).all()      # position -1: no key
    assert np.allclose(out[1], V[0]) and np.allclose(lse[1], 0.125 * q[1] @ K[0, 0])  # position 0: its own key alone
    z = 0.125 * (K[:, 0] @ q[2, 1])
    w = np.exp(z) / np.exp(z).sum()
    assert np.allclose(out[2, 1], w @ V[:, 0])


def test_angle_by_fixed_point_turns():
    """The table's arithmetic: position * round(2^64 f / 2 pi) modulo 2^64, read as a signed fraction of a turn."""
    for f in (1.0, 10000.0 ** -0.5, 10000.0 ** (-126 / 128), 3.7):
        import math
        turns = f / (2 * math.pi)
        fixed = int((turns - math.floor(turns)) * 2 ** 64) % 2 ** 64
        for pos in (0, 1, 65535, (1 << 20) + 7, -5, -(1 << 20)):
            wrapped = pos * fixed % 2 ** 64
            wrapped -= 2 ** 64 if wrapped >= 2 ** 63 else 0
            got = 2 * math.pi * wrapped / 2.0 ** 64
            assert abs(math.sin(got) - math.sin(pos * f)) < 1e-8 and abs(math.cos(got) - math.cos(pos * f)) < 1e-8


def test_symbols_are_bound():
    lib = hc.load()
    for name in ("hc_rope_table_size", "hc_prepare_rope", "hc_qk_norm_rope", "hc_kv_cache_size", "hc_kv_write", "hc_kv_read",
                 "hc_kv_workspace_size", "hc_kv_attention"):
        assert name in hc.SYMBOLS and getattr(lib, name).restype is ctypes.c_int


def test_bench_counts_the_decode_step():
    """bench.py's attention step: lengths that span its range, and the bytes that the step cannot do without."""
    import os
    import sys
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    import bench
    lens = bench.attention_lengths()
    assert len(lens) == 256 and min(lens) == 2048 and max(lens) == 4096 and len(set(lens)) == 256
    # q 5120, k and v 1024 each, out 5120 columns of bf16 a token; 1152 bytes of keys and values of 8 heads a cached token
    assert bench.attention_step_bytes() == 256 * (2 * 5120 + 2 * 1024) * 2 + (sum(lens) + 256) * 2 * 576
