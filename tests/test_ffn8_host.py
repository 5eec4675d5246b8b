"""The 8-bit operators of the feed-forward sublayer and the head where no GPU is needed: argument checks (fake device addresses that are
never dereferenced: each call returns from its checks, or is a no-op) and the 64-bit reference itself against hand-worked values."""

import os
import subprocess

import numpy as np
import pytest

import hyper_connection_residual_hc_gb300 as hc
from hyper_connection_residual_hc_gb300 import build as hcbuild

import ffn_ref as fr

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


def test_norm_quant_refusals():
    n, d = 8, 144
    q = lambda **c: hc.quant8(**{**dict(n=n, d=d), **c})  # noqa: E731
    ok = [A[0], 144, A[1], 144, A[2], q(), A[3], 144, A[4], 144, A[5], 0]
    f = hc.hc_norm_quant8
    f(*_with(ok, _5=q(n=0)))  # no rows: a no-op
    f(*_with(ok, _2=None, _4=None, _5=q(n=0), _6=None))
    for i in (0, 2, 8, 10):  # (without the residual there is no sum)
        _expect(hc.HC_ERR_NULL, f, *_with(ok, **{"_%d" % i: None}))
    for bad in (dict(n=-1), dict(n=1 << 31), dict(d=0), dict(d=8), dict(d=136), dict(d=65552), dict(d=-16)):
        _expect(hc.HC_ERR_SHAPE, f, *_with(ok, _5=q(**bad)))
    for i, by in ((1, 8), (3, 8), (7, 8), (9, 16)):
        _expect(hc.HC_ERR_SHAPE, f, *_with(ok, **{"_%d" % i: ok[i] - by}))
        _expect(hc.HC_ERR_SHAPE, f, *_with(ok, **{"_%d" % i: ok[i] + by // 2}))
        _expect(hc.HC_ERR_SHAPE, f, *_with(ok, **{"_%d" % i: (1 << 37) + by}))
        f(*_with(ok, **{"_%d" % i: ok[i] + by, "_5": q(n=0)}))
    for eps in (-1e-6, float("nan"), float("inf")):
        _expect(hc.HC_ERR_ARG, f, *_with(ok, _5=q(norm_eps=eps)))
    for i in (0, 2, 4, 6, 8):
        _expect(hc.HC_ERR_ALIGN, f, *_with(ok, **{"_%d" % i: ok[i] + 8}))
    _expect(hc.HC_ERR_ALIGN, f, *_with(ok, _10=A[5] + 2))
    for i in (6, 8, 10):  # outputs on inputs and on each other
        for j in (0, 2, 4, 6, 8, 10):
            if i != j and not (i == 6 and j in (0, 2)):
                _expect(hc.HC_ERR_ALIAS, f, *_with(ok, **{"_%d" % i: ok[j]}))
    _expect(hc.HC_ERR_ALIAS, f, *_with(ok, _6=A[0] + 16))
    _expect(hc.HC_ERR_ALIAS, f, *_with(ok, _6=A[0], _7=152))
    _expect(hc.HC_ERR_ALIAS, f, *_with(ok, _6=A[1] + 32))
    f(*_with(ok, _6=A[0], _5=q(n=0)))


def test_mul_refusals():
    s = lambda **c: hc.mul8(**{**dict(features=200, k=272), **c})  # noqa: E731
    ok = [A[0], 272, A[1], A[2], 288, A[3], 5, s(), A[4], 200, 0]
    f = hc.hc_mul8
    f(*_with(ok, _6=0))
    for i in (0, 2, 3, 5, 8):
        _expect(hc.HC_ERR_NULL, f, *_with(ok, **{"_%d" % i: None}))
    for n in (-1, 1 << 31):
        _expect(hc.HC_ERR_SHAPE, f, *_with(ok, _6=n))
    for bad in (dict(features=0), dict(features=(1 << 24) + 1), dict(k=0), dict(k=8), dict(k=264), dict(k=(1 << 20) + 16), dict(k=-16)):
        _expect(hc.HC_ERR_SHAPE, f, *_with(ok, _7=s(**bad)))
    for i, by in ((1, 16), (4, 32), (9, 8)):
        _expect(hc.HC_ERR_SHAPE, f, *_with(ok, **{"_%d" % i: ok[i] - by}))
        _expect(hc.HC_ERR_SHAPE, f, *_with(ok, **{"_%d" % i: ok[i] + 4}))
        _expect(hc.HC_ERR_SHAPE, f, *_with(ok, **{"_%d" % i: (1 << 37) + 32}))
    for t in (hc.HC_E4M3, 3, -1):
        _expect(hc.HC_ERR_ARG, f, *_with(ok, _7=s(out_type=t)))
    for i in (0, 3, 8):
        _expect(hc.HC_ERR_ALIGN, f, *_with(ok, **{"_%d" % i: ok[i] + 8}))
    for i in (2, 5):
        _expect(hc.HC_ERR_ALIGN, f, *_with(ok, **{"_%d" % i: ok[i] + 2}))
    for i in (0, 2, 3, 5):
        _expect(hc.HC_ERR_ALIAS, f, *_with(ok, _8=ok[i]))
    # the last byte of the weights, and the one behind it
    end = A[2] + 199 * 288 + 272
    _expect(hc.HC_ERR_ALIAS, f, *_with(ok, _8=end - 16))
    f(*_with(ok, _8=end, _6=0))


def test_gated_refusals():
    s = lambda **c: hc.gated8(**{**dict(features=208, k=272), **c})  # noqa: E731
    ok = [A[0], 272, A[1], A[2], A[3], A[4], A[5], 288, 5, s(), A[6], 208, A[7], 0]
    f = hc.hc_gated_mul8
    f(*_with(ok, _8=0))
    f(*_with(ok, _8=0, _9=s(out_type=hc.HC_BF16), _12=None))
    for i in (0, 2, 3, 4, 5, 6, 10, 12):
        _expect(hc.HC_ERR_NULL, f, *_with(ok, **{"_%d" % i: None}))
    for bad in (dict(features=0), dict(features=200), dict(features=(1 << 24) + 16), dict(k=0), dict(k=280), dict(k=(1 << 20) + 16)):
        _expect(hc.HC_ERR_SHAPE, f, *_with(ok, _9=s(**bad)))
    for i, by in ((1, 16), (7, 32), (11, 16)):
        _expect(hc.HC_ERR_SHAPE, f, *_with(ok, **{"_%d" % i: ok[i] - by}))
        _expect(hc.HC_ERR_SHAPE, f, *_with(ok, **{"_%d" % i: ok[i] + 8}))
    for bad in (dict(out_type=hc.HC_F32), dict(out_type=7), dict(act=2), dict(act=-1)):
        _expect(hc.HC_ERR_ARG, f, *_with(ok, _9=s(**bad)))
    for i in (0, 3, 5, 10):
        _expect(hc.HC_ERR_ALIGN, f, *_with(ok, **{"_%d" % i: ok[i] + 8}))
    for i in (2, 4, 6, 12):
        _expect(hc.HC_ERR_ALIGN, f, *_with(ok, **{"_%d" % i: ok[i] + 2}))
    for o in (10, 12):
        for i in (0, 2, 3, 4, 5, 6, 10, 12):
            if i != o:
                _expect(hc.HC_ERR_ALIAS, f, *_with(ok, **{"_%d" % o: ok[i]}))
    # gate and up as halves of one matrix, or as columns of one
    f(*_with(ok, _8=0, _5=A[2] + 208 * 288))
    f(*_with(ok, _8=0, _5=A[2] + 272, _7=544))


def test_logprob_refusals():
    s = lambda **c: hc.logprobs(**{**dict(n=6, vocab=100, top=4), **c})  # noqa: E731
    ok = [A[0], 104, A[1], s(), A[2], A[3], A[4], A[5], 0]
    f = hc.hc_token_logprobs
    f(*_with(ok, _3=s(n=0)))
    f(*_with(ok, _3=s(n=0, top=0), _6=None, _7=None))
    f(*_with(ok, _3=s(n=0), _2=None, _4=None, _5=None))  # alternatives alone
    for i in (0, 2, 6, 7):
        _expect(hc.HC_ERR_NULL, f, *_with(ok, **{"_%d" % i: None}))
    _expect(hc.HC_ERR_NULL, f, *_with(ok, _3=s(top=0), _4=None, _5=None))
    for bad in (dict(n=-1), dict(n=1 << 31), dict(vocab=0), dict(vocab=(1 << 30) + 1), dict(top=-1), dict(top=101), dict(vocab=3)):
        _expect(hc.HC_ERR_SHAPE, f, *_with(ok, _3=s(**bad)))
    _expect(hc.HC_ERR_UNSUPPORTED, f, *_with(ok, _3=s(top=33)))
    for stride in (96, 108, 1 << 38):
        _expect(hc.HC_ERR_SHAPE, f, *_with(ok, _1=stride))
    for bad in (dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=2.0 ** -65), dict(scale=2.0 ** 65), dict(type=hc.HC_E4M3), dict(type=-1)):
        _expect(hc.HC_ERR_ARG, f, *_with(ok, _3=s(**bad)))
    _expect(hc.HC_ERR_ALIGN, f, *_with(ok, _0=A[0] + 8))
    _expect(hc.HC_ERR_ALIGN, f, *_with(ok, _2=A[1] + 4))
    for i in (4, 5, 6, 7):
        _expect(hc.HC_ERR_ALIGN, f, *_with(ok, **{"_%d" % i: ok[i] + 2}))
        for j in (0, 2, 4, 5, 6, 7):
            if i != j:
                _expect(hc.HC_ERR_ALIAS, f, *_with(ok, **{"_%d" % i: ok[j]}))


def test_products_go_to_the_kernel_that_can_run(tmp_path):
    """The choice between the two kernels of the products: the shorter one, and the one for few rows where the other cannot be planned."""
    csrc = os.path.join(os.path.dirname(hc.__file__), "csrc")
    src = tmp_path / "choice.cu"
    src.write_text("""
#include "hc_mul8_host.h"
static_assert(hc::mul8_by_pairs(10, 11) && hc::mul8_by_pairs(0, 1), "the shorter one");
static_assert(!hc::mul8_by_pairs(11, 11) && !hc::mul8_by_pairs(12, 11), "the shorter one");
static_assert(!hc::mul8_by_pairs(-1, 11), "no plan: the other kernel");
""")
    subprocess.run([hcbuild.NVCC, "-std=c++17", "-I", csrc, "-c", str(src), "-o", str(tmp_path / "choice.o")], check=True)


# ---- the reference ----------------------------------------------------------------------------------------

def test_codes_have_the_formats_values():
    v = fr.e4m3_values()
    assert v[0] == 0 and v[1] == 2.0 ** -9 and v[7] == 7 / 512 and v[8] == 2.0 ** -6 and v[0x38] == 1 and v[0x7E] == 448 and np.isnan(v[0x7F])
    assert v[0xB8] == -1 and v[0xFE] == -448
    torch = pytest.importorskip("torch")
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(t, v.astype(np.float32), equal_nan=True)


def test_quantised_and_products_by_hand():
    y = np.zeros((1, 130))
    y[0, 0], y[0, 127], y[0, 128] = -896.0, 2.0, 1e-30
    q, s = fr.quantised(y)
    assert np.array_equal(s, [[2.0, 2.0 ** -64 / 448]])
    assert q[0, 0] == -448 and q[0, 127] == 1 and q[0, 128] == 1e-30 / s[0, 1]
    x, w = np.ones((1, 144)), np.ones((129, 144))
    out, bound = fr.product(x, np.array([[2.0, 10.0]]), w, np.array([[1.0, 0.5], [3.0, 0.25]]))
    assert out[0, 0] == 2 * 128 + 10 * 0.5 * 16 and out[0, 128] == 6 * 128 + 2.5 * 16 and bound[0, 0] < 1e-4 * out[0, 0]
    g, _ = fr.gated(x, np.array([[1 / 128, 0.0]]), w[:1], np.ones((1, 2)), 2 * w[:1], np.ones((1, 2)), "silu")
    assert abs(g[0, 0] - 2 / (1 + np.exp(-1))) < 1e-12
    assert abs(fr.act(np.array(1.0), "gelu") - 0.5 * (1 + np.tanh(0.7978845608028654 * 1.044715))) < 1e-12


def test_logprobs_by_hand():
    x = np.log(np.array([[1.0, 2.0, 1.0], [1.0, 0.0, 0.0]]) + 0.0, where=np.array([[True] * 3, [True, False, False]]), out=np.full((2, 3), -np.inf))
    lp, h, tl, tt, _, _ = fr.logprobs(x, np.array([1, 0]), 1.0, 3)
    assert np.allclose(lp, [np.log(0.5), 0]) and np.allclose(h, [1.5 * np.log(2), 0])
    assert np.array_equal(tt, [[1, 0, 2], [0, 1, 2]]) and np.allclose(tl[0], np.log([0.5, 0.25, 0.25])) and np.isneginf(tl[1, 1:]).all()
    lp, h, tl, _, _, _ = fr.logprobs(np.full((1, 4), -np.inf), np.array([2]), 1.0, 2)
    assert np.isneginf(lp).all() and h[0] == 0 and np.isneginf(tl).all()
