"""The 8-bit operators of the feed-forward sublayer and the head on the GPU against their plain 64-bit forms (ffn_ref, which derives
the bounds): rows quantised with and without residual and norm, products and gated products from one token to several tiles, log
probabilities with entropy and alternatives, their behaviour at the edges (short blocks, strides, masked logits, NaN, padding), other
streams, captured graphs, and a run of them together between two Hyper-Connection steps and behind the last one."""

import numpy as np
import pytest
import torch

import hyper_connection_residual_hc_gb300 as hc

import ffn_ref as fr
import gpu_util as gu

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    hc.load()
    gu.device_error_clear()
    yield
    gu.device_error_clear()


def f64(t):
    return t.double().cpu().numpy() if t.dtype != E4M3 else t.float().double().cpu().numpy()


def dev(x, dtype=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(x)).to(dtype).cuda()


def no_error():
    torch.cuda.synchronize()
    assert hc.hc_device_error(clear=True) == 0


def assert_within(got, ref, tol, what=""):
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.size, np.argwhere(bad)[:4], got[bad][:4], ref[bad][:4], np.broadcast_to(tol, ref.shape)[bad][:4])


def check_codes(codes, scales, y, e, what=""):
    """Codes and scales of y, known to within e: the scale follows the block's largest, a code the quotient."""
    top = fr.block_max(y)
    etop = np.stack([np.broadcast_to(e, y.shape)[:, i:i + 128].max(1) for i in range(0, y.shape[1], 128)], 1)
    assert_within(scales, np.maximum(top, 2.0 ** -64) / 448, (etop + 4 * fr.U * top) / 448 + 2.0 ** -96, what + " scales")
    s = fr.spread(scales, y.shape[1])
    q = y / s
    assert_within(codes, q, fr.half_step(q) * (1 + 2.0 ** -10) + e / s + 4 * fr.U * np.abs(q), what + " codes")


def strided(rows, cols, stride, dtype, fill=None):
    """A view [rows, cols] of a wider buffer, and the buffer."""
    buf = torch.empty((rows, stride), dtype=dtype, device="cuda") if fill is None else torch.full((rows, stride), fill, dtype=torch.float32, device="cuda").to(dtype)
    return buf[:, :cols], buf


# ---- norm and quantisation -----------------------------------------------------------------------------

@pytest.mark.parametrize("residual,normed,gains", [(False, False, False), (True, False, False), (False, True, False), (True, True, True)])
@pytest.mark.parametrize("n,d", [(1, 16), (3, 128), (5, 144), (7, 272), (130, 256), (4, 512), (3, 528), (9, 1040), (64, 5120), (33, 2000), (2, 32768),
                                 (2, 32784), (3, 65536)])
def test_norm_quant(n, d, residual, normed, gains):
    rng = np.random.default_rng(n * 131 + d)
    x = dev(rng.standard_normal((n, d)) * np.exp(rng.standard_normal((n, 1))), torch.bfloat16)
    r = dev(3 * rng.standard_normal((n, d)), torch.bfloat16) if residual else None
    w = dev(1 + 0.2 * rng.standard_normal(d)) if gains else None
    codes, scales = gu.guarded((n, d), E4M3), gu.guarded((n, fr.blocks(d)), torch.float32)
    out = gu.guarded((n, d)) if residual else None
    hc.hc_norm_quant8(x, d, r, d, w, hc.quant8(n, d, norm=normed), out, d, codes, d, scales)
    no_error()
    s = f64(x)
    if residual:
        total = x.float() + r.float()
        assert torch.equal(out, total.to(torch.bfloat16))
        s = f64(out)
    y, e = s, 0.0
    if normed:
        y = fr.norm(s, None if w is None else f64(w), 1e-6)
        e = (d / 2 + 16) * fr.U * np.abs(y)
    check_codes(f64(codes), f64(scales), y, e)


@pytest.mark.parametrize("place", ["x", "residual"])
def test_norm_quant_strided_in_place(place):
    rng = np.random.default_rng(5)
    n, d, stride = 37, 1200, 1608
    x, xb = strided(n, d, stride, torch.bfloat16, 7.0)
    r, rb = strided(n, d, stride, torch.bfloat16, 9.0)
    x.copy_(dev(rng.standard_normal((n, d)), torch.bfloat16))
    r.copy_(dev(rng.standard_normal((n, d)), torch.bfloat16))
    want = (x.float() + r.float()).to(torch.bfloat16)
    codes, cb = strided(n, d, 1216, E4M3, 3.0)
    scales = torch.empty((n, fr.blocks(d)), device="cuda")
    out = x if place == "x" else r
    hc.hc_norm_quant8(x, stride, r, stride, None, hc.quant8(n, d), out, stride, codes, 1216, scales)
    no_error()
    assert torch.equal(out, want)
    assert (xb[:, d:] == 7).all() and (rb[:, d:] == 9).all() and (cb[:, d:].float() == 3).all()
    y = fr.norm(f64(want), None, 1e-6)
    check_codes(f64(codes), f64(scales), y, (d / 2 + 16) * fr.U * np.abs(y))


def test_quant_edges():
    """Zeros, the largest and the smallest numbers, a block with NaN, one with infinity."""
    x = torch.zeros((6, 256), dtype=torch.bfloat16, device="cuda")
    x[1] = torch.finfo(torch.bfloat16).max
    x[1, 1] = -torch.finfo(torch.bfloat16).max
    x[2] = 2.0 ** -126
    x[3, 200] = float("nan")
    x[3, :128] = 1.0
    x[4, 3] = float("-inf")
    x[5] = -1e-3
    codes, scales = torch.empty((6, 256), dtype=E4M3, device="cuda"), torch.empty((6, 2), device="cuda")
    hc.hc_norm_quant8(x, 256, None, 0, None, hc.quant8(6, 256, norm=False), None, 0, codes, 256, scales)
    no_error()
    c, s = f64(codes), f64(scales)
    v = c * fr.spread(s, 256)
    assert (c[0] == 0).all() and np.allclose(s[0], 2.0 ** -64 / 448, rtol=4 * fr.U)
    assert c[1, 0] == 448 and c[1, 1] == -448
    assert (v[2] == 0).all()
    assert np.isnan(v[3, 128:]).all() and (c[3, :128] == 448).all()
    assert np.isnan(v[4, :128]).all() and (v[4, 128:] == 0).all()
    assert (c[5] == -448).all()


# The mean of squares in fp32: rounding a square or a scaled value that is subnormal costs at most 2^-126 of the row's largest. What the norm
# adds to that is as in test_norm_quant.
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("n,d", [(3, 256), (2, 512), (5, 1040), (3, 5120), (2, 32784)])
@pytest.mark.parametrize("kind,eps", [("largest", 1e-6), ("large", 1e-6), ("large", 0.0), ("one large", 1e-6), ("small", 0.0), ("small", 1e-40), ("small", 2.0 ** -99),
                                      ("small", 2.0 ** -101), ("smallest", 0.0), ("smallest", 1e-6), ("ordinary", 3e38), ("ordinary", 0.0), ("largest", 3e38)])
def test_norm_quant_ends_of_the_range(n, d, kind, eps, residual):
    """Finite rows are normed whether or not their squares fit into fp32."""
    rng = np.random.default_rng(d + n)
    x = rng.standard_normal((n, d))
    if kind == "largest":
        x = np.where(x > 0, 1.0, -1.0) * 2.0 ** 127 * (1 + rng.integers(0, 128, (n, d)) / 128)
    elif kind == "large":
        x *= 2.0 ** 70
    elif kind == "one large":
        x[:, d // 3] = 2.0 ** 110
    elif kind == "small":
        x *= 2.0 ** -100
    elif kind == "smallest":
        x = rng.integers(-3, 4, (n, d)) * 2.0 ** -133
    x = dev(x, torch.bfloat16)
    assert torch.isfinite(x).all()
    r = torch.zeros_like(x) if residual else None
    w = dev(1 + 0.2 * rng.standard_normal(d))
    codes, scales = gu.guarded((n, d), E4M3), gu.guarded((n, fr.blocks(d)), torch.float32)
    out = gu.guarded((n, d)) if residual else None
    q = hc.quant8(n, d, norm_eps=eps)
    hc.hc_norm_quant8(x, d, r, d, w, q, out, d, codes, d, scales)
    no_error()
    if residual:
        assert torch.equal(out, x)
    y = fr.norm(f64(x), f64(w), float(q.norm_eps))
    check_codes(f64(codes), f64(scales), y, (d / 2 + 16) * fr.U * np.abs(y) + 2.0 ** -110)


def test_norm_quant_zeros_and_infinities_beside_large_rows():
    x = torch.zeros((4, 512), dtype=torch.bfloat16, device="cuda")
    x[1] = 2.0 ** 100
    x[2, 300], x[2, 5] = float("inf"), 2.0 ** 100
    x[3, 7], x[3, 200] = float("nan"), 2.0 ** 100
    codes, scales = torch.empty((4, 512), dtype=E4M3, device="cuda"), torch.empty((4, 4), device="cuda")
    for eps in (1e-6, 0.0):
        hc.hc_norm_quant8(x, 512, None, 0, None, hc.quant8(4, 512, norm_eps=eps), None, 0, codes, 512, scales)
        no_error()
        c, s = f64(codes), f64(scales)
        assert np.isnan(c[0]).all() if eps == 0 else (c[0] == 0).all()
        assert (c[1] == 448).all() and np.allclose(s[1], 1 / 448, rtol=600 * fr.U)
        assert np.isnan(c[2, 256:384]).all() and (np.delete(c[2], np.s_[256:384]) == 0).all()
        assert np.isnan(c[3]).all()


# ---- products -----------------------------------------------------------------------------------------

def make_codes(rng, rows, cols, scales_shape, size=1.0, stride=None):
    """(codes on the device, their values, scales on the device, their values)"""
    stride = stride or cols
    x, _ = strided(rows, cols, stride, E4M3, float("nan"))
    v = np.clip(rng.standard_normal((rows, cols)) * 100, -448, 448)
    x.copy_(dev(v).to(E4M3))
    s = (size / 448 * np.exp(0.5 * rng.standard_normal(scales_shape))).astype(np.float32)
    return x, f64(x), dev(s), s.astype(np.float64)


SHAPES = [(1, 128, 128), (1, 16, 1), (2, 144, 130), (3, 1280, 257), (16, 2048, 384), (17, 400, 7), (31, 5120, 200), (33, 1152, 640), (64, 256, 1000), (65, 640, 129),
          (100, 272, 260), (128, 1024, 512), (129, 512, 300), (200, 2064, 272), (257, 384, 1027), (300, 1040, 513), (515, 896, 768), (400, 2448, 130), (270, 4112, 1544), (2100, 8208, 2600)]


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("n,k,features", SHAPES)
def test_mul(n, k, features, wide):
    rng = np.random.default_rng(n * 7 + k * 3 + features)
    x, xv, xs, xsv = make_codes(rng, n, k, (n, fr.blocks(k)), 1.0, k + 32)
    w, wv, ws, wsv = make_codes(rng, features, k, (fr.blocks(features), fr.blocks(k)), 0.05, k + 16)
    pitch = (features + 15) // 8 * 8
    out, buf = strided(n, features, pitch, torch.float32 if wide else torch.bfloat16, 5.0)
    hc.hc_mul8(x, k + 32, xs, w, k + 16, ws, n, hc.mul8(features, k, hc.HC_F32 if wide else hc.HC_BF16), out, pitch)
    no_error()
    ref, e = fr.product(xv, xsv, wv, wsv)
    assert_within(f64(out), ref, e + (0 if wide else fr.BF16 * (np.abs(ref) + e)))
    assert (buf[:, features:] == 5).all()


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("short", [True, False])
@pytest.mark.parametrize("n,k,features", [(n, k, (f + 15) // 16 * 16) for n, k, f in SHAPES])
def test_gated(n, k, features, short, kind):
    rng = np.random.default_rng(n * 11 + k + features)
    x, xv, xs, xsv = make_codes(rng, n, k, (n, fr.blocks(k)), 1.0, k + 16)
    size = 4.0 / np.sqrt(k)
    g, gv, gs, gsv = make_codes(rng, features, k, (fr.blocks(features), fr.blocks(k)), size, k + 16)
    u, uv, us, usv = make_codes(rng, features, k, (fr.blocks(features), fr.blocks(k)), size, k + 16)
    pitch = features + 16
    out, buf = strided(n, features, pitch, E4M3 if short else torch.bfloat16, 5.0)
    scales = torch.empty((n, fr.blocks(features)), device="cuda") if short else None
    s = hc.gated8(features, k, hc.HC_ACT_SILU if kind == "silu" else hc.HC_ACT_GELU, hc.HC_E4M3 if short else hc.HC_BF16)
    hc.hc_gated_mul8(x, k + 16, xs, g, gs, u, us, k + 16, n, s, out, pitch, scales)
    no_error()
    ref, e = fr.gated(xv, xsv, gv, gsv, uv, usv, kind)
    if short:
        check_codes(f64(out), f64(scales), ref, e)
    else:
        assert_within(f64(out), ref, e + fr.BF16 * (np.abs(ref) + e))
    assert (buf[:, features:].float() == 5).all()


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("n", [2, 300])
def test_gates_far_out(n, kind):
    """Gates from where the activation passes them on to where nothing is left of them. A token's gate is its code times a power of two; up is 1."""
    values = np.concatenate([np.arange(-126, 127) / 1.0, np.arange(-126, 127) / 8.0, [-448.0, 448.0, -0.5, 0.0, 2.0 ** -9]])
    features, k = (len(values) + 15) // 16 * 16, 16
    wv = np.zeros((features, k))
    wv[:len(values), 0] = values
    w, u = dev(wv).to(E4M3), torch.zeros((features, k), dtype=E4M3, device="cuda")
    u[:, 1] = 1.0
    x = torch.zeros((n, k), dtype=E4M3, device="cuda")
    x[:, :2] = 1.0
    ones = torch.ones((n, 1), device="cuda")
    ws = torch.ones((fr.blocks(features), 1), device="cuda")
    out = torch.empty((n, features), dtype=torch.bfloat16, device="cuda")
    hc.hc_gated_mul8(x, k, ones, w, ws, u, ws, k, n, hc.gated8(features, k, hc.HC_ACT_SILU if kind == "silu" else hc.HC_ACT_GELU, hc.HC_BF16), out, features, None)
    no_error()
    g = f64(w)[:, 0]
    y = -g if kind == "silu" else -2 * np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)
    with np.errstate(over="ignore"):
        ref = g / (1 + np.exp(y))
    # the exponent's argument takes up to 6 roundings (2^-24 each, of |y|), 2^t, 1/t, their sum and the products 16
    e = (6 * np.minimum(np.abs(y), 100) + 16) * fr.U * np.abs(ref) + 2.0 ** -119
    assert_within(f64(out), np.broadcast_to(ref, out.shape), e + fr.BF16 * (np.abs(ref) + e))


@pytest.mark.parametrize("n", [1, 40, 130, 400])
def test_product_nan_stays_in_its_row_and_column(n):
    rng = np.random.default_rng(n)
    k, features = 656, 300
    x, xv, xs, xsv = make_codes(rng, n, k, (n, fr.blocks(k)))
    w, wv, ws, wsv = make_codes(rng, features, k, (fr.blocks(features), fr.blocks(k)), 0.05)
    x.view(torch.uint8)[n // 2, 650] = 0x7F
    w.view(torch.uint8)[77, 3] = 0xFF
    out = torch.empty((n, 304), device="cuda")[:, :features]
    hc.hc_mul8(x, k, xs, w, k, ws, n, hc.mul8(features, k, hc.HC_F32), out, 304)
    no_error()
    nan = np.zeros((n, features), bool)
    nan[n // 2], nan[:, 77] = True, True
    assert np.array_equal(np.isnan(f64(out)), nan)
    ref, e = fr.product(np.nan_to_num(xv), xsv, np.nan_to_num(wv), wsv)
    assert_within(f64(out)[~nan], ref[~nan], e[~nan])


@pytest.mark.parametrize("n,k,features", [(1, 5120, 640), (48, 2048, 512), (200, 1024, 768), (700, 640, 1100)])
def test_product_repeats_bit_for_bit(n, k, features):
    rng = np.random.default_rng(3)
    x, _, xs, _ = make_codes(rng, n, k, (n, fr.blocks(k)))
    w, _, ws, _ = make_codes(rng, features, k, (fr.blocks(features), fr.blocks(k)), 0.05)
    pitch = (features + 7) // 8 * 8
    outs = [torch.empty((n, pitch), device="cuda") for _ in range(6)]
    for o in outs:
        hc.hc_mul8(x, k, xs, w, k, ws, n, hc.mul8(features, k, hc.HC_F32), o, pitch)
    no_error()
    assert all(torch.equal(o[:, :features], outs[0][:, :features]) for o in outs)


@pytest.mark.parametrize("n", [2, 50, 300])
def test_products_of_scales_out_of_range(n):
    """NaN, infinite, zero and very small scales do to a product what they do to the values they stand for."""
    rng = np.random.default_rng(n)
    k, features = 400, 272
    x, xv, xs, xsv = make_codes(rng, n, k, (n, 4))
    w, wv, ws, wsv = make_codes(rng, features, k, (3, 4), 0.05)
    xsv[0, 1], xsv[1, 3] = np.nan, 2.0 ** -100
    wsv[2, 0], wsv[1, 2] = np.inf, 0.0
    xs, ws = dev(xsv), dev(wsv)
    out = torch.empty((n, features), device="cuda")
    hc.hc_mul8(x, k, xs, w, k, ws, n, hc.mul8(features, k, hc.HC_F32), out, features)
    h, hs = torch.empty((n, features), dtype=E4M3, device="cuda"), torch.empty((n, 3), device="cuda")
    hc.hc_gated_mul8(x, k, xs, w, ws, w, ws, k, n, hc.gated8(features, k), h, features, hs)
    no_error()
    got = f64(out)
    assert np.isnan(got[0]).all() and (~np.isfinite(got[1:, 256:])).all()
    fine = np.nan_to_num(wsv, posinf=0.0)
    ref, e = fr.product(xv[1:], xsv[1:], wv, fine)
    assert_within(got[1:, :256], ref[:, :256], e[:, :256])
    hv = f64(h) * fr.spread(f64(hs), features)
    assert np.isnan(hv[0]).all() and np.isnan(hv[1:, 256:]).all()
    check_codes(f64(h)[1:, :256], f64(hs)[1:, :2], *[v[:, :256] for v in fr.gated(xv[1:], xsv[1:], wv, fine, wv, fine, "silu")])


# ---- log probabilities ----------------------------------------------------------------------------------

def check_logprobs(z, tokens, scale, top, x64=None, stride=None):
    n, vocab = z.shape
    lp, h = gu.guarded((n,), torch.float32), gu.guarded((n,), torch.float32)
    tl = gu.guarded((n, top), torch.float32) if top else None
    tt = gu.guarded((n, top), torch.int32) if top else None
    s = hc.logprobs(n, vocab, top, scale, hc.HC_BF16 if z.dtype == torch.bfloat16 else hc.HC_F32)
    hc.hc_token_logprobs(z, z.stride(0), dev(tokens, torch.int64), s, lp, h, tl, tt)
    torch.cuda.synchronize()
    ref = fr.logprobs(f64(z), tokens, float(np.float32(scale)), top)

    def close(got, want, tol):
        inf = np.isinf(want)
        assert np.array_equal(got[inf], want[inf])
        assert_within(got[~inf], want[~inf], (tol + 8 * fr.U * np.abs(want))[~inf])

    close(f64(lp), ref[0], np.full(n, ref[4]))
    close(f64(h), ref[1], ref[5])
    if top:
        assert np.array_equal(tt.cpu().numpy(), ref[3])
        close(f64(tl), ref[2], np.full((n, top), ref[4]))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,vocab,top,scale", [(1, 1, 1, 1.0), (3, 7, 7, 0.5), (2, 33, 32, 1.0), (5, 255, 8, 1.0), (4, 257, 32, 2.0), (3, 1000, 20, 1.25),
                                               (700, 1001, 5, 1.0), (1, 16385, 32, 0.7), (9, 20011, 1, 1.0), (2, 131072, 20, 1.0), (310, 33333, 32, 1.1),
                                               (40, 100003, 0, 1.0), (1, 262147, 32, 1.0)])
def test_logprobs(n, vocab, top, scale, dtype):
    rng = np.random.default_rng(n + vocab)
    pitch = (vocab + 15) // 8 * 8
    buf = dev(np.full((n, pitch), 1e30, np.float32), dtype)
    buf[:, :vocab] = dev((3 * rng.standard_normal((n, vocab))).astype(np.float32), dtype)
    tokens = rng.integers(0, vocab, n)
    if n > 2:
        tokens[1] = -1
    check_logprobs(buf[:, :vocab], tokens, scale, top)
    no_error()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["equal", "zeros of both signs", "two values", "rising", "falling", "banned", "all banned", "lowest", "all lowest", "lowest and banned", "one left", "far", "far below", "far up"])
@pytest.mark.parametrize("n,vocab", [(3, 5000), (2, 70001), (400, 17000)])
def test_logprobs_hard_rows(n, vocab, kind, dtype):
    rng = np.random.default_rng(vocab)
    low = torch.finfo(dtype).min
    x = (3 * rng.standard_normal((n, vocab))).astype(np.float32)
    if kind == "equal":
        x[:] = 1.5
    elif kind == "zeros of both signs":
        x = np.where(x > 0, 0.0, -0.0).astype(np.float32)
    elif kind == "two values":
        x = np.where(x > 2, 1.0, -1.0).astype(np.float32)
    elif kind in ("rising", "falling"):
        x = np.sort(x, 1)
        x = np.ascontiguousarray(x[:, ::-1]) if kind == "falling" else x
    elif kind == "banned":
        x[rng.random((n, vocab)) < 0.999] = -np.inf
    elif kind == "all banned":
        x[:] = -np.inf
    elif kind == "one left":
        x[:] = -np.inf
        x[:, vocab // 3] = -40.0
    elif kind == "far":
        x *= 300
    z = dev(x, dtype)
    if kind == "lowest":
        z[:, ::2] = low
    elif kind == "all lowest":
        z[:] = low
    elif kind == "lowest and banned":
        z[:] = float("-inf")
        z[:, ::3] = low
        z[0, vocab // 2:] = low
        z[1, -1] = 0.9 * low
    elif kind in ("far below", "far up"):
        z = z + (1e10 if kind == "far up" else -1e10)
        z[:, 1::7] = float("-inf")
        z[0, 5] = z[0].max() * (1.5 if kind == "far up" else 0.5)
    pad = -vocab % 8
    z = torch.nn.functional.pad(z, (0, pad))[:, :vocab]
    check_logprobs(z, rng.integers(0, vocab, n), 1.0, 32)
    check_logprobs(z, rng.integers(0, vocab, n), 1.0, 3)
    if kind not in ("lowest", "all lowest", "lowest and banned"):  # (nothing overflows)
        for scale in (2.0 ** -64, 2.0 ** 20):
            check_logprobs(z, rng.integers(0, vocab, n), scale, 1)
    no_error()


# Rows whose segments are many chunks, so that several share the maxima that say where alternatives are.
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["normal", "few values", "few left", "equal", "equal but late"])
@pytest.mark.parametrize("n,vocab", [(2, 1500007), (309, 110003)])
def test_logprobs_long_rows(n, vocab, kind, dtype):
    rng = np.random.default_rng(vocab)
    x = (3 * rng.standard_normal((n, vocab), dtype=np.float32))
    if kind == "few values":
        x = np.round(x)
    elif kind == "few left":
        x[:, np.arange(vocab) % 8192 != 5] = -np.inf
    elif kind == "equal":
        x[:] = -2.0
    elif kind == "equal but late":
        x[:] = -2.0
        x[:, -40:] = -1.0
        x[0, -3:] = -3.0
    z = torch.nn.functional.pad(dev(x, dtype), (0, -vocab % 8))[:, :vocab]
    check_logprobs(z, rng.integers(0, vocab, n), 1.0, 20)
    no_error()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab", [40, 5000, 70001])
def test_logprobs_nan_and_infinity(vocab, dtype):
    """NaN ranks last and makes a row's numbers NaN, plus infinity too; the rows beside keep theirs."""
    rng = np.random.default_rng(vocab)
    n, top = 5, 32
    x = (3 * rng.standard_normal((n, vocab))).astype(np.float32)
    x[1, vocab - 1] = np.nan
    x[2, 7] = np.inf
    x[3] = np.nan
    x[4, :vocab - 3] = np.nan  # fewer numbers than alternatives
    pitch = (vocab + 7) // 8 * 8
    z = torch.nn.functional.pad(dev(x, dtype), (0, pitch - vocab))[:, :vocab]
    lp, h = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    tl, tt = torch.empty((n, top), device="cuda"), torch.full((n, top), -7, dtype=torch.int32, device="cuda")
    hc.hc_token_logprobs(z, pitch, dev(np.full(n, 9), torch.int64), hc.logprobs(n, vocab, top, 1.0, hc.HC_BF16 if dtype == torch.bfloat16 else hc.HC_F32), lp, h,
                         tl, tt)
    no_error()
    assert np.array_equal(np.isnan(f64(lp)), [False, True, True, True, True]) and np.array_equal(np.isnan(f64(h)), [False, True, True, True, True])
    v = f64(z)
    for r in range(n):
        order = np.argsort(np.where(np.isnan(v[r]), np.inf, -v[r]), kind="stable")[:top]
        assert np.array_equal(tt[r].cpu().numpy(), order), r
    ref = fr.logprobs(v[:1], np.array([9]), 1.0, top)
    assert_within(f64(tl)[0], ref[2][0], ref[4] + 8 * fr.U * np.abs(ref[2][0]))


def test_logprobs_padding_and_tokens_out_of_range():
    z = dev(np.random.default_rng(1).standard_normal((4, 104)).astype(np.float32))
    lp = torch.full((4,), 9.0, device="cuda")
    hc.hc_token_logprobs(z, 104, dev(np.array([-1, 100, 3, -2 ** 62]), torch.int64), hc.logprobs(4, 100), lp, None, None, None)
    torch.cuda.synchronize()
    assert hc.hc_device_error(clear=True) == 1 << 24
    got = f64(lp)
    assert got[0] == got[1] == got[3] == 0 and got[2] < 0
    assert hc.hc_device_error(clear=True) == 0


# ---- streams, graphs, a run together --------------------------------------------------------------------

def ffn_params(rng, d, f):
    return [make_codes(rng, rows, cols, (fr.blocks(rows), fr.blocks(cols)), 6.0 / np.sqrt(cols)) for rows, cols in ((f, d), (f, d), (d, f))]


class Ffn:
    """Buffers of one feed-forward sublayer and its calls."""

    def __init__(self, rng, n, d, f):
        self.n, self.d, self.f = n, d, f
        self.gate, self.up, self.down = ffn_params(rng, d, f)
        e = lambda *s, t=torch.float32: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
        self.c, self.s, self.hc_, self.hs = e(n, d, t=E4M3), e(n, fr.blocks(d)), e(n, f, t=E4M3), e(n, fr.blocks(f))

    def __call__(self, y, delta, stream=None):
        n, d, f = self.n, self.d, self.f
        hc.hc_norm_quant8(y, d, None, 0, None, hc.quant8(n, d, norm=False), None, 0, self.c, d, self.s, stream)
        hc.hc_gated_mul8(self.c, d, self.s, self.gate[0], self.gate[2], self.up[0], self.up[2], d, n, hc.gated8(f, d), self.hc_, f, self.hs, stream)
        hc.hc_mul8(self.hc_, f, self.hs, self.down[0], f, self.down[2], n, hc.mul8(d, f), delta, d, stream)

    def check(self, y, delta):
        check_codes(f64(self.c), f64(self.s), f64(y), 0.0, "x")
        ref, e = fr.gated(f64(self.c), f64(self.s), self.gate[1], self.gate[3], self.up[1], self.up[3], "silu")
        check_codes(f64(self.hc_), f64(self.hs), ref, e, "h")
        ref, e = fr.product(f64(self.hc_), f64(self.hs), self.down[1], self.down[3])
        assert_within(f64(delta), ref, e + fr.BF16 * (np.abs(ref) + e), "delta")


def test_sublayer_between_two_steps_and_the_head():
    """The feed-forward sublayer between two Hyper-Connection calls, then the end of the stack, the vocabulary's logits and the
    tokens' log probabilities; the decode form captured into a graph and replayed on new inputs."""
    rng = np.random.default_rng(17)
    from hyper_connection_residual_hc_gb300 import synth
    n, d, f, vocab, top = 24, 512, 1040, 1003, 5
    w = synth.small("step_b1_t64", 1, n, d, seed=77)
    P = gu.DevParams(synth.params(w, 0), d, 4)
    s = hc.shape(d=d, sinkhorn_iters=w.iters, hc_eps=w.hc_eps, norm_eps=w.norm_eps)
    e = lambda *sh, t=torch.float32: torch.empty(sh, dtype=t, device="cuda")  # noqa: E731
    X, X2, y, delta, z = e(n, 4, d, t=torch.bfloat16), e(n, 4, d, t=torch.bfloat16), e(n, d, t=torch.bfloat16), e(n, d, t=torch.bfloat16), e(n, d, t=torch.bfloat16)
    pm, pre, post, comb = e(n, 4), e(n, 4), e(n, 4), e(n, 4, 4)
    ws = hc.new_workspace()
    ffn = Ffn(rng, n, d, f)
    head = make_codes(rng, vocab, d, (fr.blocks(vocab), fr.blocks(d)), 3.0 / np.sqrt(d))
    zc, zs, logits = e(n, d, t=E4M3), e(n, fr.blocks(d)), e(n, 1008)
    tokens = torch.empty(n, dtype=torch.int64, device="cuda")
    lp, h, tl, tt = e(n), e(n), e(n, top), e(n, top, t=torch.int32)
    gain = dev(1 + 0.1 * rng.standard_normal(d))

    def step():
        hc.hc_pre_step(X, pm, P.c, n, s, y, pre, post, comb, ws)
        ffn(y, delta)
        hc.hc_post_then_final(delta, X, post, comb, pre, gain, n, s, X2, z)
        hc.hc_norm_quant8(z, d, None, 0, None, hc.quant8(n, d, norm=False), None, 0, zc, d, zs)
        hc.hc_mul8(zc, d, zs, head[0], d, head[2], n, hc.mul8(vocab, d, hc.HC_F32), logits, 1008)
        hc.hc_token_logprobs(logits, 1008, tokens, hc.logprobs(n, vocab, top), lp, h, tl, tt)

    def fill(seed):
        r = np.random.default_rng(seed)
        X.copy_(dev(r.standard_normal((n, 4, d)), torch.bfloat16))
        pm.copy_(dev(1 / (1 + np.exp(-r.standard_normal((n, 4))))))
        tokens.copy_(dev(r.integers(0, vocab, n), torch.int64))

    def check():
        no_error()
        ffn.check(y, delta)
        check_codes(f64(zc), f64(zs), f64(z), 0.0, "z")
        ref, er = fr.product(f64(zc), f64(zs), head[1], head[3])
        assert_within(f64(logits)[:, :vocab], ref, er, "logits")
        want = fr.logprobs(f64(logits)[:, :vocab], tokens.cpu().numpy(), 1.0, top)
        assert_within(f64(lp), want[0], want[4] + 8 * fr.U * np.abs(want[0]))
        assert_within(f64(h), want[1], want[5] + 8 * fr.U * want[1])
        assert np.array_equal(tt.cpu().numpy(), want[3])

    fill(1)
    step()
    check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        step()
    for seed in (2, 3):
        fill(seed)
        for t in (delta, logits, lp):
            t.fill_(float("nan"))
        g.replay()
        check()


def test_two_graphs_and_an_eager_call_at_once():
    """No call has anything in common with another: two graphs replayed on two streams beside calls on a third."""
    rng = np.random.default_rng(4)
    d, f = 640, 1296
    runs = [(Ffn(rng, n, d, f), dev(rng.standard_normal((n, d)), torch.bfloat16), torch.empty((n, d), dtype=torch.bfloat16, device="cuda"), torch.cuda.Stream())
            for n in (3, 70, 300)]
    torch.cuda.synchronize()
    graphs = []
    for ffn, y, delta, stream in runs[:2]:
        with torch.cuda.stream(stream):
            ffn(y, delta)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            ffn(y, delta)
        graphs.append((g, stream))
    want = []
    for ffn, y, delta, stream in runs:
        ffn(y, delta)
        torch.cuda.synchronize()
        want.append(delta.clone())
        delta.fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(10):
        for g, stream in graphs:
            with torch.cuda.stream(stream):
                g.replay()
        runs[2][0](runs[2][1], runs[2][2], runs[2][3])
    no_error()
    for (ffn, y, delta, _), w in zip(runs, want):
        assert torch.equal(delta, w)
        ffn.check(y, delta)


@pytest.mark.parametrize("n,d,f", [(3, 640, 1296), (70, 512, 1040), (300, 1152, 2064), (2100, 2608, 8208)])
def test_chain_of_dependent_calls(n, d, f):
    """Calls that start under each other's end wait for each other's results: a chain without a pause, and replayed from a graph, gives
    the bytes of the chain with a synchronisation behind every call. (The last shape takes two launches for the way back.)"""
    rng = np.random.default_rng(n)
    layers = [Ffn(rng, n, d, f) for _ in range(2)]
    y0 = dev(rng.standard_normal((n, d)), torch.bfloat16)
    bufs = [torch.empty((n, d), dtype=torch.bfloat16, device="cuda") for _ in range(7)]
    gain = dev(1 + 0.1 * rng.standard_normal(d))

    def chain(sync):
        y = y0
        for i, b in enumerate(bufs):
            ffn = layers[i % 2]
            hc.hc_norm_quant8(y, d, y0, d, gain, hc.quant8(n, d), None, 0, ffn.c, d, ffn.s)
            sync()
            hc.hc_gated_mul8(ffn.c, d, ffn.s, ffn.gate[0], ffn.gate[2], ffn.up[0], ffn.up[2], d, n, hc.gated8(f, d), ffn.hc_, f, ffn.hs)
            sync()
            hc.hc_mul8(ffn.hc_, f, ffn.hs, ffn.down[0], f, ffn.down[2], n, hc.mul8(d, f), b, d)
            sync()
            y = b

    chain(torch.cuda.synchronize)
    want = [b.clone() for b in bufs]
    for _ in range(3):
        for b in bufs:
            b.fill_(float("nan"))
        chain(lambda: None)
        no_error()
        assert all(torch.equal(b, w) for b, w in zip(bufs, want))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        chain(lambda: None)
    for _ in range(3):
        for b in bufs:
            b.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        g.replay()
        no_error()
        assert all(torch.equal(b, w) for b, w in zip(bufs, want))


@pytest.mark.parametrize("n,k,features", [(3, 16, 300), (40, 144, 640), (300, 16, 1027), (300, 272, 2600), (2100, 144, 2600)])
def test_short_products_one_after_the_other(n, k, features):
    """Kernels of one to three blocks of k, whose last arrivals come close to their end, in a row on the same SMs."""
    rng = np.random.default_rng(k)
    x, xv, xs, xsv = make_codes(rng, n, k, (n, fr.blocks(k)))
    w, wv, ws, wsv = make_codes(rng, features, k, (fr.blocks(features), fr.blocks(k)), 0.05)
    pitch = (features + 7) // 8 * 8
    outs = [torch.full((n, pitch), float("nan"), device="cuda") for _ in range(20)]

    def run():
        for o in outs:
            hc.hc_mul8(x, k, xs, w, k, ws, n, hc.mul8(features, k, hc.HC_F32), o, pitch)

    def check():
        no_error()
        ref, e = fr.product(xv, xsv, wv, wsv)
        assert_within(f64(outs[0])[:, :features], ref, e)
        assert all(torch.equal(o[:, :features], outs[0][:, :features]) for o in outs)

    run()
    check()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        run()
    for o in outs:
        o.fill_(float("nan"))
    g.replay()
    g.replay()
    check()


def test_products_of_different_sizes_in_a_row():
    """Kernels that hold from 32 to all 512 columns of an SM's tensor memory, each set up under the end of the one ahead, in a graph."""
    rng = np.random.default_rng(8)
    k, f = 1152, 1040
    g, _, gs, _ = make_codes(rng, f, k, (fr.blocks(f), 9), 4.0 / np.sqrt(k))
    u, _, us, _ = make_codes(rng, f, k, (fr.blocks(f), 9), 4.0 / np.sqrt(k))
    calls = []
    for n in (64, 1, 128, 30, 300, 5, 64, 600, 64, 100):
        x, _, xs, _ = make_codes(rng, n, k, (n, 9))
        calls.append((n, x, xs, torch.empty((n, f), device="cuda"), torch.empty((n, f), dtype=torch.bfloat16, device="cuda")))

    def run(sync):
        for n, x, xs, y, h in calls:
            hc.hc_gated_mul8(x, k, xs, g, gs, u, us, k, n, hc.gated8(f, k, out_type=hc.HC_BF16), h, f, None)
            sync()
            hc.hc_mul8(x, k, xs, g, k, gs, n, hc.mul8(f, k, hc.HC_F32), y, f)
            sync()

    run(torch.cuda.synchronize)
    want = [(y.clone(), h.clone()) for _, _, _, y, h in calls]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        run(lambda: None)
    for _ in range(5):
        for _, _, _, y, h in calls:
            y.fill_(float("nan"))
            h.fill_(float("nan"))
        graph.replay()
        graph.replay()
        no_error()
        assert all(torch.equal(y, a) and torch.equal(h, b) for (_, _, _, y, h), (a, b) in zip(calls, want))


def unpaused(chain, reset, outs):
    """A chain of calls without a pause, and replayed, gives the bytes of the chain with a synchronisation behind every call."""
    reset()
    chain(torch.cuda.synchronize)
    no_error()
    want = [t.clone().view(torch.uint8) for t in outs]
    graph = torch.cuda.CUDAGraph()
    reset()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        chain(lambda: None)
    for run in [lambda: chain(lambda: None)] * 3 + [graph.replay] * 3:
        reset()
        run()
        no_error()
        assert all(torch.equal(t.view(torch.uint8), w) for t, w in zip(outs, want))


def test_chain_of_long_norms():
    """Quantisations long enough (an estimated 12 us) to start under the end of the product that writes their rows, and products behind
    them; the residual in place."""
    n, d = 4800, 2608
    rng = np.random.default_rng(6)
    w, _, ws, _ = make_codes(rng, d, d, (fr.blocks(d), fr.blocks(d)), 4.0 / np.sqrt(d))
    c0, _, s0, _ = make_codes(rng, n, d, (n, fr.blocks(d)))
    r0, gain = dev(rng.standard_normal((n, d)), torch.bfloat16), dev(1 + 0.1 * rng.standard_normal(d))
    c, s, r, y = c0.clone(), s0.clone(), r0.clone(), torch.empty_like(r0)

    def reset():
        for a, b in ((c, c0), (s, s0), (r, r0)):
            a.copy_(b)
        y.fill_(float("nan"))

    def chain(sync):
        for _ in range(6):
            hc.hc_mul8(c, d, s, w, d, ws, n, hc.mul8(d, d), y, d)
            sync()
            hc.hc_norm_quant8(y, d, r, d, gain, hc.quant8(n, d), r, d, c, d, s)
            sync()

    unpaused(chain, reset, [c, s, r, y])
    total = f64(r)
    check_codes(f64(c), f64(s), fr.norm(total, f64(gain), 1e-6), (d / 2 + 16) * fr.U * np.abs(fr.norm(total, f64(gain), 1e-6)))


@pytest.mark.parametrize("n,vocab", [(33, 250003), (300, 40000)])
def test_chain_of_long_heads(n, vocab):
    """Log probabilities long enough (an estimated 12 us) to start under the end of the product that writes their logits, which the next
    product writes again."""
    k, top, pitch = 272, 5, (vocab + 7) // 8 * 8
    rng = np.random.default_rng(9)
    w, _, ws, _ = make_codes(rng, vocab, k, (fr.blocks(vocab), fr.blocks(k)), 4.0 / np.sqrt(k))
    rows = [make_codes(rng, n, k, (n, fr.blocks(k))) for _ in range(5)]
    logits = torch.empty((n, pitch), device="cuda")
    tokens = dev(rng.integers(0, vocab, n), torch.int64)
    outs = [(torch.empty(n, device="cuda"), torch.empty(n, device="cuda"), torch.empty((n, top), device="cuda"), torch.empty((n, top), dtype=torch.int32, device="cuda"))
            for _ in rows]
    flat = [t for o in outs for t in o]

    def reset():
        logits.fill_(float("nan"))
        for t in flat:
            t.fill_(-7)

    def chain(sync):
        for (x, _, xs, _), o in zip(rows, outs):
            hc.hc_mul8(x, k, xs, w, k, ws, n, hc.mul8(vocab, k, hc.HC_F32), logits, pitch)
            sync()
            hc.hc_token_logprobs(logits, pitch, tokens, hc.logprobs(n, vocab, top), *o)
            sync()

    unpaused(chain, reset, flat)
    ref = fr.logprobs(f64(logits)[:, :vocab], tokens.cpu().numpy(), 1.0, top)
    assert_within(f64(outs[-1][0]), ref[0], ref[4] + 8 * fr.U * np.abs(ref[0]))
    assert np.array_equal(outs[-1][3].cpu().numpy(), ref[3])


@pytest.mark.parametrize("n", [3, 300])
def test_products_behind_copies_and_other_streams(n):
    """A captured product whose inputs come from a copy, from another stream's kernels, and from both; and whose output another stream reads."""
    rng = np.random.default_rng(n)
    k, f = 2064, 528
    w, _, ws, _ = make_codes(rng, f, k, (fr.blocks(f), fr.blocks(k)), 4.0 / np.sqrt(k))
    x0, _, s0, _ = make_codes(rng, n, k, (n, fr.blocks(k)))
    y = dev(rng.standard_normal((n, k)), torch.bfloat16)
    x, s, c, cs = torch.empty_like(x0), torch.empty_like(s0), torch.empty_like(x0), torch.empty_like(s0)
    outs = [torch.empty((n, f), device="cuda") for _ in range(3)]
    side = torch.cuda.Stream()

    def mul(a, b, o):
        hc.hc_mul8(a, k, b, w, k, ws, n, hc.mul8(f, k, hc.HC_F32), o, f)

    def step():
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        x.copy_(x0)
        s.copy_(s0)
        mul(x, s, outs[0])
        with torch.cuda.stream(side):
            hc.hc_norm_quant8(y, k, None, 0, None, hc.quant8(n, k), None, 0, c, k, cs)
            mul(c, cs, outs[1])
        main.wait_stream(side)
        outs[1].add_(outs[0])
        mul(c, cs, outs[2])
        outs[2].add_(outs[1])

    def clear():
        for t in outs + [s, cs]:
            t.fill_(float("nan"))
        x.view(torch.uint8).zero_()
        c.view(torch.uint8).zero_()

    clear()
    step()
    no_error()
    want = [o.clone() for o in outs]
    first, second = torch.empty_like(outs[0]), torch.empty_like(outs[0])
    mul(x0, s0, first)
    mul(c, cs, second)
    no_error()
    assert torch.equal(want[0], first) and torch.equal(want[1], first + second) and torch.equal(want[2], second + (first + second))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        step()
    for _ in range(3):
        clear()
        g.replay()
        g.replay()
        no_error()
        assert all(torch.equal(o, v) for o, v in zip(outs, want))


# 9 x 20 gated tiles are two turns of 76 pairs and 28 tiles, which two pairs share each in a launch of their own; the last block of k is short.
TWO_LAUNCHES = (2100, 10256, 2480)


@pytest.mark.parametrize("kind,short", [("silu", True), ("gelu", False)])
def test_gated_in_two_launches(kind, short):
    n, k, features = TWO_LAUNCHES
    test_gated(n, k, features, short, kind)


def test_chain_of_calls_of_two_launches():
    """Rows quantised into the same buffers again and again, each time read by products of two launches; plain and replayed, as with a
    synchronisation behind every call."""
    n, k, f = TWO_LAUNCHES
    rng = np.random.default_rng(5)
    g, _, gs, _ = make_codes(rng, f, k, (fr.blocks(f), fr.blocks(k)), 4.0 / np.sqrt(k))
    u, _, us, _ = make_codes(rng, f, k, (fr.blocks(f), fr.blocks(k)), 4.0 / np.sqrt(k))
    ys = [dev(rng.standard_normal((n, k)) * (i + 1), torch.bfloat16) for i in range(4)]
    c, s = torch.empty((n, k), dtype=E4M3, device="cuda"), torch.empty((n, fr.blocks(k)), device="cuda")
    hs = [torch.empty((n, f), dtype=torch.bfloat16, device="cuda") for _ in ys]
    zs = [torch.empty((n, f), device="cuda") for _ in ys]

    def chain(sync):
        for y, h, z in zip(ys, hs, zs):
            hc.hc_norm_quant8(y, k, None, 0, None, hc.quant8(n, k, norm=False), None, 0, c, k, s)
            sync()
            hc.hc_gated_mul8(c, k, s, g, gs, u, us, k, n, hc.gated8(f, k, out_type=hc.HC_BF16), h, f, None)
            sync()
            hc.hc_mul8(c, k, s, g, k, gs, n, hc.mul8(f, k, hc.HC_F32), z, f)
            sync()

    chain(torch.cuda.synchronize)
    want = [t.clone() for t in hs + zs]

    def check():
        no_error()
        assert all(torch.equal(t, w) for t, w in zip(hs + zs, want))
        for t in hs + zs:
            t.fill_(float("nan"))

    for _ in range(3):
        chain(lambda: None)
        check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        chain(lambda: None)
    for _ in range(3):
        graph.replay()
        graph.replay()
        check()


FIRST_CALLS = """
import sys
import torch
import hyper_connection_residual_hc_gb300 as hc

torch.zeros(1, device="cuda")
hc.load()
n, k, f = int(sys.argv[1]), 1152, 272
e = lambda *s, t=torch.float32: torch.ones(s, device="cuda").to(t)
x, w, u, xs, ws = e(n, k, t=torch.float8_e4m3fn), e(f, k, t=torch.float8_e4m3fn), e(f, k, t=torch.float8_e4m3fn), e(n, 9), e(3, 9) / k
y, h, hs, out = e(n, k, t=torch.bfloat16), e(n, f, t=torch.float8_e4m3fn), e(n, 3), e(n, f)
tokens, lp = torch.zeros(n, dtype=torch.int64, device="cuda"), e(n)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):  # the process's first calls
    hc.hc_norm_quant8(y, k, None, 0, None, hc.quant8(n, k), None, 0, x, k, xs)
    hc.hc_mul8(x, k, xs, w, k, ws, n, hc.mul8(f, k, hc.HC_F32), out, f)
    hc.hc_gated_mul8(x, k, xs, w, ws, u, ws, k, n, hc.gated8(f, k), h, f, hs)
    hc.hc_token_logprobs(out, f, tokens, hc.logprobs(n, f), lp, None, None, None)
g.replay()
torch.cuda.synchronize()
assert hc.hc_device_error(clear=True) == 0
assert torch.allclose(out, torch.ones_like(out), rtol=1e-5) and torch.allclose(h.float() * hs[0, 0], torch.full((n, f), 0.7310586, device="cuda"), rtol=1e-4)
assert torch.allclose(lp, torch.full_like(lp, -5.605802), rtol=1e-5)
"""


@pytest.mark.parametrize("n", [1, 40, 100, 400])
def test_first_calls_of_a_process_captured(n):
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS, str(n)], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


def test_rows_past_32_bits():
    """Logits whose rows start past 2^31 elements, and codes past 2^32 bytes."""
    n, vocab, stride = 3, 5003, 1 << 30
    buf = torch.zeros(2 * stride + 8192, dtype=torch.bfloat16, device="cuda")
    z = buf.as_strided((n, vocab), (stride, 1))
    rng = np.random.default_rng(0)
    z.copy_(dev(rng.standard_normal((n, vocab)), torch.bfloat16))
    check_logprobs(z, rng.integers(0, vocab, n), 1.0, 8)
    no_error()
    del buf, z
    k, features, pitch = 144, 136, 1 << 31
    raw = torch.zeros(2 * pitch + 256, dtype=torch.uint8, device="cuda")
    x = raw.as_strided((3, k), (pitch, 1))
    cx, xv, xs, xsv = make_codes(rng, 3, k, (3, 2))
    x.copy_(cx.view(torch.uint8))
    w, wv, ws, wsv = make_codes(rng, features, k, (2, 2))
    out = torch.empty((3, features), device="cuda")
    hc.hc_mul8(x, pitch, xs, w, k, ws, 3, hc.mul8(features, k, hc.HC_F32), out, features)
    no_error()
    ref, e = fr.product(xv, xsv, wv, wsv)
    assert_within(f64(out), ref, e)


@pytest.mark.parametrize("n", [20, 300])
def test_wide_strides_of_products(n):
    """Rows of weights and of outputs that start past 2^32 bytes, by either kernel."""
    rng = np.random.default_rng(n)
    k, features, pitch = 272, 272, 1 << 24
    x, xv, xs, xsv = make_codes(rng, n, k, (n, 3))
    raw = torch.zeros((features - 1) * pitch + 1024, dtype=torch.uint8, device="cuda")
    w = raw.as_strided((features, k), (pitch, 1))
    cw, wv, ws, wsv = make_codes(rng, features, k, (3, 3), 0.1)
    w.copy_(cw.view(torch.uint8))
    buf = torch.zeros((n - 1) * pitch + 1024, device="cuda")
    out = buf.as_strided((n, features), (pitch, 1))
    hc.hc_mul8(x, k, xs, w, pitch, ws, n, hc.mul8(features, k, hc.HC_F32), out, pitch)
    no_error()
    ref, e = fr.product(xv, xsv, wv, wsv)
    assert_within(f64(out), ref, e)
    h = buf.view(torch.uint8).as_strided((n, features), (4 * pitch, 1))
    hs = torch.empty((n, 3), device="cuda")
    hc.hc_gated_mul8(x, k, xs, w, ws, w, ws, pitch, n, hc.gated8(features, k), h, 4 * pitch, hs)
    no_error()
    ref, e = fr.gated(xv, xsv, wv, wsv, wv, wsv, "silu")
    check_codes(f64(h.contiguous().view(E4M3)), f64(hs), ref, e)


def test_norm_quant_rows_past_32_bits():
    rng = np.random.default_rng(2)
    n, d, pitch = 3, 1040, 1 << 31
    buf = torch.zeros(2 * pitch + 4096, dtype=torch.bfloat16, device="cuda")
    x, r = buf.as_strided((n, d), (pitch, 1)), buf.as_strided((n, d), (pitch, 1), 2048)
    x.copy_(dev(rng.standard_normal((n, d)), torch.bfloat16))
    r.copy_(dev(rng.standard_normal((n, d)), torch.bfloat16))
    want = (x.float() + r.float()).to(torch.bfloat16)
    codes, scales = torch.empty((n, d), dtype=E4M3, device="cuda"), torch.empty((n, 9), device="cuda")
    hc.hc_norm_quant8(x, pitch, r, pitch, None, hc.quant8(n, d), r, pitch, codes, d, scales)
    no_error()
    assert torch.equal(r, want)
    y = fr.norm(f64(want), None, 1e-6)
    check_codes(f64(codes), f64(scales), y, (d / 2 + 16) * fr.U * np.abs(y))


@pytest.mark.parametrize("n", [2, 40, 260])
def test_longest_k(n):
    rng = np.random.default_rng(n)
    k, features = 1 << 20, 16
    x, xv, xs, xsv = make_codes(rng, n, k, (n, k // 128))
    w, wv, ws, wsv = make_codes(rng, features, k, (1, k // 128), 0.01)
    out = torch.empty((n, features), device="cuda")
    hc.hc_mul8(x, k, xs, w, k, ws, n, hc.mul8(features, k, hc.HC_F32), out, features)
    no_error()
    # (8,192 blocks are added up one after the other by as few as one thread)
    a, b = dev(xv * fr.spread(xsv, k), torch.float64), dev(wv * fr.spread(wsv, k, features), torch.float64)
    ref, mag = f64(a @ b.T), f64(a.abs() @ b.abs().T)
    assert_within(f64(out), ref, (2 * fr.BLOCK + k // 128 + 16) * fr.U * mag)
