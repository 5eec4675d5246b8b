"""The attention over the 4-bit cache where softmax weights lie far below a row's largest: an attention sink before many
other keys."""

import numpy as np
import pytest
import torch

import hyper_connection_residual_hc_gb300 as hc

import attn_ref as ar
import gpu_util as gu
from test_gpu_attention import bf, f64, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    hc.load()
    gu.device_error_clear()
    yield
    gu.device_error_clear()


@pytest.mark.parametrize("lead", [22.6, 26.0])
@pytest.mark.parametrize("seqs,q_len,hq,hk,dim", [(38, 1, 8, 8, 64), (38, 1, 8, 8, 128), (76, 1, 48, 4, 128), (57, 2, 16, 8, 256), (160, 40, 1, 1, 64),
                                                  (160, 40, 1, 1, 128)])
def test_weights_far_below_the_largest(seqs, q_len, hq, hk, dim, lead):
    """One key (the first: an attention sink) `lead` doublings ahead of 2^17 near-equal others, its value 0 and theirs near 1: all
    of the output comes from weights of 2^-lead. Enough sequences (one set of pages for all) that a warp or a CTA walks long
    stretches behind the sink's maximum.

    A weight is off by half a step of fp16, 2^-11 of itself, or below fp16's normal range by half of its least step:
    weights are at least 2^7 times what they are relative to the row's largest, so by 2^-25 / 2^7 = 2^-32 of the largest
    weight. Products and sums as in attn_ref.attention; the tensor cores add 16 terms a step, each cut at 2^-23 at most."""
    kv, size = (1 << 17) + 1, 128
    rng = np.random.default_rng(dim + hq)
    pages = -(-kv // size)
    shape = hc.kv_shape(pages, size, hk, dim)
    cache = torch.empty(hc.hc_kv_cache_size(shape), dtype=torch.uint8, device="cuda").fill_(0xFF)
    g = torch.Generator(device="cuda").manual_seed(dim)
    k = torch.randn((kv, hk, dim), generator=g, device="cuda", dtype=torch.bfloat16)
    v = 1 + 0.25 * torch.randn((kv, hk, dim), generator=g, device="cuda").bfloat16()
    k[:, :, 0] = 0
    k[0] = 0
    k[0, :, 0] = 6
    v[0] = 0
    slots = torch.arange(kv, device="cuda")
    hc.hc_kv_write(k, hk * dim, v, hk * dim, slots, kv, shape, cache)
    kq, vq = torch.empty_like(k), torch.empty_like(v)
    hc.hc_kv_read(cache, slots, kv, shape, kq, hk * dim, vq, hk * dim)
    one = 2.0 ** -9 * rng.standard_normal((q_len, hq, dim))
    one[:, :, 0] = 1
    one = ar.bf16(one)
    scale = float(np.float32(lead * np.log(2.0) / 6.0))
    n = seqs * q_len
    q = bf(np.tile(one, (seqs, 1, 1)))
    out, lse = gu.guarded((n, hq, dim)), gu.guarded((n, hq), torch.float32)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").repeat(seqs, 1)
    q_start = torch.arange(0, n + 1, q_len, dtype=torch.int32, device="cuda")
    a = hc.attention(n, seqs, q_len, pages, hq, scale)
    hc.hc_kv_attention(q, hq * dim, q_start, ints([kv] * seqs, torch.int32), table, cache, a, shape, out, hq * dim, lse,
                       hc.new_kv_workspace())
    got, glse = f64(out).reshape(seqs, q_len, hq, dim), f64(lse).reshape(seqs, q_len, hq)
    for h in range(hk):
        K, V = f64(kq[:, h]), f64(vq[:, h])
        for i in range(q_len):
            Q = one[i, h * (hq // hk):(h + 1) * (hq // hk)]
            m = kv - q_len + i + 1
            z = scale * (Q @ K[:m].T)
            top = z.max(-1, keepdims=True)
            w = np.exp(z - top)
            total = w.sum(-1, keepdims=True)
            assert (total < 1.5).all()  # the sink has most of the weight
            ref, rlse = (w @ V[:m]) / total, (top + np.log(total))[:, 0]
            dz = (dim + 16) * 2 * ar.U * scale * (np.abs(Q) @ np.abs(K[:m]).T).max() + 4 * ar.U * np.abs(z).max()
            dz += scale * np.abs(K).sum(-1).max() * 2.0 ** -32
            rel = 2 * dz + 2.0 ** -21 + (m / 32 + 64) * ar.U
            off = (w @ np.abs(V[:m])) / total * (ar.F16_HALF_STEP + 2 * rel + m / 16 * 2 * ar.U) + m * 2.0 ** -32 * np.abs(V).max() / total
            tol = off + ar.BF16_HALF_STEP * (np.abs(ref) + off)
            heads = slice(h * (hq // hk), (h + 1) * (hq // hk))
            err = np.abs(got[:, i, heads] - ref)
            assert (err <= tol).all(), (h, i, err.max(), tol.min(), np.abs(ref).mean())
            assert (np.abs(glse[:, i, heads] - rlse) <= rel + 8 * ar.U * np.abs(rlse)).all()
    assert hc.hc_device_error(clear=True) == 0
