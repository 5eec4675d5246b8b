"""The rotation's table (hc_prepare_rope) for small, large and negative frequencies, entry by entry and through
hc_qk_norm_rope at far positions.

Tolerances, derived before any run: an entry has the error that include/hc.h gives, 2^-52 of the frequency and 2^-65 turns,
against pi to 60 digits; a rotation that of test_gpu_attention.py, the table's error times the position and the angle's
2^-32 turns."""

from fractions import Fraction

import numpy as np
import pytest
import torch

import hyper_connection_residual_hc_gb300 as hc

import attn_ref as ar
import gpu_util as gu
from test_gpu_attention import bf, f64, ints

pytestmark = pytest.mark.gpu

PI = Fraction(314159265358979323846264338327950288419716939937510582097494, 10 ** 59)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    hc.load()


FREQS = [1.0, -1.0, 1e-6, -1e-6, 3e-9, -3e-9, 1e-17, -1e-17, 2.0 ** -60, -2.0 ** -60, 3.7, -3.7, 1e5 + 0.125, -(1e5 + 0.125), 0.0, -0.0]


def test_rope_table_is_as_near_as_stated():
    """Each entry is the frequency in turns as a fraction of 2^64, off by no more than 2^-52 of it and 2^-65 turns."""
    table = torch.empty(hc.hc_rope_table_size(32), dtype=torch.uint8, device="cuda")
    hc.hc_prepare_rope(FREQS, None, 32, 1, table)
    turns = table.cpu().numpy().view(np.uint64)[0::2]
    for f, t in zip(FREQS, turns):
        exact = Fraction(f) / (2 * PI)
        d = (Fraction(int(t), 1 << 64) - exact) % 1
        assert min(d, 1 - d) <= abs(exact) / (1 << 52) + Fraction(1, 1 << 65), (f, int(t), float(min(d, 1 - d)))


def test_norm_rope_of_small_and_negative_frequencies_far_away():
    rng = np.random.default_rng(8)
    n, h, dim, rot = 12, 2, 64, 32
    x = ar.bf16(rng.standard_normal((n, h, dim)))
    positions = rng.integers(-(1 << 46), 1 << 46, (1, n))
    table = torch.empty(hc.hc_rope_table_size(rot), dtype=torch.uint8, device="cuda")
    hc.hc_prepare_rope(FREQS, None, rot, 1, table)
    qo = gu.guarded((n, h, dim))
    hc.hc_qk_norm_rope(bf(x), h * dim, None, 0, None, None, ints(positions, torch.int64), hc.rope(table, rot), n, hc.heads(h, 0, dim), qo,
                       h * dim, None, 0)
    got = f64(qo)
    u = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + 1e-6)
    for j, f in enumerate(FREQS):
        exact = Fraction(f) / (2 * PI)
        for t in range(n):
            pos = int(positions[0, t])
            phi = 2 * np.pi * float(pos * exact % 1)
            a, b = u[t, :, j], u[t, :, j + rot // 2]
            slack = 2 * np.pi * (abs(pos) * (float(abs(exact)) * 2.0 ** -52 + 2.0 ** -65) + 2.0 ** -32)
            e = ((dim + 32) * ar.U + slack) * (np.abs(a) + np.abs(b))
            for col, ref in ((j, a * np.cos(phi) - b * np.sin(phi)), (j + rot // 2, b * np.cos(phi) + a * np.sin(phi))):
                assert (np.abs(got[t, :, col] - ref) <= e + ar.BF16_HALF_STEP * (np.abs(ref) + e)).all(), (f, pos)
