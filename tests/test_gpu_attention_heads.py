"""The attention over the 4-bit cache with many query heads to a kv head, single tokens and drafts: up to the 128 that are
allowed, where one query fills tiles of rows on its own. Tolerances: attn_ref.attention's."""

import pytest
import torch

import hyper_connection_residual_hc_gb300 as hc

import gpu_util as gu
from test_gpu_attention import Problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    hc.load()
    gu.device_error_clear()
    yield
    gu.device_error_clear()


@pytest.mark.parametrize("window", [0, 30])
@pytest.mark.parametrize("hq,hk,dim", [(64, 1, 64), (96, 2, 128), (128, 1, 128), (128, 1, 64), (128, 1, 256), (36, 1, 256)])
def test_attention_of_many_heads_to_a_kv_head(hq, hk, dim, window):
    p = Problem([(1, 70), (1, 0), (3, 50), (5, 2), (0, 9), (1, 33)], hq, hk, dim, 16, seed=hq + dim, extra_rows=1).to_device()
    out, lse = p.run(window=window)
    p.check(out, lse, window=window)
    m = int(p.q_start[-1])
    assert (out[m:] == 7).all() and (lse[m:] == 7).all()
    assert hc.hc_device_error(clear=True) == 0


@pytest.mark.parametrize("hq,hk,dim", [(128, 1, 128), (100, 1, 64), (128, 1, 256)])
def test_attention_of_many_heads_over_long_contexts_and_chunks(hq, hk, dim):
    """Keys in slices, and chunks among single tokens."""
    for lens in ([(1, 5000)], [(1, 70), (40, 1300), (2, 33), (1, 2100)]):
        p = Problem(lens, hq, hk, dim, 64, seed=hq + dim).to_device()
        out, lse = p.run()
        p.check(out, lse)
        again, lagain = p.run()
        assert torch.equal(out, again) and torch.equal(lse, lagain)
    assert hc.hc_device_error(clear=True) == 0
