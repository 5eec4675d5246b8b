"""The attention over the 4-bit cache with bounds that are out of range: told of by the device error word, clamped, and
without a trace in the workspace. Tolerances: attn_ref.attention's."""

import pytest
import torch

import hyper_connection_residual_hc_gb300 as hc

import gpu_util as gu
from test_gpu_attention import Problem, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    hc.load()
    gu.device_error_clear()
    yield
    gu.device_error_clear()


@pytest.mark.parametrize("pairs,kv", [(50, 3200), (45, 6000)])
def test_decreasing_starts_leave_the_workspace_as_it_was(pairs, kv):
    """Starts that go back claim the same rows again and again, more row tiles than the call can have: told of, and calls
    that follow with the same workspace are not disturbed."""
    ws = hc.new_kv_workspace()
    good = Problem([(40, 5000), (300, 4000)], 5, 1, 128, 64, seed=24).to_device()
    out, lse = good.run(ws=ws)
    n = 1024
    p = Problem([(n, kv)], 1, 1, 64, 64, seed=25).to_device()
    seqs = 2 * pairs
    p.lens = [(n, kv)] * seqs
    p.d["q_start"] = ints([0, n] * pairs + [0], torch.int32)
    p.d["kv_len"] = ints([kv] * seqs, torch.int32)
    p.d["table"] = p.d["table"].repeat(seqs, 1).contiguous()
    p.run(causal=False, ws=ws)
    assert hc.hc_device_error(clear=True) == 1 << 21
    assert (ws[:2048] == 0).all()  # the counters
    again, lagain = good.run(ws=ws)
    assert torch.equal(out, again) and torch.equal(lse, lagain)
    assert hc.hc_device_error(clear=True) == 0


@pytest.mark.parametrize("hq,dim", [(1, 128), (16, 64), (3, 256)])
def test_decreasing_starts_of_few_queries(hq, dim):
    """The same by the kernel for few rows: more segments than the rows can have, and fewer."""
    ws = hc.new_kv_workspace()
    good = Problem([(1, 9000), (1, 700)], hq, 1, dim, 64, seed=26).to_device()
    out, lse = good.run(ws=ws)
    for n, seqs in ((20, 40), (20, 2), (2, 500)):
        p = Problem([(n, 900)], hq, 1, dim, 64, seed=27).to_device()
        p.lens = [(n, 900)] * seqs
        p.d["q_start"] = ints(([0, n] * seqs)[:seqs] + [0], torch.int32)
        p.d["kv_len"] = ints([900] * seqs, torch.int32)
        p.d["table"] = p.d["table"].repeat(seqs, 1).contiguous()
        got, _ = p.run(causal=False, max_q_len=1, ws=ws)
        assert hc.hc_device_error(clear=True) == 1 << 21
        p.d["q_start"] = ints([0] + [n] * seqs, torch.int32)  # the first sequence has all rows
        want, _ = p.run(causal=False, max_q_len=1, ws=ws)
        assert torch.equal(got, want) or (got == 7).all()
        assert (ws[:2048] == 0).all()
    again, lagain = good.run(ws=ws)
    assert torch.equal(out, again) and torch.equal(lse, lagain)
    assert hc.hc_device_error(clear=True) == 0
