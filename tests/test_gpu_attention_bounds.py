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


@pytest.mark.parametrize("lens", [[(1, 160), (3, 96)], [(120, 160), (140, 320)]], ids=["few", "many"])
@pytest.mark.parametrize("causal", [True, False])
def test_clamped_bounds_give_the_results_of_the_clamped_call(lens, causal):
    """Lengths past the table, rows past n, a start below 0: told of, and the results are those of the bounds as clamped."""
    def problem():
        return Problem(lens, 5, 1, 128, 32, seed=19).to_device()

    def check(p, page=False):
        out, lse = p.run(causal=causal)
        word = hc.hc_device_error(clear=True)
        assert word == (3 << 20 if page else 1 << 21)
        p.check(out, lse, causal=causal)
        m = int(p.q_start[-1])
        assert (out[m:] == 7).all() and (lse[m:] == 7).all()

    p = problem()  # keys past the table: as many as it has; the entry of its last page is -1
    p.d["kv_len"] = ints([10 ** 9, lens[1][1]], torch.int32)
    p.kv_len[0] = p.max_pages * 32
    check(p, page=True)
    p = problem()
    p.d["kv_len"] = ints([lens[0][1], -(2 ** 31)], torch.int32)
    p.kv_len[1] = 0
    check(p)
    p = problem()  # five rows more than there are
    p.d["q_start"] = ints([0, lens[0][0], p.n + 5], torch.int32)
    check(p)
    p = problem()  # two rows of q are not the call's: the last sequence is shorter, its queries still the last of its keys
    p.n -= 2
    p.q_start[2] -= 2
    check(p)
    p = problem()
    p.d["q_start"] = ints([-2, lens[0][0], p.n], torch.int32)
    check(p)
    p = problem()  # starts past n: no rows
    p.d["q_start"] = ints([0, lens[0][0], 2 ** 31 - 1], torch.int32)
    p.n = lens[0][0]
    p.q_start[2] = lens[0][0]
    check(p)


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
