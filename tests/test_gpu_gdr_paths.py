"""The forms that the chunked gated delta rule's state pass takes by its sizes: whole sequences on
the tensor memory (D = 128 and more heads than fit two CTAs each on the SMs), and a few long
sequences in segments.  Both through the cases that the small sizes of test_gpu_gdr.py cover for
the form of two CTAs per head; the tolerances are derived there.

A segment's first state is one product further from its inputs per segment before it, M_g E_g of two
split operands; the state decays or is corrected on its way, so the errors of the earlier products
shrink with it and CHUNK, which counts four products in a row, holds: the scan's is one more in place
of the chunks' it stands for.
"""
import pytest
import torch

from test_gpu_gdr import BF16, CHUNK, DEV, F16, Problem, check_backward, check_forward, kda

pytestmark = pytest.mark.gpu
__all__ = ["kda"]  # the fixture

MANY = [70, 3, 0, 64, 129, 1] * 4     # 24 sequences, HV = 4: 96 chains
LONG = [40, 1700, 0, 1100]            # cut into segments for up to four heads
FORMS = [(MANY, 2, 4), (LONG, 1, 2)]
ids = dict(ids=["tensor memory", "segments"])


def problem(lens, HK, HV, **kw):
    p = Problem(lens, HK, HV, 128, **kw)
    if lens is LONG:
        p.g *= 0.3  # the slowest head's state outlives a segment
    return p


def is_cut(kda, p):
    """A segment's M, B and first state add to the records' bytes, which grow with N alone else."""
    size = [kda.kda_gdr_chunk_fwd_workspace_bytes(n, p.T, p.HK, p.HV, p.D, p.dtype)
            for n in (p.N, 1000, 1001)]
    return size[0] > size[1] - (1000 - p.N) * (size[2] - size[1])


@pytest.mark.parametrize("lens,HK,HV,cut", [(MANY, 2, 4, False), (LONG, 1, 2, True), (LONG, 1, 1, True),
                                            ([1400, 1400, 1200], 1, 1, True)])
def test_the_cases_take_their_form(kda, lens, HK, HV, cut):
    assert is_cut(kda, Problem(lens, HK, HV, 128)) == cut


def workspace(kda, p, fill=255):
    n = kda.kda_gdr_chunk_fwd_workspace_bytes(p.N, p.T, p.HK, p.HV, p.D, p.dtype)
    return torch.full((n,), fill, dtype=torch.uint8, device=DEV)


@pytest.mark.parametrize("lens,HK,HV", FORMS, **ids)
@pytest.mark.parametrize("decay", ["none", "strong", "resets"])
def test_decays(kda, lens, HK, HV, decay):
    p = problem(lens, HK, HV, dtype=F16, seed=1, decay=decay)
    p.forward(kda.kda_gdr_chunk_fwd)
    check_forward(p, CHUNK)


@pytest.mark.parametrize("lens,HK,HV", FORMS, **ids)
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("state", [True, False])
def test_tokens_outside_every_sequence(kda, lens, HK, HV, dtype, state):
    p = problem(lens, HK, HV, dtype=dtype, seed=2, before=5, after=130, state=state)
    p.forward(kda.kda_gdr_chunk_fwd)
    check_forward(p, CHUNK)


@pytest.mark.parametrize("lens,HK,HV", FORMS, **ids)
def test_state_in_place(kda, lens, HK, HV):
    """The last states into the first ones' buffer: the same bits as into their own."""
    p = problem(lens, HK, HV, dtype=BF16, seed=3)
    p.forward(kda.kda_gdr_chunk_fwd)
    o, sN = p.o.clone(), p.sN.clone()
    for _ in range(3):
        state = p.s0.clone()
        p.o.fill_(777.0)
        kda.kda_gdr_chunk_fwd(*p.args(), p.o, scale=p.scale, initial_state=state,
                              final_state=state, cu_seqlens=p.cu, workspace=workspace(kda, p))
        assert torch.equal(p.o, o) and torch.equal(state, sN)


@pytest.mark.parametrize("lens,HK,HV", FORMS, **ids)
def test_without_the_last_states(kda, lens, HK, HV):
    p = problem(lens, HK, HV, dtype=BF16, seed=4)
    p.forward(kda.kda_gdr_chunk_fwd)
    o = p.o.clone()
    kda.kda_gdr_chunk_fwd(*p.args(), p.o.fill_(777.0), scale=p.scale, initial_state=p.s0,
                          cu_seqlens=p.cu)
    assert torch.equal(p.o, o)


@pytest.mark.parametrize("lens,HK,HV", FORMS, **ids)
@pytest.mark.parametrize("power", [-60, 40])
def test_values_of_any_size(kda, lens, HK, HV, power):
    p = problem(lens, HK, HV, dtype=BF16, seed=5)
    p.forward(kda.kda_gdr_chunk_fwd)
    o, sN = p.o.clone(), p.sN.clone()
    p.v, p.s0 = p.v * 2.0 ** power, p.s0 * 2.0 ** power
    p.forward(kda.kda_gdr_chunk_fwd)
    assert torch.equal(p.o, o * 2.0 ** power) and torch.equal(p.sN, sN * 2.0 ** power)


@pytest.mark.parametrize("lens,HK,HV", FORMS, **ids)
@pytest.mark.parametrize("place", [2, -1])
def test_nan_stays_in_its_channel_and_sequence(kda, lens, HK, HV, place):
    """A value that is not a number: from its chunk of 64 tokens on, in its channel alone."""
    p = problem(lens, HK, HV, dtype=BF16, seed=6)
    p.forward(kda.kda_gdr_chunk_fwd)
    o, sN = p.o.clone(), p.sN.clone()
    n = 1
    a, b = int(p.cu_host[n]), int(p.cu_host[n + 1])
    t = (b if place < 0 else a) + place
    p.v[t, 0, 5] = float("nan")
    p.forward(kda.kda_gdr_chunk_fwd)
    assert bool(torch.isnan(p.o[t:b, 0, 5]).all()) and bool(torch.isnan(p.sN[n, 0, 5]).all())
    first = a + (t - a) // 64 * 64
    p.o[first:b, 0, 5], p.sN[n, 0, 5] = o[first:b, 0, 5], sN[n, 0, 5]
    assert torch.equal(p.o, o) and torch.equal(p.sN, sN)


@pytest.mark.parametrize("lens,HK,HV", FORMS, **ids)
def test_dirty_workspaces_and_graphs(kda, lens, HK, HV):
    """Equal bits from any workspace contents, and from a graph replayed on other inputs."""
    p, q = (problem(lens, HK, HV, dtype=BF16, seed=s) for s in (7, 8))
    q.forward(kda.kda_gdr_chunk_fwd)
    want = q.o.clone(), q.sN.clone()
    for fill in (0, 127):
        q.forward(kda.kda_gdr_chunk_fwd, workspace=workspace(kda, q, fill))
        assert torch.equal(q.o, want[0]) and torch.equal(q.sN, want[1])
    ws = workspace(kda, p)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.kda_gdr_chunk_fwd(*p.args(), p.o, scale=p.scale, initial_state=p.s0,
                              final_state=p.sN, cu_seqlens=p.cu, workspace=ws)
    for a, b in zip(p.args() + (p.s0,), q.args() + (q.s0,)):
        a.copy_(b)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(p.o, want[0]) and torch.equal(p.sN, want[1])


@pytest.mark.parametrize("lens,HK,HV", FORMS, **ids)
def test_other_sequences_do_not_change_the_bits(kda, lens, HK, HV):
    """A sequence's results with other values beside it."""
    p = problem(lens, HK, HV, dtype=F16, seed=9)
    p.forward(kda.kda_gdr_chunk_fwd)
    a, b = int(p.cu_host[1]), int(p.cu_host[2])
    o, sN = p.o[a:b].clone(), p.sN[1].clone()
    r = problem(lens, HK, HV, dtype=F16, seed=10)
    for x, y in zip(p.args(), r.args()):
        x[:a], x[b:] = y[:a], y[b:]
    p.forward(kda.kda_gdr_chunk_fwd)
    assert torch.equal(p.o[a:b], o) and torch.equal(p.sN[1], sN)


@pytest.mark.parametrize("decay", ["none", "strong", "resets"])
def test_backward_decays(kda, decay):
    p = Problem(MANY, 2, 4, 128, F16, seed=11, decay=decay)
    check_backward(p, p.backward(kda))


@pytest.mark.parametrize("state", [True, False])
def test_backward_outside_every_sequence(kda, state):
    p = Problem(MANY, 1, 4, 128, BF16, seed=12, before=5, after=130, state=state)
    check_backward(p, p.backward(kda))


def test_more_sequences_than_are_ranked(kda):
    """Up to 64 sequences start longest first, more as they come."""
    for lens in ([3, 70, 1, 0, 65] * 14, [3, 70, 1, 0, 65] * 12 + [64] * 4):
        p = Problem(lens, 1, 2, 128, BF16, seed=16)
        p.forward(kda.kda_gdr_chunk_fwd)
        check_forward(p, CHUNK)
        check_backward(p, p.backward(kda))


def test_backward_of_a_long_sequence(kda):
    p = Problem([1500], 1, 1, 128, BF16, seed=13)
    p.g *= 0.3
    check_backward(p, p.backward(kda))


@pytest.mark.parametrize("cu", [[0, 3900, 40, 4000], [-5, 20, 3600, 4000], [0, 20, 3600, 1 << 30]])
def test_malformed_cu_seqlens_are_reported_by_segments(kda, cu):
    p = problem([1400, 1400, 1200], 1, 1, dtype=BF16, seed=14)
    assert kda.kda_get_device_status() == 0
    p.cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
    p.forward(kda.kda_gdr_chunk_fwd)
    assert kda.kda_get_device_status() == kda.KDA_ERR_DEVICE_BOUNDS


@pytest.mark.parametrize("cu", [[0, 90, 40, 100], [-5, 20, 60, 100], [0, 20, 60, 1 << 30]])
def test_malformed_cu_seqlens_are_reported_by_the_tensor_memory_form(kda, cu):
    p = Problem([40, 30, 30], 1, 32, 128, BF16, seed=15)
    assert kda.kda_get_device_status() == 0
    p.cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
    p.forward(kda.kda_gdr_chunk_fwd)
    assert kda.kda_get_device_status() == kda.KDA_ERR_DEVICE_BOUNDS
    p.backward(kda)
    assert kda.kda_get_device_status() == kda.KDA_ERR_DEVICE_BOUNDS
