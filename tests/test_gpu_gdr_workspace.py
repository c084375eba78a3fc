"""One workspace for many sizes of the chunked one-decay rule.  The size that is asked for is the fastest
form's, which holds maps and states of segments for few long sequences and nothing of them for others, so it
does not grow with the sizes; what has to be there, the chunks' records, does.  A workspace for the largest
sizes therefore serves all smaller ones."""
import pytest
import torch

from test_gpu_gdr import BF16, CHUNK, DEV, F16, Problem, check_forward, kda

pytestmark = pytest.mark.gpu
__all__ = ["kda"]  # the fixture


def need(kda, p):
    return kda.kda_gdr_chunk_fwd_workspace_bytes(p.N, p.T, p.HK, p.HV, p.D, p.dtype)


def records(kda, p):
    """Bytes of the records alone: sizes of so many sequences that nothing is cut grow by one slot each."""
    a, b = (kda.kda_gdr_chunk_fwd_workspace_bytes(n, p.T, p.HK, p.HV, p.D, p.dtype) for n in (1000, 1001))
    return a - (1000 - p.N) * (b - a)


@pytest.mark.parametrize("D,HK,HV,lens,smaller", [
    (128, 2, 2, [3000] + [1] * 74, [[1700, 1300], [1000] * 3, [3000], [64] * 40, [1]]),
    (64, 1, 4, [350, 325, 325], [[500, 500], [1000], [700], [65, 3]]),
    (128, 8, 8, [704], [[640], [512], [300, 300]]),
])
def test_the_largest_sizes_workspace_serves_the_smaller(kda, D, HK, HV, lens, smaller):
    big = Problem(lens, HK, HV, D, BF16, seed=1)
    ws = torch.full((need(kda, big),), 255, dtype=torch.uint8, device=DEV)
    short = False
    for i, few in enumerate([lens] + smaller):
        p = Problem(few, HK, HV, D, BF16, seed=2 + i)
        p.g *= 0.3
        short = short or need(kda, p) > ws.numel()
        p.forward(kda.kda_gdr_chunk_fwd, workspace=ws)
        check_forward(p, CHUNK)
    assert short  # some smaller size asks for more than there is


@pytest.mark.parametrize("D,lens", [(128, [2500]), (64, [3000, 1500])])
def test_any_workspace_that_holds_the_records(kda, D, lens):
    """From the records alone to all that the fastest form takes; nothing behind its end is written, and
    equal calls give equal bits."""
    p = Problem(lens, 1, 2, D, F16, seed=9)
    p.g *= 0.3
    least, most = records(kda, p), need(kda, p)
    assert least < most
    for n in sorted({least, least + 16, (least + most) // 32 * 16, most - 16, most, most + 64}):
        buf = torch.full((n + 256,), 201, dtype=torch.uint8, device=DEV)
        seen = []
        for _ in range(2):
            p.o.fill_(777.0)
            p.forward(kda.kda_gdr_chunk_fwd, workspace=buf[:n])
            check_forward(p, CHUNK)
            seen.append((p.o.clone(), p.sN.clone()))
        assert bool((buf[n:] == 201).all())
        assert torch.equal(seen[0][0], seen[1][0]) and torch.equal(seen[0][1], seen[1][1])
    with pytest.raises(kda.KdaError, match="workspace holds"):
        p.forward(kda.kda_gdr_chunk_fwd,
                  workspace=torch.empty(least - 1, dtype=torch.uint8, device=DEV))


def test_graphs_of_two_sizes_share_a_workspace_in_turn(kda):
    """A captured call keeps the form that it was captured with."""
    a, b = Problem([2500], 1, 2, 128, BF16, seed=11), Problem([30, 40], 1, 2, 128, BF16, seed=12)
    ws = torch.empty(max(records(kda, a), need(kda, b)), dtype=torch.uint8, device=DEV)
    graphs = []
    for p in (a, b):
        p.g *= 0.3
        p.forward(kda.kda_gdr_chunk_fwd, workspace=ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            kda.kda_gdr_chunk_fwd(*p.args(), p.o, scale=p.scale, initial_state=p.s0, final_state=p.sN,
                                  cu_seqlens=p.cu, workspace=ws)
        graphs.append(graph)
    for p in (a, b):
        p.o.fill_(777.0)
    for _ in range(2):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    check_forward(a, CHUNK)
    check_forward(b, CHUNK)
