"""Launches whose chains do not all run at once take the sequences longest first, up to 64 of them: the
boundary, with equal lengths and empty sequences, and every kernel that ranks them (the tensor-memory state
pass and the whole-head reverse pass at D = 128, the state pass at D = 64)."""
import pytest

from test_gpu_gdr import BF16, CHUNK, F16, Problem, check_backward, check_forward, kda

pytestmark = pytest.mark.gpu
__all__ = ["kda"]  # the fixture

HV = 4  # more chains than there are SMs from 38 sequences on


def lengths(n):
    return ([3, 70, 1, 0, 65, 65, 130, 0] * n)[:n]


@pytest.mark.parametrize("D,dtype", [(128, BF16), (64, F16)])
@pytest.mark.parametrize("N", [38, 64, 65])
def test_more_chains_than_run_at_once(kda, D, dtype, N):
    assert N * HV > 148
    p = Problem(lengths(N), 2, HV, D, dtype, seed=N + D, before=2, after=5)
    p.forward(kda.kda_gdr_chunk_fwd)
    check_forward(p, CHUNK)
    check_backward(p, p.backward(kda))
    assert kda.kda_get_device_status() == 0


@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("N", [64, 65])
def test_lengths_in_either_order(kda, D, N):
    """One long sequence at the end, or at the start, among equal ones."""
    for lens in ([64] * (N - 1) + [400], [400] + [64] * (N - 1), [0] * (N - 1) + [90]):
        p = Problem(lens, 1, HV, D, BF16, seed=N)
        p.forward(kda.kda_gdr_chunk_fwd)
        check_forward(p, CHUNK)
        check_backward(p, p.backward(kda))
