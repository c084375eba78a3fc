"""The chunked one-decay rule row by row: what one token, or one key channel, gets is as
exact for itself where others of the same 64-token chunk are larger by many powers of two.

dq of a token is made of its own d_o alone, with the state's key channels and the other tokens' keys and
corrected values, so it grows and shrinks with it: divided by its d_o's power of two, every token's errors
are those of test_gpu_gdr.py, CHUNK of the RMS of all tokens' rows so divided (three products that follow
one another, counted there as four) and half a step of the output's type.  A single row's own RMS is no
measure: a token with few others in reach has a row that is one dot product of d_o and U times a key,
and dot products of 128 terms come out a hundred times below their terms' size here and there.
A key channel of dq and dk where the keys and queries are zero is made of that channel of the two states
alone, and errors are relative to that channel's own.
"""
import numpy as np
import pytest
import torch

from test_gpu_gdr import BF16, CHUNK, DEV, F16, Problem, check_backward, close, f64, kda

pytestmark = pytest.mark.gpu
__all__ = ["kda"]  # the fixture


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("HK,HV", [(2, 2), (1, 3)])
@pytest.mark.parametrize("state", [True, False])
@pytest.mark.parametrize("order", ["up", "down", "mixed"])
def test_dq_of_tokens_with_small_gradients(kda, D, HK, HV, state, order):
    """d_o of a chunk's tokens from 2^-24 to 1, as weights of a loss per token give them."""
    T = 150
    p = Problem([T], HK, HV, D, BF16, seed=D + HV, state=state)
    power = torch.linspace(-24, 0, 64).repeat(3)[:T]
    if order == "down":
        power = -24 - power
    elif order == "mixed":
        power = power[torch.randperm(T, generator=torch.Generator().manual_seed(1))]
    size = 2.0 ** power.round()
    p.d_o *= size.to(DEV)[:, None, None]
    got = p.backward(kda)
    ref = p.reference_backward()
    check_backward(p, got)
    size = size.double().numpy()[:, None, None]
    close("dq for its size", f64(got[0]) / size, ref[0] / size, CHUNK, p.dtype)


def test_tokens_without_a_gradient(kda):
    """d_o of zero: dq of zero, whatever the others have."""
    p = Problem([100], 1, 2, 128, BF16, seed=3)
    p.d_o[::3] = 0.0
    p.d_o[1::3] *= 2.0 ** 60
    got = p.backward(kda)
    assert not bool(got[0][::3].any())
    check_backward(p, got)


@pytest.mark.parametrize("D", [64, 128])
def test_key_channels_of_small_states(kda, D):
    """Key channels that keys and queries leave alone, with states 2^-20 of the others'."""
    p = Problem([100], 2, 2, D, BF16, seed=D)
    few = slice(0, D, 4)
    for x in (p.q, p.k):
        x[..., few] = 0.0
    for x in (p.s0, p.d_sN):
        x[..., few] *= 2.0 ** -20
    got = p.backward(kda)
    ref = p.reference_backward()
    check_backward(p, got)
    for i, name in ((0, "dq"), (1, "dk")):
        x, y = f64(got[i])[..., few], ref[i][..., few]
        assert np.sqrt(np.mean(y * y)) < 2.0 ** -14 * np.sqrt(np.mean(ref[i] ** 2))
        close(name, x, y, CHUNK, p.dtype)


@pytest.mark.parametrize("power", [-60, 40])
def test_gradients_of_any_size(kda, power):
    """d_o and the last states' gradient times a power of two: all gradients times the same power."""
    p = Problem([150], 1, 2, 128, BF16, seed=10)
    one = [x.clone() for x in p.backward(kda)]
    p.d_o, p.d_sN = p.d_o * 2.0 ** power, p.d_sN * 2.0 ** power
    for a, b in zip(p.backward(kda), one):
        assert torch.equal(a.float(), b.float() * 2.0 ** power)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128])
def test_read_out_of_tokens_with_small_queries_and_keys(kda, dtype, D):
    """Queries and keys of norms from 2^-8 to 1 in one chunk: a token's read-out for its query's size.

    fp16 inputs are exact.  bf16 values below 2^-14 of the tile's largest are off by 2^-25 of it: in a
    query of norm 2^-8 that is the twentieth of its values below 2^-6 of its largest (a quarter to a third
    of its norm), and the read-out is off by sqrt(128 / 20) * 2^-25 * 0.35 / sqrt(3) * 2^8 = 4e-6 of its
    RMS, five times that at worst, 2e-5 beside CHUNK."""
    T = 150
    r = torch.Generator().manual_seed(D)
    size, ksize = (2.0 ** -torch.randint(0, 9, (T,), generator=r) for _ in range(2))
    p = Problem([T], 2, 4, D, dtype, seed=D,
                qk=lambda q, k: (q * size[:, None, None], k * ksize[:, None, None]))
    p.forward(kda.kda_gdr_chunk_fwd)
    o, last = p.reference()
    size = size.double().numpy()[:, None, None]
    close("o for its size", f64(p.o) / size, o / size, CHUNK + 2e-5)
    close("state", p.sN, last, CHUNK + 2e-5)
