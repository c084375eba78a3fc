"""The gated delta rule with one decay per head on the GPU (chunked forward and backward,
recurrent form, decode step) against the float64 recurrence and its adjoint.

Tolerances.  Errors are compared with the reference's RMS (largest |difference| / RMS).
  Chunked form: an operand's two fp16 terms are off by 2^-23 of the row's largest value and the
    dropped product of two second terms by 2^-22, 2^-21 together per product of largest values.
    With rows whose largest value is about four times their RMS and errors of random sign, a
    product is off by 16 * 2^-21 / sqrt(3) = 4.4e-6 of its RMS, the worst of 10^5 values by five
    times that, 2.2e-5; four products follow one another (K S, T R, P U and the state's), 9e-5:
    CHUNK = 1e-4.  dg and dbeta are differences of sums of such products that are a few times
    larger than what is left: DECAY = 3e-4.
  Recurrent form: fp32 sums of D = 128 terms, sqrt(128) * 2^-24 = 7e-7 of the RMS, five times that
    at worst, carried on for about ten tokens of memory: RECURRENT = 3e-5.
  16-bit outputs add half a step of their type: 2^-8 (bf16) or 2^-11 (fp16) of the value.
"""
import numpy as np
import pytest
import torch

from oracle import (gdr_recurrent, gdr_recurrent_backward, state_from_abi, state_to_abi)

pytestmark = pytest.mark.gpu

DEV = "cuda"
CHUNK, DECAY, RECURRENT = 1e-4, 3e-4, 3e-5
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
HALF_STEP = {BF16: 2.0 ** -8, F16: 2.0 ** -11, F32: 0.0}


@pytest.fixture(scope="module")
def kda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import gated_delta_rule_prologue_b200 as m
    return m


def f64(t):
    return t.detach().double().cpu().numpy()


class Problem:
    """Packed sequences on the GPU with `before` and `after` tokens outside every sequence."""

    def __init__(self, lens, HK=2, HV=4, D=128, dtype=BF16, seed=0, state=True, decay="mixed",
                 before=0, after=0, v_scale=1.0, qk=None):
        r = torch.Generator().manual_seed(seed)
        rn = lambda *s: torch.randn(s, generator=r)  # noqa: E731
        self.N, self.T = len(lens), before + sum(lens) + after
        self.lens, self.HK, self.HV, self.D, self.dtype = lens, HK, HV, D, dtype
        T = self.T
        cu = before + np.concatenate([[0], np.cumsum(lens)])
        self.cu_host = cu
        self.inside = np.zeros(T, bool)
        self.inside[cu[0]:cu[-1]] = True
        self.cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
        if self.N == 1 and before == 0 and after == 0:
            self.cu = None
        unit = lambda z: z / z.norm(dim=-1, keepdim=True)  # noqa: E731
        # keys with a common direction, as SiLU's outputs have
        q, k = unit(rn(T, HK, D) + 0.3), unit(rn(T, HK, D) + 0.3)
        if qk is not None:
            q, k = qk(q, k)
        self.q, self.k = q.to(dtype).to(DEV), k.to(dtype).to(DEV)
        self.v = (v_scale * rn(T, HV, D)).to(dtype).to(DEV)
        z = rn(T, HV)
        if decay == "mixed":   # from almost none to a fast one, head by head
            rate = torch.logspace(-3, 0.5, HV)
            g = -rate * torch.nn.functional.softplus(z)
        elif decay == "none":
            g = torch.zeros(T, HV)
        elif decay == "strong":
            g = -20.0 - 40.0 * torch.rand(T, HV, generator=r)
        elif decay == "resets":  # erased now and then, slow in between
            g = -0.01 * torch.rand(T, HV, generator=r)
            g[torch.rand(T, HV, generator=r) < 0.05] = -float("inf")
            g[torch.rand(T, HV, generator=r) < 0.05] = -1e4
        self.g = g.to(DEV)
        self.beta = torch.sigmoid(rn(T, HV)).to(DEV)
        self.s0 = (v_scale * 0.5 * rn(self.N, HV, D, D)).to(DEV) if state else None
        self.scale = 0.7
        self.o = torch.full((T, HV, D), 777.0, device=DEV)
        self.sN = torch.full((self.N, HV, D, D), 777.0, device=DEV)
        self.d_o = rn(T, HV, D).to(DEV)
        self.d_sN = rn(self.N, HV, D, D).to(DEV) if state else None

    def args(self):
        return (self.q, self.k, self.v, self.g, self.beta)

    def forward(self, fn, **kw):
        fn(*self.args(), self.o, scale=self.scale, initial_state=self.s0, final_state=self.sN,
           cu_seqlens=self.cu, **kw)
        torch.cuda.synchronize()

    def _ref(self):
        g = np.maximum(f64(self.g), -1e5)  # exp is 0 either way; the adjoint has no inf - inf
        s0 = None if self.s0 is None else state_from_abi(f64(self.s0))
        return (f64(self.q), f64(self.k), f64(self.v), g, f64(self.beta)), s0

    def reference(self):
        a, s0 = self._ref()
        o, last = gdr_recurrent(*a, self.scale, s0, self.cu_host)
        return o, state_to_abi(last)

    def reference_backward(self):
        a, s0 = self._ref()
        dsN = None if self.d_sN is None else state_from_abi(f64(self.d_sN))
        out = list(gdr_recurrent_backward(*a, f64(self.d_o), dsN, self.scale, s0, self.cu_host))
        out[5] = state_to_abi(out[5])
        return out

    def outputs(self):
        full = lambda like: torch.full_like(like, 777.0)  # noqa: E731
        return dict(dq=full(self.q), dk=full(self.k), dv=full(self.v), dg=full(self.g),
                    dbeta=full(self.beta), d_initial_state=full(self.sN))

    def backward(self, kda, **kw):
        out = kda.kda_gdr_chunk_bwd(*self.args(), self.d_o, scale=self.scale,
                                    initial_state=self.s0, d_final_state=self.d_sN,
                                    cu_seqlens=self.cu, **{**self.outputs(), **kw})
        torch.cuda.synchronize()
        return out

    def untouched(self, t):
        """Rows outside every sequence still hold what they held."""
        assert np.all(f64(t)[~self.inside] == float(torch.tensor(777.0).to(t.dtype)))


def close(name, got, ref, tol, dtype=F32):
    got = f64(got) if torch.is_tensor(got) else got
    if ref.size == 0:
        return
    assert np.all(np.isfinite(got)), name
    rms = np.sqrt(np.mean(ref * ref))
    bad = np.abs(got - ref) - HALF_STEP[dtype] * np.abs(ref)
    assert np.max(bad) <= tol * rms, (name, float(np.max(bad) / max(rms, 1e-300)))


def check_forward(p, tol):
    o, last = p.reference()
    close("o", f64(p.o)[p.inside], o[p.inside], tol)
    close("state", p.sN, last, tol)
    p.untouched(p.o)


def check_backward(p, got):
    ref = p.reference_backward()
    for name, x, y, tol, dt in zip(("dq", "dk", "dv", "dg", "dbeta", "ds0"), got, ref,
                                   (CHUNK, CHUNK, CHUNK, DECAY, DECAY, CHUNK),
                                   (p.dtype, p.dtype, p.dtype, F32, F32, F32)):
        if name != "ds0":
            p.untouched(x)
            x, y = f64(x)[p.inside], y[p.inside]
        close(name, x, y, tol, dt)


LENS = [130, 0, 1, 64, 63, 65, 17]


# ---- recurrent form --------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("HK,HV", [(1, 1), (2, 6)])
def test_recurrent(kda, dtype, D, HK, HV):
    p = Problem([5, 0, 1, 40], HK, HV, D, dtype, seed=D + HV)
    p.forward(kda.kda_gdr_recurrent)
    check_forward(p, RECURRENT)


def test_recurrent_whole_heads(kda):
    """More heads than two per SM: a CTA takes a whole head."""
    p = Problem([2, 1, 3], 50, 100, 128, BF16, seed=3)
    p.forward(kda.kda_gdr_recurrent)
    check_forward(p, RECURRENT)


@pytest.mark.parametrize("decay", ["none", "strong", "resets"])
def test_recurrent_decays(kda, decay):
    p = Problem([50], 1, 2, 64, F32, seed=4, decay=decay)
    p.forward(kda.kda_gdr_recurrent)
    check_forward(p, RECURRENT)


def test_recurrent_in_place_and_without_states(kda):
    p = Problem([9, 0, 3], seed=5, before=2, after=4)
    ref = p.reference()
    state = p.s0.clone()
    kda.kda_gdr_recurrent(*p.args(), p.o, scale=p.scale, initial_state=state, final_state=state,
                          cu_seqlens=p.cu)
    close("o", f64(p.o)[p.inside], ref[0][p.inside], RECURRENT)
    close("state", state, ref[1], RECURRENT)
    p.untouched(p.o)
    p.s0 = None
    kda.kda_gdr_recurrent(*p.args(), p.o, scale=p.scale, cu_seqlens=p.cu)
    close("o from zero", f64(p.o)[p.inside], p.reference()[0][p.inside], RECURRENT)


@pytest.mark.parametrize("N,HK,HV,D,dtype", [(1, 1, 1, 128, BF16), (7, 2, 4, 64, F16),
                                             (90, 4, 4, 128, BF16), (3, 1, 3, 16, F32)])
def test_decode_step(kda, N, HK, HV, D, dtype):
    p = Problem([1] * N, HK, HV, D, dtype, seed=N)
    ref = p.reference()
    state = p.s0.clone()
    kda.kda_gdr_decode_step(*p.args(), state, p.o, scale=p.scale)
    close("o", p.o, ref[0], RECURRENT)
    close("state", state, ref[1], RECURRENT)


# ---- chunked forward -------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("HK,HV,state", [(2, 2, True), (1, 4, False)])
def test_chunk_forward(kda, dtype, D, HK, HV, state):
    p = Problem(LENS, HK, HV, D, dtype, seed=D + HV, state=state, before=3, after=70)
    p.forward(kda.kda_gdr_chunk_fwd)
    check_forward(p, CHUNK)


@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 128, 500])
def test_chunk_forward_lengths(kda, T):
    p = Problem([T], 1, 2, 128, BF16, seed=T)
    p.forward(kda.kda_gdr_chunk_fwd)
    check_forward(p, CHUNK)


@pytest.mark.parametrize("decay", ["none", "strong", "resets"])
def test_chunk_forward_decays(kda, decay):
    p = Problem([150, 64], 2, 4, 128, BF16, seed=6, decay=decay)
    p.forward(kda.kda_gdr_chunk_fwd)
    check_forward(p, CHUNK)


def test_chunk_forward_whole_head_ctas(kda):
    """More chains than the split form takes (two CTAs per head up to 148)."""
    p = Problem([70, 3] * 20, 2, 4, 128, BF16, seed=7)
    p.forward(kda.kda_gdr_chunk_fwd)
    check_forward(p, CHUNK)


@pytest.mark.parametrize("lens,HV,D,dtype", [([2000], 2, 128, BF16), ([2113], 1, 64, F16),
                                             ([40, 1700, 0, 1100], 1, 128, F16),
                                             ([3000, 2900], 2, 64, BF16)])
@pytest.mark.parametrize("state", [True, False])
def test_chunk_forward_in_segments(kda, lens, HV, D, dtype, state):
    """Few long sequences: the state pass runs segments of them at once."""
    p = Problem(lens, 1, HV, D, dtype, seed=sum(lens), state=state, decay="mixed")
    p.g *= 0.3  # the slowest head's state outlives a segment
    p.forward(kda.kda_gdr_chunk_fwd)
    check_forward(p, CHUNK)


@pytest.mark.parametrize("beta", [0.0, 1.0])
def test_chunk_forward_beta_ends(kda, beta):
    p = Problem([100], 1, 2, 128, F16, seed=8, decay="none")
    p.beta.fill_(beta)
    p.forward(kda.kda_gdr_chunk_fwd)
    check_forward(p, CHUNK)
    if beta == 0.0:  # nothing is written and nothing decays: the state comes back as it was
        assert torch.equal(p.sN, p.s0)


def test_chunk_forward_equal_keys(kda):
    """The same unit key at every token: the triangular system at its stiffest."""
    p = Problem([129], 1, 2, 128, BF16, seed=9, decay="none",
                qk=lambda q, k: (q, k[:1].expand_as(k).contiguous()))
    p.forward(kda.kda_gdr_chunk_fwd)
    check_forward(p, CHUNK)


@pytest.mark.parametrize("power", [-60, 40])
def test_chunk_forward_values_of_any_size(kda, power):
    """Values and state times a power of two: the read-out and the state times the same power,
    bit for bit (every operand is scaled by its own row)."""
    p = Problem([150], 1, 2, 128, BF16, seed=10)
    p.forward(kda.kda_gdr_chunk_fwd)
    o, sN = p.o.clone(), p.sN.clone()
    p.v, p.s0 = p.v * 2.0 ** power, p.s0 * 2.0 ** power
    p.forward(kda.kda_gdr_chunk_fwd)
    assert torch.equal(p.o, o * 2.0 ** power) and torch.equal(p.sN, sN * 2.0 ** power)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_chunk_forward_large_values(kda, dtype):
    """Values of 10^4: products that fp16 could not hold."""
    p = Problem([150], 1, 2, 128, dtype, seed=11, v_scale=1e4)
    p.forward(kda.kda_gdr_chunk_fwd)
    check_forward(p, CHUNK)


def test_chunk_forward_nan_stays_in_its_sequence(kda):
    p = Problem([70, 70], 1, 2, 128, BF16, seed=12)
    p.forward(kda.kda_gdr_chunk_fwd)
    o, sN = p.o.clone(), p.sN.clone()
    p.v[100, 0, 5] = float("nan")  # the second sequence, head 0, channel 5
    p.forward(kda.kda_gdr_chunk_fwd)
    assert torch.equal(p.o[:70], o[:70]) and torch.equal(p.sN[0], sN[0])
    assert torch.equal(p.o[:, 1], o[:, 1])
    assert bool(torch.isnan(p.o[100:, 0, 5]).all())


def test_chunk_forward_equals_recurrent(kda):
    p = Problem([700, 90], 2, 4, 128, F16, seed=13)
    p.forward(kda.kda_gdr_recurrent)
    o, sN = f64(p.o), f64(p.sN)
    p.forward(kda.kda_gdr_chunk_fwd)
    close("o", p.o, o, CHUNK)
    close("state", p.sN, sN, CHUNK)


def test_chunk_forward_other_types_run_the_recurrent_form(kda):
    for D, dtype in ((32, BF16), (128, F32)):
        p = Problem([70, 2], 1, 2, D, dtype, seed=14)
        p.forward(kda.kda_gdr_recurrent)
        o, sN = p.o.clone(), p.sN.clone()
        p.forward(kda.kda_gdr_chunk_fwd)
        assert torch.equal(p.o, o) and torch.equal(p.sN, sN)


def test_chunk_forward_without_tokens(kda):
    p = Problem([0, 0], seed=15)
    p.forward(kda.kda_gdr_chunk_fwd)
    assert torch.equal(p.sN, p.s0)
    p.s0 = None
    p.forward(kda.kda_gdr_chunk_fwd)
    assert not bool(p.sN.any())


def test_chunk_forward_in_parts(kda):
    """A sequence in two calls that hand the state over, then single tokens."""
    p = Problem([300], 1, 2, 128, BF16, seed=16)
    ref = p.reference()
    state, o = p.s0.clone(), torch.empty_like(p.o)
    for a, b in ((0, 170), (170, 298)):
        kda.kda_gdr_chunk_fwd(*(x[a:b] for x in p.args()), o[a:b], scale=p.scale,
                              initial_state=state, final_state=state)
    for t in (298, 299):
        kda.kda_gdr_decode_step(*(x[t:t + 1] for x in p.args()), state, o[t:t + 1], scale=p.scale)
    close("o", o, ref[0], CHUNK)
    close("state", state, ref[1], CHUNK)


# ---- chunked backward ------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("HK,HV,state", [(2, 2, True), (1, 3, False)])
def test_chunk_backward(kda, dtype, D, HK, HV, state):
    p = Problem(LENS, HK, HV, D, dtype, seed=20 + D + HV, state=state, before=3, after=70)
    check_backward(p, p.backward(kda))


@pytest.mark.parametrize("T", [1, 64, 65, 400])
def test_chunk_backward_lengths(kda, T):
    p = Problem([T], 1, 2, 128, BF16, seed=30 + T)
    check_backward(p, p.backward(kda))


@pytest.mark.parametrize("decay", ["none", "strong", "resets"])
def test_chunk_backward_decays(kda, decay):
    p = Problem([150, 64], 2, 4, 128, BF16, seed=40, decay=decay)
    check_backward(p, p.backward(kda))


def test_chunk_backward_whole_head_ctas(kda):
    p = Problem([70, 3] * 20, 2, 4, 128, F16, seed=41)
    check_backward(p, p.backward(kda))


@pytest.mark.parametrize("beta", [0.0, 1.0])
def test_chunk_backward_beta_ends(kda, beta):
    """beta = 0 has a gradient of its own although nothing was written."""
    p = Problem([100], 1, 2, 128, F16, seed=42)
    p.beta.fill_(beta)
    got = p.backward(kda)
    check_backward(p, got)
    assert bool(got[4].any())


def test_chunk_backward_against_differences(kda):
    """Directional derivatives of the float64 recurrence, by central differences."""
    p = Problem([100], 1, 2, 64, F16, seed=43)
    got = p.backward(kda)
    a, s0 = p._ref()
    x = list(a) + [s0]
    r = np.random.default_rng(44)
    do, dsN = f64(p.d_o), state_from_abi(f64(p.d_sN))

    def loss(y):
        o, last = gdr_recurrent(*y[:5], p.scale, y[5], p.cu_host)
        return np.sum(do * o) + np.sum(dsN * last)

    for i, grad in enumerate(got):
        d = r.normal(size=x[i].shape)
        h = 1e-5
        up = loss([y + h * d if j == i else y for j, y in enumerate(x)])
        down = loss([y - h * d if j == i else y for j, y in enumerate(x)])
        slope = (up - down) / (2 * h)
        grad = f64(grad) if i < 5 else state_from_abi(f64(grad))
        # each element off by its rounding and DECAY of the RMS, with random signs
        size = np.sqrt(np.sum((np.abs(grad) * HALF_STEP[F16] * np.abs(d)) ** 2)
                       + np.sum((DECAY * np.sqrt(np.mean(grad ** 2)) * d) ** 2))
        assert abs(np.sum(grad * d) - slope) <= 5 * size + 1e-6 * abs(slope), i


def test_chunk_backward_without_the_states_gradient(kda):
    p = Problem([90], 1, 1, 64, BF16, seed=45)
    full = p.backward(kda)
    kw = p.outputs()
    kw.pop("d_initial_state")
    got = kda.kda_gdr_chunk_bwd(*p.args(), p.d_o, scale=p.scale, initial_state=p.s0,
                                d_final_state=p.d_sN, want_d_initial_state=False, **kw)
    assert got[5] is None
    for a, b in zip(got[:5], full[:5]):
        assert torch.equal(a, b)


# ---- calls -----------------------------------------------------------------------------

def test_dirty_workspaces_and_repeats_give_the_same_bits(kda):
    p = Problem(LENS, 1, 2, 128, BF16, seed=50)
    n = kda.kda_gdr_chunk_fwd_workspace_bytes(p.N, p.T, 1, 2, 128, BF16)
    m = kda.kda_gdr_chunk_bwd_workspace_bytes(p.N, p.T, 1, 2, 128, BF16)
    seen = []
    for fill in (0, 255, 127):
        ws = torch.full((n,), fill, dtype=torch.uint8, device=DEV)
        wb = torch.full((m,), fill, dtype=torch.uint8, device=DEV)
        p.forward(kda.kda_gdr_chunk_fwd, workspace=ws)
        seen.append([p.o.clone(), p.sN.clone()] + list(p.backward(kda, workspace=wb)))
    for other in seen[1:]:
        for a, b in zip(seen[0], other):
            assert torch.equal(a, b)


def test_two_streams_and_graphs(kda):
    """Two graphs with a workspace each, replayed on two streams at once on new inputs."""
    ps = [Problem([200, 70], 1, 2, 128, BF16, seed=60 + i) for i in range(2)]
    graphs, outs, kept = [], [], []  # a graph's workspaces live as long as it does
    for p in ps:
        ws = torch.empty(kda.kda_gdr_chunk_fwd_workspace_bytes(p.N, p.T, 1, 2, 128, BF16),
                         dtype=torch.uint8, device=DEV)
        wb = torch.empty(kda.kda_gdr_chunk_bwd_workspace_bytes(p.N, p.T, 1, 2, 128, BF16),
                         dtype=torch.uint8, device=DEV)
        out = p.outputs()
        p.forward(kda.kda_gdr_chunk_fwd, workspace=ws)
        p.backward(kda, workspace=wb, **out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            kda.kda_gdr_chunk_fwd(*p.args(), p.o, scale=p.scale, initial_state=p.s0,
                                  final_state=p.sN, cu_seqlens=p.cu, workspace=ws)
            kda.kda_gdr_chunk_bwd(*p.args(), p.d_o, scale=p.scale, initial_state=p.s0,
                                  d_final_state=p.d_sN, cu_seqlens=p.cu, workspace=wb, **out)
        graphs.append(graph)
        outs.append(out)
        kept += [ws, wb]
    new = [Problem([200, 70], 1, 2, 128, BF16, seed=70 + i) for i in range(2)]
    for p, q in zip(ps, new):
        for a, b in zip(p.args(), q.args()):
            a.copy_(b)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for p, out in zip(ps, outs):
        check_forward(p, CHUNK)
        check_backward(p, list(out.values()))


def test_runs_on_the_given_stream(kda):
    """The call waits for what was queued on its stream, and nothing else."""
    p = Problem([100], 1, 2, 128, BF16, seed=80)
    v = p.v.clone()
    p.v.zero_()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        p.v.copy_(v)
    kda.kda_gdr_chunk_fwd(*p.args(), p.o, scale=p.scale, initial_state=p.s0, final_state=p.sN,
                          stream=s, workspace=torch.empty(
                              kda.kda_gdr_chunk_fwd_workspace_bytes(1, 100, 1, 2, 128, BF16),
                              dtype=torch.uint8, device=DEV))
    s.synchronize()
    check_forward(p, CHUNK)


@pytest.mark.parametrize("cu", [[0, 90, 40, 100], [-5, 20, 60, 100], [0, 20, 60, 500]])
def test_malformed_cu_seqlens_are_reported(kda, cu):
    p = Problem([40, 30, 30], 1, 2, 128, BF16, seed=90)
    assert kda.kda_get_device_status() == 0
    p.cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
    p.forward(kda.kda_gdr_recurrent)
    assert kda.kda_get_device_status() == kda.KDA_ERR_DEVICE_BOUNDS
    p.forward(kda.kda_gdr_chunk_fwd)
    assert kda.kda_get_device_status() == kda.KDA_ERR_DEVICE_BOUNDS
    p.backward(kda)
    assert kda.kda_get_device_status() == kda.KDA_ERR_DEVICE_BOUNDS


def test_binding_checks_shapes(kda):
    p = Problem([40], 2, 4, 128, BF16, seed=91)
    ok = dict(scale=p.scale, initial_state=p.s0, final_state=p.sN)
    for i, wrong in ((1, p.k[:39]), (2, p.v[..., :64].contiguous()), (3, p.g[:, :3].contiguous()),
                     (4, p.beta[:39])):
        a = list(p.args())
        a[i] = wrong
        with pytest.raises(ValueError, match="shape"):
            kda.kda_gdr_chunk_fwd(*a, p.o, **ok)
    with pytest.raises(ValueError, match="contiguous"):
        kda.kda_gdr_recurrent(p.q.transpose(0, 1).contiguous().transpose(0, 1), *p.args()[1:], p.o,
                              **ok)
    with pytest.raises(TypeError, match="beta"):
        kda.kda_gdr_recurrent(*p.args()[:4], p.beta.double(), p.o, **ok)
    with pytest.raises(ValueError, match="initial_state"):
        kda.kda_gdr_recurrent(*p.args(), p.o, initial_state=p.s0[:, :2].contiguous())
    with pytest.raises(kda.KdaError, match="workspace holds"):
        kda.kda_gdr_chunk_fwd(*p.args(), p.o, **ok,
                              workspace=torch.empty(1024, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError, match="d_o"):
        kda.kda_gdr_chunk_bwd(*p.args(), p.d_o[:39])
