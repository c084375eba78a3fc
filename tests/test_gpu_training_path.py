"""Backward passes of the prologue and of the output epilogue on the GPU against the float64
oracle, and the whole path of a layer: prologue, gated delta rule, epilogue and back again.

Tolerances: fp32 outputs within FP32 = 2e-5 of the reference's RMS plus 2e-6 of the value (a few
dozen fp32 operations of 2^-24 and approximate exponential, reciprocal and root of a few 2^-23
each; sums of up to 10^3 terms, 10^3 * 2^-24 at worst); 16-bit outputs half a step of their type
more, 2^-8 (bf16) or 2^-11 (fp16) of the value.
"""
import numpy as np
import pytest
import torch

from oracle import (gdr_recurrent, gdr_recurrent_backward, output_epilogue,
                    output_epilogue_backward, prologue, prologue_backward, state_from_abi,
                    state_to_abi)

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
FP32 = 2e-5
HALF_STEP = {BF16: 2.0 ** -8, F16: 2.0 ** -11, F32: 0.0}


@pytest.fixture(scope="module")
def kda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import gated_delta_rule_prologue_b200 as m
    return m


def f64(t):
    return t.detach().double().cpu().numpy()


def close(name, got, ref, tol=FP32):
    dtype = got.dtype
    got = f64(got)
    assert np.all(np.isfinite(got)), name
    if ref.size == 0:
        return
    rms = np.sqrt(np.mean(ref * ref))
    bad = np.abs(got - ref) - (HALF_STEP[dtype] + 2e-6) * np.abs(ref)
    assert np.max(bad) <= tol * rms, (name, float(np.max(bad) / max(rms, 1e-300)))


class Pro:
    def __init__(self, lens, H, D, dtype, grad, cache, seed):
        r = torch.Generator().manual_seed(seed)
        rn = lambda *s: torch.randn(s, generator=r)  # noqa: E731
        self.H, self.D, self.N, self.T, C = H, D, len(lens), sum(lens), 3 * H * D
        self.cu_host = np.concatenate([[0], np.cumsum(lens)])
        self.cu = None if len(lens) == 1 else torch.tensor(self.cu_host, dtype=torch.int32, device=DEV)
        self.x = rn(self.T, C).to(dtype).to(DEV)
        self.w = (0.5 * rn(C, 4)).to(DEV)
        self.cache = rn(self.N, 3, C).to(dtype).to(DEV) if cache else None
        self.up = [rn(self.T, H, D).to(grad).to(DEV) for _ in range(3)]
        full = lambda t: torch.full_like(t, 777.0)  # noqa: E731
        self.dx, self.dw = full(self.x), full(self.w)
        self.dcache = full(self.cache) if cache else None

    def run(self, kda, **kw):
        kda.kda_prologue_bwd(self.x, self.w, *self.up, self.dx, self.dw, H=self.H, D=self.D,
                             cache_in=self.cache, d_cache_in=self.dcache, cu_seqlens=self.cu, **kw)
        torch.cuda.synchronize()

    def check(self):
        ref = prologue_backward(f64(self.x), f64(self.w), *map(f64, self.up), self.H, self.D,
                                self.cu_host, None if self.cache is None else f64(self.cache))
        close("dx", self.dx, ref[0])
        close("dw", self.dw, ref[1])
        if self.dcache is not None:
            close("dcache", self.dcache, ref[2])


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("grad", [BF16, F16, F32])
@pytest.mark.parametrize("D", [16, 32, 64, 128])
def test_prologue_backward(kda, dtype, grad, D):
    p = Pro([30, 0, 1, 2, 41, 3], 2, D, dtype, grad, True, seed=D)
    p.run(kda)
    p.check()


@pytest.mark.parametrize("T", [1, 2, 3, 4, 15, 16, 17, 31, 33, 300])
@pytest.mark.parametrize("cache", [False, True])
def test_prologue_backward_lengths(kda, T, cache):
    """Lengths around the tiles' ends."""
    p = Pro([T], 1, 64, BF16, F32, cache, seed=100 + T)
    p.run(kda)
    p.check()


def test_prologue_backward_long_tiles(kda):
    """Enough channels that a tile is longer than the shortest one, sequences that end inside."""
    p = Pro([200, 77, 0, 300, 1, 22], 24, 128, BF16, BF16, True, seed=120)
    p.run(kda)
    p.check()


def test_prologue_backward_of_no_tokens(kda):
    p = Pro([0, 0], 1, 64, F16, F16, True, seed=121)
    p.run(kda)
    assert not bool(p.dw.any()) and not bool(p.dcache.any())


def test_prologue_backward_without_the_weights_gradient(kda):
    p = Pro([100, 33], 2, 128, BF16, F32, False, seed=122)
    p.run(kda)
    dx = p.dx.clone()
    p.dx.fill_(777.0)
    kda.kda_prologue_bwd(p.x, p.w, *p.up, p.dx, H=p.H, D=p.D, cu_seqlens=p.cu, workspace=None)
    assert torch.equal(p.dx, dx)


def test_prologue_backward_extreme_inputs(kda):
    """SiLU far out on both sides, and a head of zeros (the norm's epsilon)."""
    p = Pro([40], 2, 32, F32, F32, False, seed=123)
    p.x[:, :32] = 0.0
    p.x[5, 40] = 80.0
    p.x[9, 41] = -80.0
    p.run(kda)
    p.check()


def test_prologue_backward_refuses_sequences_that_do_not_cover_the_tokens(kda):
    p = Pro([30, 20], 1, 32, F32, F32, False, seed=124)
    assert kda.kda_get_device_status() == 0
    p.cu = torch.tensor([0, 30, 45], dtype=torch.int32, device=DEV)
    p.run(kda)
    assert kda.kda_get_device_status() == kda.KDA_ERR_DEVICE_BOUNDS


def epilogue_problem(T, H, D, dtype, seed):
    r = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=r)  # noqa: E731
    o, gate = 2.0 * rn(T, H, D), (3.0 * rn(T, H, D)).to(dtype)
    return [x.to(DEV) for x in (o, gate, 1.0 + 0.2 * rn(D), rn(T, H, D).to(dtype))]


def epilogue_run(kda, o, gate, weight, d, **kw):
    d_o, d_gate = torch.full_like(o, 777.0), torch.full_like(gate, 777.0)
    d_weight = torch.full_like(weight, 777.0)
    kda.kda_output_epilogue_bwd(o, gate, weight, d, d_o, d_gate, d_weight, eps=1e-3, **kw)
    torch.cuda.synchronize()
    return d_o, d_gate, d_weight


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("T,H", [(1, 1), (7, 3), (301, 2), (1000, 9)])
def test_epilogue_backward(kda, dtype, D, T, H):
    o, gate, weight, d = epilogue_problem(T, H, D, dtype, seed=T + D)
    o[0, 0] = 0.0  # a row of zeros
    if T > 1:
        gate[1, 0, :4] = torch.tensor([60.0, -60.0, 1000.0, -1000.0])
    got = epilogue_run(kda, o, gate, weight, d)
    ref = output_epilogue_backward(f64(o), f64(gate), f64(weight), f64(d), 1e-3)
    for name, x, y in zip(("d_o", "d_gate", "d_weight"), got, ref):
        close(name, x, y)


def test_epilogue_backward_repeats_and_optional_weight(kda):
    o, gate, weight, d = epilogue_problem(5000, 4, 128, BF16, seed=9)
    a = epilogue_run(kda, o, gate, weight, d)
    ws = torch.full((kda.kda_output_epilogue_bwd_workspace_bytes(5000, 4, 128),), 255,
                    dtype=torch.uint8, device=DEV)
    b = epilogue_run(kda, o, gate, weight, d, workspace=ws)
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    d_o, d_gate = torch.empty_like(o), torch.empty_like(gate)
    kda.kda_output_epilogue_bwd(o, gate, weight, d, d_o, d_gate, eps=1e-3, workspace=None)
    assert torch.equal(d_o, a[0]) and torch.equal(d_gate, a[1])
    empty = [x[:0] for x in (o, gate)]
    got = epilogue_run(kda, empty[0], empty[1], weight, d[:0])
    assert not bool(got[2].any())


@pytest.mark.parametrize("captured", [False, True])
def test_layer_there_and_back(kda, captured):
    """Projections through prologue, chunked gated delta rule and epilogue, the gradients of a
    loss back to the projections and every parameter, and generation on from the prefill's state
    and conv cache; once eagerly and once as a captured and replayed graph.

    Every operator's outputs are compared with the float64 oracle on the tensors that the path
    stored before it, so each comparison has the tolerance of its one operator: FP32 here and
    in the epilogue, CHUNK = 1e-4 and DECAY = 3e-4 of the RMS for the chunked rule (as in
    test_gpu_gdr.py)."""
    CHUNK, DECAY = 1e-4, 3e-4
    H, D, lens = 2, 128, [150, 0, 1, 90]
    N, T, C = len(lens), sum(lens), 3 * H * D
    r = torch.Generator().manual_seed(130)
    rn = lambda *s: torch.randn(s, generator=r)  # noqa: E731
    cu_host = np.concatenate([[0], np.cumsum(lens)])
    cu = torch.tensor(cu_host, dtype=torch.int32, device=DEV)
    x, w = rn(T, C).to(BF16).to(DEV), (0.5 * rn(C, 4)).to(DEV)
    g = (-0.3 * torch.rand(T, H, generator=r)).to(DEV)
    beta = torch.sigmoid(rn(T, H)).to(DEV)
    gate, weight = rn(T, H, D).to(BF16).to(DEV), (1 + 0.1 * rn(D)).to(DEV)
    d_out = rn(T, H, D).to(BF16).to(DEV)
    scale = D ** -0.5
    q = torch.empty((T, H, D), dtype=F16, device=DEV)
    k, v = torch.empty_like(q), torch.empty_like(q)
    cache = torch.empty((N, 3, C), dtype=BF16, device=DEV)
    o, state = torch.empty((T, H, D), device=DEV), torch.empty((N, H, D, D), device=DEV)
    out, d_o = torch.empty_like(gate), torch.empty_like(o)
    d_gate, d_weight = torch.empty_like(gate), torch.empty_like(weight)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    grads = [torch.empty_like(t) for t in (q, k, v, g, beta)]

    def step():
        kda.kda_prologue(x, w, q, k, v, H=H, D=D, cache_out=cache, cu_seqlens=cu)
        kda.kda_gdr_chunk_fwd(q, k, v, g, beta, o, scale=scale, final_state=state, cu_seqlens=cu)
        kda.kda_output_epilogue(o, gate, weight, out)
        kda.kda_output_epilogue_bwd(o, gate, weight, d_out, d_o, d_gate, d_weight)
        kda.kda_gdr_chunk_bwd(q, k, v, g, beta, d_o, scale=scale, cu_seqlens=cu,
                              want_d_initial_state=False, dq=grads[0], dk=grads[1], dv=grads[2],
                              dg=grads[3], dbeta=grads[4])
        kda.kda_prologue_bwd(x, w, *grads[:3], dx, dw, H=H, D=D, cu_seqlens=cu)

    step()
    if captured:
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for t in (q, o, state, out, d_o, dx, dw, *grads):
            t.fill_(777.0)
        graph.replay()
    torch.cuda.synchronize()
    assert kda.kda_get_device_status() == 0

    for name, got, ref in zip("qkv", (q, k, v), prologue(f64(x), f64(w), H, D, cu_host)):
        close(name, got, ref)
    rule = (f64(q), f64(k), f64(v), f64(g), f64(beta))
    o_ref, s_ref = gdr_recurrent(*rule, scale, None, cu_host)
    close("o", o, o_ref, CHUNK)
    close("state", state, state_to_abi(s_ref), CHUNK)
    close("out", out, output_epilogue(f64(o), f64(gate), f64(weight), 1e-5))
    ref = output_epilogue_backward(f64(o), f64(gate), f64(weight), f64(d_out), 1e-5)
    for name, got, want in zip(("d_o", "d_gate", "d_weight"), (d_o, d_gate, d_weight), ref):
        close(name, got, want)
    ref = gdr_recurrent_backward(*rule, f64(d_o), None, scale, None, cu_host)
    for name, got, want in zip(("dq", "dk", "dv", "dg", "dbeta"), grads, ref):
        close(name, got, want, CHUNK if got.dtype == F16 else DECAY)
    ref = prologue_backward(f64(x), f64(w), *map(f64, grads[:3]), H, D, cu_host)
    close("dx", dx, ref[0])
    close("dw", dw, ref[1])

    # Three more tokens for every sequence: prologue with the cache, then the decode step.
    one = torch.arange(N + 1, dtype=torch.int32, device=DEV)
    s_now = state_from_abi(f64(state))
    for i in range(3):
        xt = rn(N, C).to(BF16).to(DEV)
        gt, bt = (-0.3 * torch.rand(N, H, generator=r)).to(DEV), torch.sigmoid(rn(N, H)).to(DEV)
        qt, kt, vt = (torch.empty((N, H, D), dtype=F16, device=DEV) for _ in range(3))
        nxt, ot = torch.empty_like(cache), torch.empty((N, H, D), device=DEV)
        kda.kda_prologue(xt, w, qt, kt, vt, H=H, D=D, cache_in=cache, cache_out=nxt, cu_seqlens=one)
        kda.kda_gdr_decode_step(qt, kt, vt, gt, bt, state, ot, scale=scale)
        ref = prologue(f64(xt), f64(w), H, D, np.arange(N + 1), f64(cache))
        for name, got, want in zip("qkv", (qt, kt, vt), ref):
            close("decoded " + name, got, want)
        cache = nxt
        on, s_now = gdr_recurrent(f64(qt), f64(kt), f64(vt), f64(gt), f64(bt), scale, s_now,
                                  np.arange(N + 1))
        close("decoded o", ot, on, CHUNK)
    close("decoded state", state, state_to_abi(s_now), CHUNK)
