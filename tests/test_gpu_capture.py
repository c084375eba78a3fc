"""The operators with a second kernel behind the first in captured graphs, whatever stands before them in the
graph: nothing, a memset, a copy, another kernel; with tokens and without."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16 = torch.bfloat16
H, D = 2, 128


@pytest.fixture(scope="module")
def kda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import gated_delta_rule_prologue_b200 as m
    return m


def operator(kda, name, T):
    """The call, and its outputs."""
    r = torch.Generator(DEV).manual_seed(T)
    rn = lambda *s: torch.randn(s, generator=r, device=DEV)  # noqa: E731
    bf = lambda *s: rn(*s).to(BF16)  # noqa: E731
    ws = torch.empty(1 << 24, dtype=torch.uint8, device=DEV)
    if name == "epilogue backward":
        o, gate, w, d = rn(T, H, D), bf(T, H, D), rn(D), bf(T, H, D)
        out = [torch.empty_like(o), torch.empty_like(gate), torch.empty_like(w)]
        return lambda: kda.kda_output_epilogue_bwd(o, gate, w, d, *out, workspace=ws), out
    if name == "prologue backward":
        x, w, cache = bf(T, 3 * H * D), rn(3 * H * D, 4), bf(1, 3, 3 * H * D)
        up = [bf(T, H, D) for _ in range(3)]
        out = [torch.empty_like(x), torch.empty_like(w), torch.empty_like(cache)]
        return lambda: kda.kda_prologue_bwd(x, w, *up, out[0], out[1], H=H, D=D, cache_in=cache,
                                            d_cache_in=out[2], workspace=ws), out
    q, k = (torch.nn.functional.normalize(rn(T, H, D), dim=-1).to(BF16) for _ in range(2))
    v, g, beta, s0 = bf(T, H, D), -torch.rand(T, H, device=DEV), torch.rand(T, H, device=DEV), rn(1, H, D, D)
    if name == "chunk forward":
        out = [torch.empty(T, H, D, device=DEV), torch.empty_like(s0)]
        return lambda: kda.kda_gdr_chunk_fwd(q, k, v, g, beta, out[0], initial_state=s0,
                                             final_state=out[1], workspace=ws), out
    d_o, d_s = rn(T, H, D), rn(1, H, D, D)
    out = [torch.empty_like(x) for x in (q, k, v, g, beta, s0)]
    return lambda: kda.kda_gdr_chunk_bwd(
        q, k, v, g, beta, d_o, initial_state=s0, d_final_state=d_s, workspace=ws,
        **dict(zip(("dq", "dk", "dv", "dg", "dbeta", "d_initial_state"), out))), out


@pytest.mark.parametrize("name,T", [("epilogue backward", 0), ("epilogue backward", 3),
                                    ("epilogue backward", 900), ("prologue backward", 0),
                                    ("prologue backward", 2), ("prologue backward", 300),
                                    ("chunk forward", 0), ("chunk forward", 100),
                                    ("chunk forward", 1500), ("chunk backward", 200)])
@pytest.mark.parametrize("before", ["nothing", "memset", "copy", "kernel", "itself"])
def test_captured_behind_anything(kda, name, T, before):
    call, out = operator(kda, name, T)
    call()
    torch.cuda.synchronize()
    want = [x.clone() for x in out]
    a, b = torch.ones(1 << 20, device=DEV), torch.zeros(1 << 20, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        if before == "memset":
            a.zero_()
        elif before == "copy":
            b.copy_(a)
        elif before == "kernel":
            b.add_(1.0)
        elif before == "itself":
            call()
        call()
    for _ in range(2):
        for x in out:
            x.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(out, want):
            assert torch.equal(x, y)
    assert kda.kda_get_device_status() == 0
