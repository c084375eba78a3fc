"""Calls on an explicit stream that take their own scratch and outputs: the caller's stream goes on
allocating and writing while they wait and run, and neither side sees the other's memory."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16 = torch.bfloat16
T, H, D = 330, 2, 128
SCALE = 0.5


@pytest.fixture(scope="module")
def kda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import gated_delta_rule_prologue_b200 as m
    return m


@pytest.fixture(scope="module")
def data():
    r = torch.Generator(DEV).manual_seed(5)
    rn = lambda *s: torch.randn(s, generator=r, device=DEV)  # noqa: E731
    unit = lambda z: z / z.norm(dim=-1, keepdim=True)  # noqa: E731
    C = 3 * H * D
    return dict(q=unit(rn(T, H, D)).to(BF16), k=unit(rn(T, H, D)).to(BF16), v=rn(T, H, D).to(BF16),
                g=-torch.rand(T, H, generator=r, device=DEV),
                gk=-torch.rand(T, H, D, generator=r, device=DEV), beta=torch.sigmoid(rn(T, H)),
                raw=rn(T, H, D).to(BF16), x=rn(T, C).to(BF16), w=0.5 * rn(C, 4), d_o=rn(T, H, D),
                gate=rn(T, H, D).to(BF16), up=rn(T, H, D).to(BF16), weight=1 + 0.1 * rn(D),
                M=rn(1, H, D, D), B=rn(1, H, D, D))


def call(kda, name, a, stream):
    """The call on `stream`, and its outputs."""
    o = torch.zeros(T, H, D, device=DEV)
    st = dict(stream=stream)
    att = (a["q"], a["k"], a["v"])
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())  # o is there
        with torch.cuda.stream(stream):
            torch.cuda._sleep(10_000_000)
    if name == "gdr forward":
        kda.kda_gdr_chunk_fwd(*att, a["g"], a["beta"], o, scale=SCALE, **st)
        return [o]
    if name == "gdr backward":
        return list(kda.kda_gdr_chunk_bwd(*att, a["g"], a["beta"], a["d_o"], scale=SCALE, **st))
    if name == "prologue backward":
        dx, dw = torch.empty_like(a["x"]), torch.empty_like(a["w"])
        kda.kda_prologue_bwd(a["x"], a["w"], a["up"], a["gate"], a["v"], dx, dw, H=H, D=D, **st)
        return [dx, dw]
    if name == "epilogue backward":
        outs = [torch.empty_like(a["d_o"]), torch.empty_like(a["gate"]), torch.empty_like(a["weight"])]
        kda.kda_output_epilogue_bwd(a["d_o"], a["gate"], a["weight"], a["up"], *outs, **st)
        return outs
    if name == "chunk forward":
        kda.kda_chunk_fwd(*att, a["gk"], a["beta"], o, scale=SCALE, **st)
    elif name == "segmented":
        kda.kda_chunk_fwd(*att, a["gk"], a["beta"], o, scale=SCALE, segment_chunks=2, **st)
    elif name == "windowed":
        kda.kda_chunk_fwd(*att, a["gk"], a["beta"], o, scale=SCALE, window_chunks=2, **st)
    elif name == "gated":
        kda.kda_chunk_fwd_gated(*att, a["raw"], a["beta"], o, scale=SCALE, **st)
    elif name == "fused":
        kda.kda_prologue_chunk_fwd(a["x"], a["w"], a["gk"], a["beta"], o, H=H, D=D, scale=SCALE, **st)
    elif name == "fused windowed":
        kda.kda_prologue_chunk_fwd(a["x"], a["w"], a["gk"], a["beta"], o, H=H, D=D, scale=SCALE,
                                   window_chunks=2, **st)
    elif name == "fused gated":
        kda.kda_prologue_chunk_fwd_gated(a["x"], a["w"], a["raw"], a["beta"], o, H=H, D=D,
                                         scale=SCALE, **st)
    elif name == "chunk backward":
        return list(kda.kda_chunk_bwd(*att, a["gk"], a["beta"], a["d_o"], scale=SCALE, **st))
    elif name == "map":
        return list(kda.kda_chunk_map(*att, a["gk"], a["beta"], **st))
    elif name == "compose":
        return [kda.kda_state_compose(a["M"], a["B"], a["B"], **st)]
    return [o]


def sizes(kda):
    """Bytes that the calls take, for blocks of the caller's own."""
    f = [kda.kda_gdr_chunk_fwd_workspace_bytes(1, T, H, H, D, BF16),
         kda.kda_gdr_chunk_bwd_workspace_bytes(1, T, H, H, D, BF16),
         kda.kda_prologue_bwd_workspace_bytes(1, T, H, D, BF16),
         kda.kda_output_epilogue_bwd_workspace_bytes(T, H, D),
         kda.kda_chunk_fwd_workspace_bytes(1, T, H, D, D, 64, BF16),
         kda.kda_chunk_fwd_segmented_workspace_bytes(1, T, H, D, D, 64, BF16, 2),
         kda.kda_chunk_fwd_windowed_workspace_bytes(1, T, H, D, D, 64, BF16, 2),
         kda.kda_chunk_bwd_workspace_bytes(1, T, H, D, D, 64, BF16)]
    assert all(f)
    return f + [T * H * D * 4, T * H * D * 2, T * H * 4, H * D * D * 4]


@pytest.mark.parametrize("name", ["gdr forward", "gdr backward", "prologue backward", "epilogue backward",
                                  "chunk forward", "segmented", "windowed", "gated", "fused",
                                  "fused windowed", "fused gated", "chunk backward", "map", "compose"])
def test_scratch_belongs_to_the_calls_stream(kda, data, name):
    want = [None if x is None else x.clone() for x in call(kda, name, data, None)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = call(kda, name, data, side)
    held = [torch.full((n,), 255, dtype=torch.uint8, device=DEV) for n in sizes(kda) * 2]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert (a is None and b is None) or torch.equal(a, b)
    assert all(bool((x == 255).all()) for x in held)
    assert kda.kda_get_device_status() == 0


def test_outputs_that_are_dropped(kda, data):
    """Gradients that nobody keeps: the call still writes them, and into nothing else."""
    side = torch.cuda.Stream()
    for name in ("gdr backward", "chunk backward", "map"):
        call(kda, name, data, side)
        held = [torch.full((n,), 255, dtype=torch.uint8, device=DEV) for n in sizes(kda) * 4]
        torch.cuda.synchronize()
        assert all(bool((x == 255).all()) for x in held)


def test_another_librarys_stream(kda, data):
    """A stream that is known by its handle alone."""
    class Handle:
        def __init__(self, s):
            self.cuda_stream = s.cuda_stream

    want = call(kda, "gdr forward", data, None)[0].clone()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    o = torch.zeros(T, H, D, device=DEV)
    torch.cuda.synchronize()
    kda.kda_gdr_chunk_fwd(data["q"], data["k"], data["v"], data["g"], data["beta"], o, scale=SCALE,
                          stream=Handle(s))
    s.synchronize()
    assert torch.equal(o, want)
