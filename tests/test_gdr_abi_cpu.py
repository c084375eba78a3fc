"""Argument checks of the kda_gdr_* entry points and of the backward passes of the prologue and
the output epilogue, without a GPU: every call here is refused before anything is launched."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch


@pytest.fixture(scope="module")
def kda():
    import __graft_entry__
    __graft_entry__.build()
    import gated_delta_rule_prologue_b200 as m
    return m


def at(i):
    """A fake 16-byte aligned address, 1 TiB from the next; never dereferenced."""
    return ctypes.c_void_p((i + 1) << 40)


def refused(kda, status, code, text):
    assert status == code, (status, kda.lib.kda_last_error())
    assert text in kda.lib.kda_last_error(), kda.lib.kda_last_error()


def gdr(kda, fn="kda_gdr_recurrent", **over):
    a = dict(q=at(0), k=at(1), v=at(2), g=at(3), beta=at(4), s0=None, cu=at(5), N=2, T=100, HK=2,
             HV=4, D=128, dt=1, o=at(6), sN=None, ws=at(7), nbytes=1 << 40)
    a.update(over)
    head = (a["q"], a["k"], a["v"], a["g"], a["beta"], 1.0, a["s0"], a["cu"], a["N"], a["T"],
            a["HK"], a["HV"], a["D"], a["dt"])
    tail = (a["ws"], a["nbytes"], None) if fn.endswith("_ws") else (None,)
    return getattr(kda.lib, fn)(*head, a["o"], a["sN"], *tail)


@pytest.mark.parametrize("fn", ["kda_gdr_recurrent", "kda_gdr_chunk_fwd_ws"])
@pytest.mark.parametrize("over,code,text", [
    (dict(q=None), 1, b"q is NULL"),
    (dict(k=ctypes.c_void_p(8 + (2 << 40))), 1, b"k is not 16-byte aligned"),
    (dict(g=ctypes.c_void_p(2 + (4 << 40))), 1, b"g is not 4-byte aligned"),
    (dict(beta=None), 1, b"beta is NULL"),
    (dict(o=None), 1, b"o is NULL"),
    (dict(cu=None), 1, b"cu_seqlens is NULL but N=2"),
    (dict(cu=ctypes.c_void_p(2 + (6 << 40))), 1, b"cu_seqlens is not 4-byte aligned"),
    (dict(N=0), 1, b"bad sizes"),
    (dict(T=-1), 1, b"bad sizes"),
    (dict(HK=0), 1, b"bad sizes"),
    (dict(HK=3), 1, b"HV=4 is not a multiple of HK=3"),
    (dict(HK=8), 1, b"HV=4 is not a multiple of HK=8"),
    (dict(D=96), 2, b"D=96"),
    (dict(dt=7), 1, b"unknown dtype"),
    (dict(N=1 << 28), 1, b"too large"),
    (dict(o=at(2)), 1, b"o overlaps v"),
    (dict(o=at(0)), 1, b"o overlaps q"),
    (dict(sN=at(6)), 1, b"o overlaps final_state"),
    (dict(s0=at(8), sN=ctypes.c_void_p(4096 + (9 << 40))), 1, b"final_state overlaps initial_state"),
    (dict(sN=at(5)), 1, b"final_state overlaps cu_seqlens"),
])
def test_forward_refuses(kda, fn, over, code, text):
    refused(kda, gdr(kda, fn, **over), code, text)


def test_chunk_forward_refuses_its_workspace(kda):
    need = kda.lib.kda_gdr_chunk_fwd_workspace_bytes(2, 100, 2, 4, 128, 1)
    assert need > 0
    fn = "kda_gdr_chunk_fwd_ws"
    refused(kda, gdr(kda, fn, nbytes=need - 1), 1, b"workspace holds")
    refused(kda, gdr(kda, fn, ws=ctypes.c_void_p(8 + (8 << 40))), 1, b"workspace is not 16-byte")
    refused(kda, gdr(kda, fn, ws=at(6)), 1, b"o overlaps workspace")
    refused(kda, gdr(kda, fn, ws=at(1)), 1, b"workspace overlaps k")
    refused(kda, gdr(kda, fn, ws=at(8), s0=at(8)), 1, b"workspace overlaps initial_state")


def test_workspace_sizes(kda):
    f, b = kda.lib.kda_gdr_chunk_fwd_workspace_bytes, kda.lib.kda_gdr_chunk_bwd_workspace_bytes
    for fn in (f, b):
        assert fn(1, 100, 2, 4, 128, 1) > 0 and fn(1, 100, 2, 4, 64, 2) > 0
        # types, sizes and arguments without a chunked form
        for a in ((1, 100, 2, 4, 128, 0), (1, 100, 2, 4, 32, 1), (1, 0, 2, 4, 128, 1),
                  (0, 100, 2, 4, 128, 1), (1, 100, 3, 4, 128, 1), (1, 100, 2, 4, 128, 9)):
            assert fn(*a) == 0, a
    # every sequence adds its own ragged chunk (the forward's one long sequence is cut, with segments'
    # maps and states in its workspace, so it is compared where nothing is cut)
    assert b(9, 1000, 2, 4, 128, 1) > b(1, 1000, 2, 4, 128, 1)
    assert f(9, 100, 2, 4, 128, 1) > f(1, 100, 2, 4, 128, 1)
    assert f(1, 1000, 2, 4, 128, 1) > f(9, 1000, 2, 4, 128, 1)
    assert b(1, 1000, 2, 4, 128, 1) > f(1, 1000, 2, 4, 128, 1)
    # sizes whose records pass 32 bits
    assert f(1, 1 << 20, 64, 64, 128, 1) > 1 << 32
    assert kda.kda_gdr_chunk_fwd_workspace_bytes(1, 100, 2, 4, 128, torch.bfloat16) == \
        f(1, 100, 2, 4, 128, 1)


def test_decode_step_refuses(kda):
    def step(state=at(5), N=3, HK=2, HV=4, D=128, dt=1, o=at(6), q=at(0)):
        return kda.lib.kda_gdr_decode_step(q, at(1), at(2), at(3), at(4), 1.0, state, N, HK, HV, D,
                                           dt, o, None)
    refused(kda, step(state=None), 1, b"state is NULL")
    refused(kda, step(q=None), 1, b"q is NULL")
    refused(kda, step(N=0), 1, b"bad sizes")
    refused(kda, step(HV=5), 1, b"multiple")
    refused(kda, step(D=256), 2, b"D=256")
    refused(kda, step(o=at(5)), 1, b"o overlaps final_state")
    refused(kda, step(state=at(2)), 1, b"overlaps v")


def bwd(kda, **over):
    a = dict(q=at(0), k=at(1), v=at(2), g=at(3), beta=at(4), s0=None, cu=at(5), N=2, T=100, HK=2,
             HV=4, D=128, dt=1, do=at(6), dsN=None, dq=at(7), dk=at(8), dv=at(9), dg=at(10),
             db=at(11), ds0=None, ws=at(12), nbytes=1 << 40)
    a.update(over)
    return kda.lib.kda_gdr_chunk_bwd_ws(
        a["q"], a["k"], a["v"], a["g"], a["beta"], 1.0, a["s0"], a["cu"], a["N"], a["T"], a["HK"],
        a["HV"], a["D"], a["dt"], a["do"], a["dsN"], a["dq"], a["dk"], a["dv"], a["dg"], a["db"],
        a["ds0"], a["ws"], a["nbytes"], None)


@pytest.mark.parametrize("over,code,text", [
    (dict(dt=0), 2, b"needs bf16/f16"),
    (dict(D=32), 2, b"needs bf16/f16"),
    (dict(T=0), 2, b"T > 0"),
    (dict(D=48), 2, b"D=48"),
    (dict(HK=3), 1, b"multiple"),
    (dict(cu=None), 1, b"cu_seqlens is NULL"),
    (dict(do=None), 1, b"d_o is NULL"),
    (dict(dq=None), 1, b"dq is NULL"),
    (dict(dg=None), 1, b"dg is NULL"),
    (dict(db=ctypes.c_void_p(1 + (12 << 40))), 1, b"dbeta is not 4-byte aligned"),
    (dict(ws=None), 1, b"workspace is NULL"),
    (dict(nbytes=1000), 1, b"workspace holds"),
    (dict(dq=at(0)), 1, b"dq overlaps q"),
    (dict(dk=at(7)), 1, b"dq overlaps dk"),
    (dict(dv=at(6)), 1, b"dv overlaps d_o"),
    (dict(s0=at(13), ds0=at(13)), 1, b"d_initial_state overlaps initial_state"),
    (dict(dsN=at(13), ds0=at(13)), 1, b"d_initial_state overlaps d_final_state"),
    (dict(ws=at(11)), 1, b"dbeta overlaps workspace"),
])
def test_backward_refuses(kda, over, code, text):
    refused(kda, bwd(kda, **over), code, text)


def pro(kda, **over):
    a = dict(x=at(0), w=at(1), ci=None, cu=None, N=1, T=100, H=2, D=128, dt=1, gdt=0, dq=at(2),
             dk=at(3), dv=at(4), dx=at(5), dw=at(6), dc=None, ws=at(7), nbytes=1 << 40)
    a.update(over)
    return kda.lib.kda_prologue_bwd(a["x"], a["w"], a["ci"], a["cu"], a["N"], a["T"], a["H"], a["D"],
                                    a["dt"], a["gdt"], a["dq"], a["dk"], a["dv"], a["dx"], a["dw"],
                                    a["dc"], a["ws"], a["nbytes"], None)


@pytest.mark.parametrize("over,code,text", [
    (dict(dt=5), 1, b"unknown dtype"),
    (dict(gdt=5), 1, b"unknown gradient dtype"),
    (dict(N=2), 1, b"cu_seqlens is NULL"),
    (dict(T=-1), 1, b"bad sizes"),
    (dict(D=100), 2, b"D=100"),
    (dict(H=1 << 25), 1, b"too large"),
    (dict(x=None), 1, b"x is NULL"),
    (dict(w=None), 1, b"conv_w is NULL"),
    (dict(dx=ctypes.c_void_p(8 + (6 << 40))), 1, b"dx is not 16-byte aligned"),
    (dict(ws=None, T=100000), 1, b"workspace is NULL"),
    (dict(nbytes=16, T=100000), 1, b"workspace holds"),
    (dict(dx=at(0)), 1, b"dx overlaps x"),
    (dict(dx=at(3)), 1, b"dx overlaps dk"),
    (dict(ci=at(8), dc=at(8)), 1, b"d_cache_in overlaps cache_in"),
    (dict(dw=at(1)), 1, b"d_conv_w overlaps conv_w"),
])
def test_prologue_backward_refuses(kda, over, code, text):
    refused(kda, pro(kda, **over), code, text)


def epi(kda, **over):
    a = dict(o=at(0), gate=at(1), w=at(2), eps=1e-5, d=at(3), T=10000, H=2, D=128, dt=1, do=at(4),
             dg=at(5), dw=at(6), ws=at(7), nbytes=1 << 40)
    a.update(over)
    return kda.lib.kda_output_epilogue_bwd(a["o"], a["gate"], a["w"], a["eps"], a["d"], a["T"],
                                           a["H"], a["D"], a["dt"], a["do"], a["dg"], a["dw"],
                                           a["ws"], a["nbytes"], None)


@pytest.mark.parametrize("over,code,text", [
    (dict(dt=3), 1, b"unknown dtype"),
    (dict(H=0), 1, b"bad sizes"),
    (dict(D=8), 2, b"D=8"),
    (dict(eps=-1.0), 1, b"eps"),
    (dict(eps=float("nan")), 1, b"eps"),
    (dict(w=None), 1, b"weight is NULL"),
    (dict(d=None), 1, b"d_out is NULL"),
    (dict(do=None), 1, b"d_o is NULL"),
    (dict(ws=None), 1, b"workspace is NULL"),
    (dict(nbytes=8), 1, b"workspace holds"),
    (dict(do=at(0)), 1, b"d_o overlaps o"),
    (dict(dg=at(1)), 1, b"d_gate overlaps gate"),
    (dict(dg=at(4)), 1, b"d_o overlaps d_gate"),
])
def test_epilogue_backward_refuses(kda, over, code, text):
    refused(kda, epi(kda, **over), code, text)


def test_binding_refuses_cpu_tensors(kda):
    q = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_gdr_recurrent(q, q, q, torch.zeros(4, 2), torch.zeros(4, 2), q)
    with pytest.raises(ValueError, match="three dimensions"):
        kda.kda_gdr_chunk_fwd(q[0], q[0], q[0], q, q, q)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_output_epilogue_bwd(q, q, q[0, 0], q, q, q)


def test_chunk_forward_refuses_less_than_the_records(kda):
    """Few long sequences: the size that is asked for holds segments beside the records, and what is
    refused is what does not hold the records."""
    f = kda.lib.kda_gdr_chunk_fwd_workspace_bytes
    records = f(1000, 4000, 1, 2, 128, 1) - 999 * (f(1001, 4000, 1, 2, 128, 1) - f(1000, 4000, 1, 2, 128, 1))
    assert f(1, 4000, 1, 2, 128, 1) > records
    refused(kda, gdr(kda, "kda_gdr_chunk_fwd_ws", N=1, T=4000, HK=1, HV=2, nbytes=records - 1), 1,
            b"workspace holds %d bytes, these sizes need %d" % (records - 1, records))


def test_loads_on_a_torch_without_cuda(kda):
    """Where torch has no CUDA functions the module loads and its calls refuse what they are given."""
    code = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
import gated_delta_rule_prologue_b200 as kda
x = torch.zeros(4, 2, 64)
for call in (lambda: kda.kda_gdr_recurrent(x, x, x, x[..., 0], x[..., 0], x),
             lambda: kda.kda_chunk_fwd(x, x, x, x, x[..., 0].contiguous(), x),
             lambda: kda.kda_output_epilogue_bwd(x, x, x[0, 0], x, x, x)):
    try:
        call()
    except ValueError as e:
        assert "CUDA" in str(e), e
    else:
        raise AssertionError("not refused")
print("loaded")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert r.returncode == 0 and "loaded" in r.stdout, r.stderr[-2000:]
