"""Calls from several host threads at once, each with its own stream and workspace."""
import threading

import pytest
import torch

from test_gpu_gdr import BF16, DEV, Problem, kda

pytestmark = pytest.mark.gpu
__all__ = ["kda"]  # the fixture


def run_together(jobs, times):
    """Every job, `times` times, each in a thread of its own; the errors that they raised."""
    errors = []

    def work(job):
        try:
            for _ in range(times):
                job()
        except Exception as e:  # noqa: BLE001: whatever it is, the test reports it
            errors.append(e)

    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return errors


@pytest.mark.parametrize("backward", [False, True])
def test_sizes_that_launch_one_kernel_differently(kda, backward):
    """D = 64 with few chains and with more than there are SMs: the state pass's shared memory differs,
    and one thread's launch has no say in the other's."""
    ps = [Problem([70], 1, 2, 64, BF16, seed=1), Problem([3, 70] * 20, 1, 4, 64, BF16, seed=2)]
    jobs, seen = [], []
    for p in ps:
        s = torch.cuda.Stream()
        size = kda.kda_gdr_chunk_bwd_workspace_bytes if backward else kda.kda_gdr_chunk_fwd_workspace_bytes
        ws = torch.empty(size(p.N, p.T, p.HK, p.HV, p.D, p.dtype), dtype=torch.uint8, device=DEV)
        out = p.outputs()

        def job(p=p, s=s, ws=ws, out=out):
            if backward:
                kda.kda_gdr_chunk_bwd(*p.args(), p.d_o, scale=p.scale, initial_state=p.s0,
                                      d_final_state=p.d_sN, cu_seqlens=p.cu, workspace=ws, stream=s, **out)
            else:
                kda.kda_gdr_chunk_fwd(*p.args(), p.o, scale=p.scale, initial_state=p.s0,
                                      final_state=p.sN, cu_seqlens=p.cu, workspace=ws, stream=s)

        def results(p=p, out=out):
            return [x.clone() for x in (out.values() if backward else (p.o, p.sN))]

        torch.cuda.synchronize()
        job()
        torch.cuda.synchronize()
        jobs.append(job)
        seen.append((results, results()))
    assert not run_together(jobs, 3000)
    for results, want in seen:
        for a, b in zip(results(), want):
            assert torch.equal(a, b)
    assert kda.kda_get_device_status() == 0
