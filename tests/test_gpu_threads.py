"""Calls from several host threads at once: the binding lets go of the interpreter while a C entry point runs."""
import os
import subprocess
import threading

import pytest
import torch

from _harness import moe

pytestmark = pytest.mark.gpu

CALLS = 1000


def _together(jobs):
    """Runs each job CALLS times in a thread of its own, on a stream of its own; what the threads raised."""
    start, raised = threading.Barrier(len(jobs)), []

    def work(job):
        stream = torch.cuda.Stream()
        torch.zeros(1, device="cuda")        # the thread has a CUDA context of its own accord
        start.wait()
        try:
            for i in range(CALLS):
                job(stream)
                if i % 200 == 199:
                    stream.synchronize()
        except Exception as e:  # noqa: BLE001 (what the main thread is told)
            raised.append(e)

    threads = [threading.Thread(target=work, args=(job,)) for job in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return raised


def _layer_job(m, T, K, status):
    """moe_layer_few_tokens, whose kernels need more shared memory the more tokens and pairs there are."""
    E, H, I = 4, 128, 64
    gen = torch.Generator(device="cuda").manual_seed(T)
    w = m.quantize_experts(*(torch.randn(E, *s, device="cuda", generator=gen).bfloat16() for s in ((2 * I, H), (H, I))))
    x = torch.randn(T, H, device="cuda", generator=gen).bfloat16()
    ids = torch.randint(0, E, (T, K), dtype=torch.int32, device="cuda", generator=gen)
    g = torch.rand(T, K, device="cuda", generator=gen)
    ws = m.new_layer_workspace(T, K, H, I, E)
    out = torch.empty_like(x)

    def job(stream):
        m.moe_layer_few_tokens(x, ids, g, w.w13, w.w2, out, ws, status, w.w13_scales, w.w2_scales, w.alpha13, w.alpha2,
                               stream=stream)
    return job, out


def _product_job(m, E, status):
    """moe_expert_gemm, whose shared memory grows with the number of experts."""
    gen = torch.Generator(device="cuda").manual_seed(E)
    g = torch.full((E,), 500.0, device="cuda")
    w = m.quantize_nvfp4(torch.randn(E, 64, 64, device="cuda", generator=gen).bfloat16(), g)
    a = m.quantize_nvfp4(torch.randn(E * 2, 64, device="cuda", generator=gen).bfloat16(), g[:1], scale_layout="row")
    count = torch.full((E,), 2, dtype=torch.int32, device="cuda")
    out = torch.empty((E * 2, 64), dtype=torch.bfloat16, device="cuda")

    def job(stream):
        m.moe_expert_gemm("masked", a.codes, a.scales, count, w.codes, w.scales, out, status, max_tokens_per_expert=2,
                          scale_layout="row", stream=stream)
    return job, out


def _route_job(m, E, status):
    """moe_route_meta, whose histogram in shared memory grows with the number of experts."""
    T, K = 700, 4
    gen = torch.Generator(device="cuda").manual_seed(E)
    ids = torch.randint(0, E, (T, K), dtype=torch.int32, device="cuda", generator=gen)
    seg = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    dst, order = (torch.zeros(T * K, dtype=torch.int32, device="cuda") for _ in range(2))
    count = torch.zeros(E, dtype=torch.int32, device="cuda")
    ws = m.new_workspace(T, K, E)

    def job(stream):
        m.moe_route_meta_ex(ids, E, seg, dst, order, count, status, ws, stream=stream)
    return job, seg


def _dispatch_job(m, H, status):
    """moe_dispatch of whole rows, whose ring in shared memory goes by the hidden size."""
    T, K, E = 1024, 2, 8
    gen = torch.Generator(device="cuda").manual_seed(H)
    x = torch.randn(T, H, device="cuda", generator=gen).bfloat16()
    ids = torch.randint(0, E, (T, K), dtype=torch.int32, device="cuda", generator=gen)
    seg = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    dst, order = (torch.zeros(T * K, dtype=torch.int32, device="cuda") for _ in range(2))
    count = torch.zeros(E, dtype=torch.int32, device="cuda")
    m.moe_route_meta_ex(ids, E, seg, dst, order, count, status, m.new_workspace(T, K, E))
    out = torch.zeros((T * K, H), dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()

    def job(stream):
        m.moe_dispatch_ex("normal", "none", "row", x, ids, E, dst, seg, out, None, status, out_rows=T * K, stream=stream)
    return job, out


JOBS = {
    "layer": lambda m, s: [_layer_job(m, T, K, s) for T, K in ((1, 1), (64, 16), (20, 4))],
    "product": lambda m, s: [_product_job(m, E, s) for E in (4, 1024, 300)],
    "route": lambda m, s: [_route_job(m, E, s) for E in (500, 1024, 800)],
    "dispatch": lambda m, s: [_dispatch_job(m, H, s) for H in (1024, 7168, 2048)],
}


@pytest.mark.parametrize("kind", list(JOBS))
def test_calls_of_different_sizes_from_several_threads(kind):
    """Each call leaves what it leaves alone."""
    m = moe()
    status = m.new_status()
    jobs = JOBS[kind](m, status)
    torch.cuda.synchronize()
    want = []
    for job, out in jobs:
        job(None)
        torch.cuda.synchronize()
        want.append(out.clone())
    raised = _together([job for job, _ in jobs])
    assert not raised, raised
    m.check_status(status)
    for (_, out), w in zip(jobs, want):
        assert torch.equal(out.view(torch.uint8), w.view(torch.uint8))


def test_no_call_lowers_another_threads_shared_memory(tmp_path):
    """The limit of a kernel's shared memory is the kernel's, not the launch's. Threads without an interpreter between their
    calls meet inside the entry points often enough: where each call set the limit to its own size, one to three launches
    in a hundred were refused."""
    from combine_moe_route_meta_gb300 import build
    here = os.path.dirname(os.path.abspath(__file__))
    exe, lib = str(tmp_path / "native_threads"), build.LIB_PATH
    subprocess.run([build.nvcc(), *build.ARCH, "-std=c++17", f"-I{build.INCLUDE}", os.path.join(here, "native_threads.cpp"),
                    lib, "-Xlinker", "-rpath", "-Xlinker", os.path.dirname(lib), "-o", exe], check=True, timeout=300)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
    assert r.stdout.split() == ["product", "0", "layer", "0", "route", "0"], r.stdout


@pytest.mark.parametrize("kind", list(JOBS))
def test_the_first_cuda_call_of_a_thread(kind):
    """A call may be what makes the device's context current in its thread."""
    m = moe()
    status = m.new_status()
    job, out = JOBS[kind](m, status)[0]
    job(None)
    torch.cuda.synchronize()
    want = out.clone()
    out.zero_()
    torch.cuda.synchronize()
    raised = []

    def work():
        try:
            job(0)                            # the legacy default stream
        except Exception as e:  # noqa: BLE001
            raised.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not raised, raised
    m.check_status(status)
    assert torch.equal(out.view(torch.uint8), want.view(torch.uint8))
