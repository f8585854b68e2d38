"""GPU tests of the 8-bit operators called as a serving program may call them: the process's first call inside a
capture, several host threads, steps that run the operators together, status words that are set."""
import os
import subprocess
import sys
import threading

import pytest
import torch

from test_gpu_fp8 import E4M3, check_product, random_matrix
from test_gpu_moe import Case, check

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def B():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from lut_dequant_gemv_b200 import binding, build

    build.build()
    binding.lib()
    return binding


FIRST = r"""
import sys
import torch
sys.path[:0] = [{root!r}, {root!r} + "/tests"]
from lut_dequant_gemv_b200 import binding as B
from test_gpu_fp8 import E4M3, check_product, random_matrix
from test_gpu_moe import Case
what = {what!r}
gen = torch.Generator().manual_seed(1)
graph = torch.cuda.CUDAGraph()
if what == "moe":
    case = Case(8, 256, 128, torch.float16)
    moe, x = case.handle(B, 2), case.x(3)
    ws, y = B.sqz_moe_workspace(moe, 3), torch.empty_like(x)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        B.sqz_moe_forward(moe, x, y, workspace=ws)
    graph.replay()
    first = y.clone()
    B.sqz_moe_forward(moe, x, y, workspace=ws)
    assert torch.equal(first, y) and bool(y.isfinite().all()) and B.sqz_moe_status(ws) == 0
else:
    m = 700 if what == "many" else 5
    x = torch.randn((m, 1000), generator=gen).half().cuda()
    w, sw = random_matrix(gen, 1000, 1000, E4M3, 128)
    q, s = torch.empty((m, 1008), dtype=E4M3, device="cuda")[:, :1000], torch.empty((m, 8), device="cuda")
    y = torch.empty((m, 1000), device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        B.sqz_fp8_quantize(x, q=q, scale=s)
        B.sqz_fp8_gemm(q, s, w, sw, y)
    graph.replay()
    torch.cuda.synchronize()
    check_product(y, q, s, w, sw)
    assert B.sqz_fp8_status() == 0
print("ok")
"""


@pytest.mark.parametrize("what", ["few", "many", "moe"])
def test_the_first_call_of_a_process_inside_a_capture(B, what):
    done = subprocess.run([sys.executable, "-c", FIRST.format(root=ROOT, what=what)], capture_output=True, text=True,
                          timeout=300, cwd=ROOT)
    assert done.returncode == 0 and done.stdout.strip().endswith("ok"), done.stderr[-2000:]


def test_threads_with_streams_of_their_own(B):
    """Four host threads, each quantizing, multiplying and running a layer on its own stream and workspace."""
    gen = torch.Generator().manual_seed(2)
    case = Case(8, 256, 128, torch.float16, seed=1)
    moe = case.handle(B, 2)
    jobs = []
    for m in (1, 7, 30, 300):
        x = torch.randn((m, 256), generator=gen).half().cuda()
        w, sw = random_matrix(gen, 700, 256, E4M3, 128)
        q, s = B.sqz_fp8_quantize(x)
        y = torch.empty((m, 700), device="cuda")
        B.sqz_fp8_gemm(q, s, w, sw, y)
        xm = case.x(min(m, 32))
        jobs.append(dict(x=x, w=w, sw=sw, want=(q.clone(), s.clone(), y, check(B, case, xm, 2, moe=moe)), xm=xm,
                         ws=B.sqz_moe_workspace(moe, 32)))
    torch.cuda.synchronize()
    failures = []

    def work(job):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(20):
                    q, s = B.sqz_fp8_quantize(job["x"])
                    y, ym = torch.empty_like(job["want"][2]), torch.empty_like(job["xm"])
                    B.sqz_fp8_gemm(q, s, job["w"], job["sw"], y)
                    B.sqz_moe_forward(moe, job["xm"], ym, workspace=job["ws"])
                stream.synchronize()
                got = (q, s, y, ym)
            for a, b in zip(job["want"], got):
                if not torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)):
                    failures.append(tuple(a.shape))
        except Exception as e:  # noqa: BLE001
            failures.append(repr(e))

    threads = [threading.Thread(target=work, args=(job,)) for job in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures
    assert B.sqz_fp8_status() == 0 and all(B.sqz_moe_status(job["ws"]) == 0 for job in jobs)


def test_a_workspace_status_that_is_set_is_reported_until_zeroed(B):
    """Bit 0 of the status word (behind the 8-byte count the workspace starts with), as a kernel whose wait gave up
    sets it."""
    case = Case(4, 128, 64, torch.float16, seed=2)
    moe = case.handle(B, 2)
    ws = B.sqz_moe_workspace(moe, 2)
    assert B.sqz_moe_status(ws) == 0
    ws[8] = 1
    for _ in range(2):
        with pytest.raises(B.SqzError) as e:
            B.sqz_moe_status(ws)
        assert e.value.status == B.SQZ_ERR_TIMEOUT and "zero the workspace" in str(e.value)
    ws.zero_()
    check(B, case, case.x(2), 2, moe=moe, ws=ws)


@pytest.mark.parametrize("tokens", [1, 40, 300])
def test_a_decoding_step(B, tokens):
    """Quantize, project, mix (in batches the layer takes), quantize and project back, captured and replayed: the
    same bits as call by call, each product within its bound."""
    gen = torch.Generator().manual_seed(3)
    case = Case(8, 512, 256, torch.bfloat16, seed=3)
    moe = case.handle(B, 2)
    ws = B.sqz_moe_workspace(moe, 32)
    w1, s1 = random_matrix(gen, 512, 1040, E4M3, 128)
    w2, s2 = random_matrix(gen, 1040, 512, E4M3, 128)
    s1 *= 1040 ** -0.5
    s2 *= 512 ** -0.5
    x = torch.randn((tokens, 1040), generator=gen).bfloat16().cuda()
    h, y = torch.empty((tokens, 512), dtype=torch.bfloat16, device="cuda"), torch.empty_like(x)
    mixed = torch.empty_like(h)
    q1, a1 = torch.empty((tokens, 1040), dtype=E4M3, device="cuda"), torch.empty((tokens, 9), device="cuda")
    q2, a2 = torch.empty((tokens, 512), dtype=E4M3, device="cuda"), torch.empty((tokens, 4), device="cuda")

    def step():
        B.sqz_fp8_quantize(x, q=q1, scale=a1)
        B.sqz_fp8_gemm(q1, a1, w1, s1, h)
        for t in range(0, tokens, 32):
            B.sqz_moe_forward(moe, h[t:t + 32], mixed[t:t + 32], workspace=ws)
        B.sqz_fp8_quantize(mixed, q=q2, scale=a2)
        B.sqz_fp8_gemm(q2, a2, w2, s2, y)

    step()
    check_product(h, q1, a1, w1, s1)
    check_product(y, q2, a2, w2, s2)
    for t in range(0, tokens, 32):
        assert torch.equal(mixed[t:t + 32], check(B, case, h[t:t + 32], 2, moe=moe, ws=ws))
    want = [v.clone() for v in (h, mixed, y)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for v in (h, mixed, y):
        v.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (h, mixed, y)))


@pytest.mark.parametrize("raw", [False, True])
def test_outputs_made_for_another_stream(B, raw):
    """q and scales that the call allocates belong to the stream it is given: memory that was freed on the current
    stream may still be written there."""
    x = torch.randn((300, 1024), generator=torch.Generator().manual_seed(4)).half().cuda()
    want_q, want_s = B.sqz_fp8_quantize(x)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.empty_cache()
        busy = [torch.empty(300 * 1024, dtype=torch.uint8, device="cuda"), torch.empty(300 * 8, device="cuda")]
        torch.cuda._sleep(20_000_000)  # about 10 ms, then the current stream writes what it has freed
        for t in busy:
            t.fill_(7)
        del t, busy
        q, s = B.sqz_fp8_quantize(x, stream=side.cuda_stream if raw else side)
        torch.cuda.synchronize()
        assert torch.equal(q.view(torch.uint8), want_q.view(torch.uint8)) and torch.equal(s, want_s)
        del q, s
