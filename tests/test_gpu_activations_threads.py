"""RMS norm, 8-bit activations and the weight gradient called from several host threads at once,
each on a stream of its own: the same bits as one thread's calls."""
import threading

import pytest
import torch

from gpu_helpers import env

pytestmark = pytest.mark.gpu


def step(b2g, x, res, w, dy, dz):
    y, total, rstd, y8, t8 = b2g.rms_norm_8bit(x, w, res, with_y=True, keep_total=True)
    dx, dw = b2g.rms_norm_backward(dy, t8, w, rstd, dy)
    dx2, dw2 = b2g.rms_norm_backward(dy, total, w, rstd)
    grad = b2g.linear_weight_grad_8bit(dz, *y8)
    b2g.linear_weight_grad_8bit(dz, *t8, dw=grad, accumulate=True)
    q = b2g.quantize_8bit(x)
    return [y, total, rstd, dx, dw, dx2, dw2, grad, b2g.dequantize_8bit(*q, x.dtype),
            *(t.contiguous().view(torch.uint8) for t in (*y8, *t8, *q))]


def test_threads_on_separate_streams():
    _, b2g = env()
    jobs = []
    for k, (rows, cols, outs, dt) in enumerate([(1200, 512, 264, torch.bfloat16), (16, 4096, 300, torch.bfloat16),
                                                (700, 777, 130, torch.float32), (3000, 1024, 72, torch.float32)]):
        torch.manual_seed(k)
        x, res, dy = (torch.randn(rows, cols, device="cuda").to(dt) for _ in range(3))
        jobs.append((x, res, torch.randn(cols, device="cuda").to(dt), dy, torch.randn(rows, outs, device="cuda").to(dt)))
    want = [step(b2g, *j) for j in jobs]
    torch.cuda.synchronize()
    start, errors = threading.Barrier(len(jobs)), []

    def worker(k):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                start.wait()
                got = [step(b2g, *jobs[k]) for _ in range(10)]
            stream.synchronize()
            for i, run in enumerate(got):
                for n, (a, b) in enumerate(zip(run, want[k])):
                    if not torch.equal(a, b):
                        errors.append((k, i, n))
        except Exception as e:  # reported below, on the main thread
            errors.append((k, repr(e)))

    threads = [threading.Thread(target=worker, args=(k,)) for k in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not any(t.is_alive() for t in threads) and not errors, errors
    assert b2g.b2g_status(torch.cuda.current_stream().cuda_stream) == (0, 0)
