"""Calls from several host threads: a thread's first call, and one kernel with
calls of different sizes at once, whose launches want different shared memory."""

import threading

import pytest

from tests.gpu_util import require_gpu
from transformer_linear_layer_tcgen05_gb300 import lin

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _calls():
    """A small call of each kind: (the call with a stream, its results)."""
    import torch
    rnd = lambda *s: torch.randn(*s, device="cuda")  # noqa: E731
    x, w, y = rnd(64, 128), rnd(128, 64), rnd(64, 64)
    q, k, v = (rnd(40, 2, 64).half() for _ in range(3))
    o, lse = torch.empty_like(q), torch.empty(2, 40, device="cuda")
    h, n, ones = torch.empty_like(x), torch.empty_like(x), torch.ones(128, device="cuda")
    p, zero = rnd(500), torch.zeros(3, 500, device="cuda")
    z, dz, loss = rnd(8, 400), rnd(8, 400), torch.empty(9, device="cuda")
    ids = torch.arange(8, dtype=torch.int32, device="cuda").repeat(8, 1)
    teacher = rnd(8, 8)
    xh, wh, yh = x.cpu(), w.cpu(), torch.empty(64, 64)
    return {
        "matmul_host": lambda s: lin.lin_matmul_host(xh, wh, yh, stream=s),
        "status": lambda s: lin.check("status", lin.lin_get_device_status()),
        "matmul": lambda s: lin.lin_matmul(x, w, y, stream=s),
        "attention": lambda s: lin.lin_attention(q, k, v, o, lse, stream=s),
        "block_norms": lambda s: lin.lin_block_norms(x, None, None, None, ones, h, n, stream=s),
        "adamw": lambda s: lin.lin_adamw([p], [zero[0]], [zero[1]], [zero[2]], stream=s),
        "distill_topk": lambda s: lin.lin_distill_topk(z, ids, teacher, dz, loss[:8], loss[8:], stream=s),
    }


@pytest.mark.parametrize("name", ["matmul_host", "status", "matmul", "attention", "block_norms", "adamw", "distill_topk"])
def test_a_threads_first_call(name):
    # (a thread that has made no CUDA call of its own yet)
    import torch
    call, errors = _calls()[name], []
    stream = torch.cuda.Stream().cuda_stream
    torch.cuda.synchronize()
    call(stream)

    def first():
        try:
            call(stream)
        except Exception as e:   # (told by the thread that joins)
            errors.append(e)

    t = threading.Thread(target=first)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not errors
    assert lin.lin_get_device_status() == lin.LIN_SUCCESS


def _at_once(calls, times=1500):
    """Each call `times` times in a host thread of its own; their errors."""
    import torch
    errors, start = [], threading.Barrier(len(calls))

    def loop(call):
        stream = torch.cuda.Stream()
        start.wait()
        try:
            for _ in range(times):
                call(stream)
        except Exception as e:   # (told by the thread that joins)
            errors.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=loop, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert lin.lin_get_device_status() == lin.LIN_SUCCESS
    return errors


@pytest.mark.parametrize("gradient", [False, True])
def test_block_norms(gradient):
    # (width 2048, bfloat16: 48 and 96 KB forward, 120 and 216 KB of the gradient)
    import torch
    width = 2048
    weights = torch.ones(width, device="cuda"), torch.ones(width, device="cuda")
    calls, results = [], []
    for tokens in (600, 1024) if gradient else (1024, 2048):
        x = torch.randn(tokens, width, device="cuda")
        y = x.flip(0).bfloat16()
        h, n = torch.empty_like(x), torch.empty_like(y)
        out = [torch.empty_like(t) for t in (x, y, weights[0], weights[1])]

        def call(stream, x=x, y=y, h=h, n=n, out=out):
            if gradient:
                lin.lin_block_norms_backward(x, y, None, *weights, h, n, out[0], out[1], None,
                                             out[2], out[3], stream=stream)
            else:
                lin.lin_block_norms(x, y, None, *weights, h, n, stream=stream)

        h.copy_(x.flip(1)), n.copy_(y.flip(1))
        calls.append(call)
        results.append(out if gradient else [h, n])
    torch.cuda.synchronize()
    for c in calls:
        c(None)
    torch.cuda.synchronize()
    want = [[t.clone() for t in r] for r in results]
    assert not _at_once(calls)
    for r, w in zip(results, want):
        assert all(torch.equal(a, b) for a, b in zip(r, w))


def test_distillation():
    # (rows of eight warps: 40 and 64 KB to a slot)
    import torch
    calls, results = [], []
    for v in (10000, 16384):
        m, k = 300, 12
        z = torch.randn(m, v, device="cuda")
        ids = torch.arange(k, dtype=torch.int32, device="cuda").repeat(m, 1) * 700
        teacher = torch.randn(m, k, device="cuda")
        out = [torch.empty_like(z), torch.empty(m, device="cuda"), torch.empty(1, device="cuda")]

        def call(stream, z=z, ids=ids, teacher=teacher, out=out):
            lin.lin_distill_topk(z, ids, teacher, *out, stream=stream)

        call(None)
        calls.append(call)
        results.append(out)
    torch.cuda.synchronize()
    want = [[t.clone() for t in r] for r in results]
    assert not _at_once(calls)
    for r, w in zip(results, want):
        assert all(torch.equal(a, b) for a, b in zip(r, w))
