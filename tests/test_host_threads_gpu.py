"""Calls from several host threads."""

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
    return {
        "matmul": lambda s: lin.lin_matmul(x, w, y, stream=s),
        "attention": lambda s: lin.lin_attention(q, k, v, o, lse, stream=s),
        "block_norms": lambda s: lin.lin_block_norms(x, None, None, None, ones, h, n, stream=s),
        "adamw": lambda s: lin.lin_adamw([p], [zero[0]], [zero[1]], [zero[2]], stream=s),
        "distill_topk": lambda s: lin.lin_distill_topk(z, ids, teacher, dz, loss[:8], loss[8:], stream=s),
    }


@pytest.mark.parametrize("name", ["matmul", "attention", "block_norms", "adamw", "distill_topk"])
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
