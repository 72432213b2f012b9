"""lin_attention and lin_attention_backward at the edges of their rules. Bounds
as in test_attention_gpu.py unless a test says otherwise.
"""

import pytest

from tests.gpu_util import require_gpu
from tests.test_attention_gpu import _cu, _setup
from transformer_linear_layer_tcgen05_gb300 import lin

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def test_gradient_without_keys_where_parts_are_asked_for():
    # every sequence is empty of keys, while max_k asks for parts of them: dQ
    # is the sum of parts of zeros, and must not be taken before they are
    # written (a few times: the order was a matter of time)
    import torch
    t = _setup("float16", [(70, 2000)], 1, 1, 64, seed=80)
    none = torch.zeros(2, dtype=torch.int32, device="cuda")
    how = dict(cu_q=_cu([70]), cu_k=none, max_q=70, max_k=2000, causal=False)
    lin.lin_attention(t["q"], t["k"], t["v"], t["o"], t["lse"], **how)
    assert torch.all(t["o"] == 0) and torch.all(t["lse"] == -float("inf"))
    for _ in range(20):
        t["dq"].fill_(float("nan"))
        lin.lin_attention_backward(t["q"], t["k"], t["v"], t["o"], t["lse"], t["do"], t["dq"],
                                   t["dk"], t["dv"], **how)
        kernels, _ = lin.lin_last_launch_info()
        assert kernels == 3
        assert torch.all(t["dq"] == 0)
    assert t["dk"].isnan().all() and t["dv"].isnan().all()   # (rows of no sequence)
    assert lin.lin_get_device_status() == lin.LIN_SUCCESS
