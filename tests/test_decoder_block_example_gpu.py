"""The example's training step against automatic differentiation of the same
block in 64 bits.

The step rounds where the library does: binary16 weights and A operands, TF32
in the weights' gradients, bfloat16 heads and their gradients (unit 2^-8).
Each rounding is independent over the entries, so a gradient is off by a few
units of its own norm; 2^-5 of the norm leaves room for those that meet on the
way (attention's are the largest: heads, probabilities, their gradient and the
output, 2^-8 each).
"""

import importlib.util
import os

import pytest

from tests.gpu_util import require_gpu
from transformer_linear_layer_tcgen05_gb300 import lin

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "decoder_block_step.py")


@pytest.fixture(scope="module")
def example():
    require_gpu()
    spec = importlib.util.spec_from_file_location("decoder_block_step", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _reference(block, x, cu, positions, ids, teacher, tau):
    import torch
    w = {k: (block.w16[k] if k in block.w16 else v).double().requires_grad_()
         for k, v in block.weights.items()}
    x = x.double().requires_grad_()
    t, h, hk, d = x.shape[0], block.heads, block.heads_kv, block.dim
    qkv = (x @ w["qkv"]).view(t, h + 2 * hk, d)
    c, s = (y.double()[positions.long()][:, None] for y in (block.cos, block.sin))

    def head(part, weight):
        n = part / (part.square().mean(-1, keepdim=True) + 1e-6).sqrt() * weight
        a, b = n[..., :d // 2], n[..., d // 2:]
        return torch.cat([a * c - b * s, a * s + b * c], -1)

    q, k, v = head(qkv[:, :h], w["wq"]), head(qkv[:, h:h + hk], w["wk"]), qkv[:, h + hk:]
    k, v = (y.repeat_interleave(h // hk, dim=1) for y in (k, v))
    i = torch.arange(t, device="cuda")
    doc = torch.searchsorted(cu[1:].long(), i, right=True)
    keep = (i[None] <= i[:, None]) & (doc[None] == doc[:, None])
    scores = torch.einsum("ihd,jhd->hij", q, k) * d ** -0.5
    p = scores.masked_fill(~keep, float("-inf")).softmax(-1)
    o = torch.einsum("hij,jhd->ihd", p, v).reshape(t, h * d)
    mid = o @ w["o"] + x
    gate = mid @ w["gate"]
    y = (gate * gate.sigmoid() * (mid @ w["up"])) @ w["down"] + mid
    log_q = (y @ w["lm_head"] / tau).log_softmax(-1).gather(1, ids.long())
    log_p = (teacher.double() / tau).log_softmax(-1)
    loss = tau ** 2 * (log_p.exp() * (log_p - log_q)).sum(-1).mean()
    loss.backward()
    return loss.item(), {**{k: v.grad for k, v in w.items()}, "x": x.grad}


def test_gradients_of_a_step(example):
    import torch
    block = example.Block(d_model=128, heads=4, heads_kv=2, dim=64, d_ff=256, vocab=1024, seed=3)
    data = example.batch(block, 200, entries=8, seed=4)
    loss, grads = example.step(block, *data)
    torch.cuda.synchronize()
    assert lin.lin_get_device_status() == lin.LIN_SUCCESS
    x, cu, _, positions, ids, teacher = data
    want, ref = _reference(block, x, cu, positions, ids, teacher, 2.0)
    assert abs(loss.item() - want) <= 2.0 ** -9 * abs(want)
    assert set(ref) == set(grads)
    for name, g in ref.items():
        err = (grads[name].double() - g).norm() / g.norm()
        assert err <= 2.0 ** -5, (name, float(err))


def test_the_loss_falls(example):
    block = example.Block(seed=5)
    data = example.batch(block, 512, seed=6)
    losses = []
    for _ in range(4):
        loss, grads = example.step(block, *data)
        for name, weight in block.weights.items():
            weight -= 0.5 * grads[name]
        block.cast()
        losses.append(loss.item())
    assert losses[-1] < losses[0] and all(a == a for a in losses)
