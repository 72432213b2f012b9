"""The gated block example's training step against automatic differentiation of
the same block in 64 bits, and its update against the AdamW oracle.

The step rounds where the library does: binary16 weights and A operands, TF32
in the weights' gradients, bfloat16 heads and their gradients (unit 2^-8).
Each rounding is independent over the entries, so a gradient is off by a few
units of its own norm; 2^-5 of the norm leaves room for those that meet on the
way (attention's are the largest: heads, probabilities, their gradient and the
output, 2^-8 each).
"""

import importlib.util
import os

import numpy as np
import pytest

from oracle import train_oracle as to
from tests.gpu_util import require_gpu
from transformer_linear_layer_tcgen05_gb300 import lin

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "gated_block_step.py")


@pytest.fixture(scope="module")
def example():
    require_gpu()
    spec = importlib.util.spec_from_file_location("gated_block_step", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _reference(example, block, x, first, end, positions, ids, teacher, tau):
    import torch
    w = {k: (block.w16[k] if k in block.w16 else v).double().requires_grad_()
         for k, v in block.weights.items()}
    x = x.double().requires_grad_()
    t, h, hk, d = x.shape[0], block.heads, block.heads_kv, block.dim
    norm = lambda y, u: y / (y.square().mean(-1, keepdim=True) + 1e-6).sqrt() * u  # noqa: E731
    rs, bs = example.SCALES["residual_scale"], example.SCALES["block_scale"]
    qkv = (norm(x, w["norm_in"]) @ w["qkv"]).view(t, h + 2 * hk, d)
    place = positions.long()[block.axis.long()].t()           # [tokens, pairs]
    pair = torch.arange(d // 2, device="cuda")
    c, s = (y.double()[place, pair][:, None] for y in (block.cos, block.sin))

    def head(part, weight):
        n = norm(part, weight)
        a, b = n[..., :d // 2], n[..., d // 2:]
        return torch.cat([a * c - b * s, a * s + b * c], -1)

    q, k, v = head(qkv[:, :h], w["wq"]), head(qkv[:, h:h + hk], w["wk"]), qkv[:, h + hk:]
    k, v = (y.repeat_interleave(h // hk, dim=1) for y in (k, v))
    i = torch.arange(t, device="cuda")
    keep = (i[None] <= i[:, None]) & (i[None] >= first[:, None]) & (i[None] < end[:, None])
    scores = block.cap * torch.tanh(torch.einsum("ihd,jhd->hij", q, k) * d ** -0.5 / block.cap)
    p = scores.masked_fill(~keep, float("-inf")).softmax(-1)
    o = torch.einsum("hij,jhd->ihd", p, v).reshape(t, h * d)
    h1 = rs * x + bs * w["gate_o"] * norm(o @ w["o"], w["norm_o"])
    n1 = norm(h1, w["norm_mid"])
    gate = n1 @ w["gate"]
    y2 = (gate * gate.sigmoid() * (n1 @ w["up"])) @ w["down"]
    h2 = rs * h1 + bs * w["gate_down"] * norm(y2, w["norm_down"])
    log_q = (norm(h2, w["norm_out"]) @ w["lm_head"] / tau).log_softmax(-1).gather(1, ids.long())
    log_p = (teacher.double() / tau).log_softmax(-1)
    loss = tau ** 2 * (log_p.exp() * (log_p - log_q)).sum(-1).mean()
    loss.backward()
    return loss.item(), {**{k: v.grad for k, v in w.items()}, "x": x.grad}


def test_gradients_of_a_step(example):
    import torch
    block = example.Block(d_model=128, heads=4, heads_kv=2, dim=64, d_ff=256, vocab=1024, cap=4.0, seed=3)
    data = example.batch(block, 200, entries=8, seed=4)
    loss, grads = example.step(block, *data)
    torch.cuda.synchronize()
    assert lin.lin_get_device_status() == lin.LIN_SUCCESS
    want, ref = _reference(example, block, *data, 2.0)
    assert abs(loss.item() - want) <= 2.0 ** -9 * abs(want)
    assert set(ref) == set(grads)
    for name, g in ref.items():
        err = (grads[name].double() - g).norm() / g.norm()
        assert err <= 2.0 ** -5, (name, float(err))


def test_steps_with_updates(example):
    import torch
    block = example.Block(d_model=192, heads=3, heads_kv=1, dim=64, d_ff=520, vocab=1000, seed=5)
    data = example.batch(block, 333, entries=8, seed=6)
    host = lambda t: t.detach().double().cpu().numpy()  # noqa: E731
    for i in range(3):
        _, grads = example.step(block, *data)
        before = {k: host(v) for k, v in block.weights.items()}
        block.update(grads)
        torch.cuda.synchronize()
        assert lin.lin_get_device_status() == lin.LIN_SUCCESS
        for k, w in block.weights.items():
            got = host(w)
            assert np.isfinite(got).all()
            if k in block.w16:
                assert torch.equal(block.w16[k], w.half())
            if i == 0:   # from zero states: nothing of 8 bits has entered yet
                g = host(grads[k])
                decay = 0.1 if k in block.w16 else 0.0
                want, _, _ = to.adamw(before[k], g, 0 * g, 0 * g, 1, 1e-3, 0.9, 0.999, 1e-8, decay)
                # (the weight, its decay and its change, each rounded a few times)
                assert np.all(np.abs(got - want) <= 2.0 ** -20 * (np.abs(before[k]) + 1e-3))
