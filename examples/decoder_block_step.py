"""Training steps of one decoder block distilled from a teacher's top logits.

Runs the library's operators together as a training program would: the QKV
projection, per-head norms and rotation, attention over packed documents, the
output projection with its residual, the SwiGLU FFN, the lm_head, the
distillation loss, and the whole way back to every weight, followed by a plain
SGD update of float32 masters with binary16 copies. torch only holds the
tensors, casts between the float32 activations and attention's bfloat16, and
applies the update.

    python examples/decoder_block_step.py [--steps 5] [--tokens 512]

Synthetic data: random documents, and a random teacher that the block learns
to follow, so the loss falls.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from transformer_linear_layer_tcgen05_gb300 import lin  # noqa: E402


class Block:
    """Sizes, float32 master weights and their binary16 copies."""

    def __init__(self, d_model=768, heads=12, heads_kv=4, dim=64, d_ff=3072, vocab=16384,
                 max_tokens=4096, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.heads, self.heads_kv, self.dim, self.d_model = heads, heads_kv, dim, d_model
        w = lambda k, n: torch.randn(k, n, generator=g, device="cuda") * k ** -0.5  # noqa: E731
        self.weights = {"qkv": w(d_model, (heads + 2 * heads_kv) * dim), "o": w(heads * dim, d_model),
                        "gate": w(d_model, d_ff), "up": w(d_model, d_ff), "down": w(d_ff, d_model),
                        "lm_head": w(d_model, vocab), "wq": torch.ones(dim, device="cuda"),
                        "wk": torch.ones(dim, device="cuda")}
        angle = torch.arange(max_tokens, device="cuda")[:, None] * 10000.0 ** (
            -torch.arange(dim // 2, device="cuda") * 2 / dim)
        self.cos, self.sin = angle.cos().contiguous(), angle.sin().contiguous()
        self.cast()

    def cast(self):
        self.w16 = {k: v.half() for k, v in self.weights.items() if v.dim() == 2}


def step(block, x, cu, longest, positions, ids, teacher, temperature=2.0):
    """One forward and backward pass over x [tokens, d_model] (packed documents
    with offsets `cu`): the mean loss and the gradients of x and every weight."""
    b, w = block, block.w16
    t, h, hk, d = x.shape[0], b.heads, b.heads_kv, b.dim
    new = lambda *s: torch.empty(s, device="cuda")  # noqa: E731
    new16 = lambda *s: torch.empty(s, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    wq, wk = b.weights["wq"], b.weights["wk"]
    docs = dict(cu_q=cu, cu_k=cu, max_q=longest, max_k=longest, causal=True)

    # forward
    qkv = lin.lin_matmul_w16(x, w["qkv"], new(t, (h + 2 * hk) * d))
    heads = new16(t, h + 2 * hk, d)   # q, k and v of a token in one row
    q, k, v = heads[:, :h], heads[:, h:h + hk], heads[:, h + hk:]
    lin.lin_qk_norm_rope(qkv, wq, wk, b.cos, b.sin, positions, q, k, v)
    o, lse = lin.lin_attention(q, k, v, new16(t, h, d), new(h, t), **docs)
    o32 = o.view(t, h * d).float()
    mid = lin.lin_matmul_residual_w16(o32, w["o"], x, new(t, b.d_model))
    gate, up = lin.lin_gate_up_w16(mid, w["gate"], w["up"], new(t, w["gate"].shape[1]),
                                   new(t, w["up"].shape[1]))
    y = lin.lin_matmul_residual_swiglu_a_w16(gate, up, w["down"], mid, new(t, b.d_model))
    logits = lin.lin_matmul_w16(y, w["lm_head"], new(t, w["lm_head"].shape[1]))
    dlogits, losses, loss = lin.lin_distill_topk(logits, ids, teacher, logits, new(t), new(1),
                                                 temperature, 1.0 / t)

    # backward
    g = {}
    dy = lin.lin_matmul_t_w16(dlogits, w["lm_head"], new(t, b.d_model))
    g["lm_head"] = lin.lin_matmul_at(y, dlogits, torch.empty_like(b.weights["lm_head"]))
    dgate, dup = lin.lin_matmul_t_swiglu_backward_w16(dy, w["down"], gate, up,
                                                      torch.empty_like(gate), torch.empty_like(up))
    g["down"] = lin.lin_matmul_at_swiglu_a(gate, up, dy, torch.empty_like(b.weights["down"]))
    g["gate"] = lin.lin_matmul_at(mid, dgate, torch.empty_like(b.weights["gate"]))
    g["up"] = lin.lin_matmul_at(mid, dup, torch.empty_like(b.weights["up"]))
    dmid = dy   # the residual's share; the two branches are added to it
    lin.lin_matmul_t_acc_w16(dgate, w["gate"], dmid)
    lin.lin_matmul_t_acc_w16(dup, w["up"], dmid)
    do = lin.lin_matmul_t_w16(dmid, w["o"], new(t, h * d))
    g["o"] = lin.lin_matmul_at(o32, dmid, torch.empty_like(b.weights["o"]))
    dheads = new16(t, h + 2 * hk, d)
    dq, dk, dv = dheads[:, :h], dheads[:, h:h + hk], dheads[:, h + hk:]
    lin.lin_attention_backward(q, k, v, o, lse, do.view(t, h, d).bfloat16(), dq, dk, dv, **docs)
    dqkv, g["wq"], g["wk"] = lin.lin_qk_norm_rope_backward(
        qkv, wq, wk, b.cos, b.sin, positions, dq, dk, dv, torch.empty_like(qkv),
        torch.empty_like(wq), torch.empty_like(wk))
    g["qkv"] = lin.lin_matmul_at(x, dqkv, torch.empty_like(b.weights["qkv"]))
    lin.lin_matmul_t_acc_w16(dqkv, w["qkv"], dmid)
    g["x"] = dmid
    return loss / t, g


def batch(block, tokens, entries=32, seed=1):
    """Packed documents of uneven lengths, and a random teacher's entries."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    cuts = sorted({0, tokens, tokens // 5, tokens * 3 // 7})
    cu = torch.tensor(cuts, dtype=torch.int32, device="cuda")
    longest = max(b - a for a, b in zip(cuts[:-1], cuts[1:]))
    positions = torch.cat([torch.arange(b - a) for a, b in zip(cuts[:-1], cuts[1:])]).int().cuda()
    x = torch.randn(tokens, block.d_model, generator=g, device="cuda")
    vocab = block.weights["lm_head"].shape[1]
    ids = torch.rand(tokens, vocab, generator=g, device="cuda").topk(entries, dim=1)[1].int()
    teacher = 3 * torch.randn(tokens, entries, generator=g, device="cuda")
    return x, cu, longest, positions, ids, teacher


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=5)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--rate", type=float, default=0.5)
    args = ap.parse_args()
    block = Block()
    data = batch(block, args.tokens)
    for i in range(args.steps):
        loss, grads = step(block, *data)
        for name, weight in block.weights.items():
            weight -= args.rate * grads[name]
        block.cast()
        print(f"step {i}: loss {loss.item():.4f}")
    if lin.lin_get_device_status() != lin.LIN_SUCCESS:
        raise SystemExit("a kernel reported a failure")


if __name__ == "__main__":
    main()
