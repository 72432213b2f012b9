"""Training steps of one decoder block over packed images and text, with norms
before and after its layers, gates on what they add to the residual stream,
capped attention within documents and rotation by three position axes, trained
by AdamW with 8-bit states.

Runs the library's operators together as a training program would: the norm
that the block begins with, the QKV projection, per-head norms and rotation by
the patches' time, height and width, attention whose scores are capped and kept
to the query's own document, the output projection, the norms and the gated sum
between the two layers, the SwiGLU FFN, the norms behind it, the lm_head and the
distillation loss; the whole way back to every weight; and the optimizer's step,
which also writes the binary16 copies that the linear layers read. torch only
holds the tensors and casts between the float32 activations and attention's
bfloat16.

    python examples/gated_block_step.py [--steps 5] [--tokens 512]

Synthetic data: random documents of patches, and a random teacher.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from transformer_linear_layer_tcgen05_gb300 import lin  # noqa: E402

SCALES = dict(residual_scale=1.0, block_scale=0.5)


class Block:
    """Sizes, float32 master weights, their binary16 copies and AdamW's states
    (8 bits for the matrices, float32 for the vectors, which have no decay)."""

    def __init__(self, d_model=768, heads=12, heads_kv=4, dim=64, d_ff=2048, vocab=16384, cap=30.0,
                 table=1024, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.heads, self.heads_kv, self.dim, self.d_model, self.cap = heads, heads_kv, dim, d_model, cap
        w = lambda k, n: torch.randn(k, n, generator=g, device="cuda") * k ** -0.5  # noqa: E731
        ones = lambda n, v=1.0: torch.full((n,), v, device="cuda")  # noqa: E731
        self.weights = {
            "qkv": w(d_model, (heads + 2 * heads_kv) * dim), "o": w(heads * dim, d_model),
            "gate": w(d_model, d_ff), "up": w(d_model, d_ff), "down": w(d_ff, d_model),
            "lm_head": w(d_model, vocab), "wq": ones(dim), "wk": ones(dim), "norm_in": ones(d_model),
            "norm_o": ones(d_model), "gate_o": ones(d_model, 0.7), "norm_mid": ones(d_model),
            "norm_down": ones(d_model), "gate_down": ones(d_model, 0.6), "norm_out": ones(d_model)}
        pairs = dim // 2
        angle = torch.arange(table, device="cuda")[:, None] * 10000.0 ** (
            -torch.arange(pairs, device="cuda") / pairs)
        self.cos, self.sin = angle.cos().contiguous(), angle.sin().contiguous()
        self.axis = (torch.arange(pairs, device="cuda") % 3).int()   # pairs dealt to the axes in turn
        self.matrices = [k for k, v in self.weights.items() if v.dim() == 2]
        self.vectors = [k for k, v in self.weights.items() if v.dim() == 1]
        self.w16 = {k: self.weights[k].half() for k in self.matrices}
        codes = lambda t: torch.zeros(t.shape, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)  # noqa: E731,E501
        scales = lambda t: torch.zeros(-(-t.numel() // 256), device="cuda")  # noqa: E731
        self.m = {k: codes(v) if v.dim() == 2 else torch.zeros_like(v) for k, v in self.weights.items()}
        self.v = {k: codes(v) if v.dim() == 2 else torch.zeros_like(v) for k, v in self.weights.items()}
        self.m_scale = {k: scales(self.weights[k]) for k in self.matrices}
        self.v_scale = {k: scales(self.weights[k]) for k in self.matrices}
        self.steps = 0

    def update(self, grads, lr=1e-3, weight_decay=0.1):
        """The AdamW step of every weight: matrices with decay, 8-bit states and
        binary16 copies, vectors without."""
        self.steps += 1
        pick = lambda d, names: [d[k] for k in names]  # noqa: E731
        for names, decay in ((self.matrices, weight_decay), (self.vectors, 0.0)):
            more = {}
            if names is self.matrices:
                more = dict(m_scale=pick(self.m_scale, names), v_scale=pick(self.v_scale, names),
                            w16=pick(self.w16, names))
            lin.lin_adamw(pick(self.weights, names), pick(grads, names), pick(self.m, names),
                          pick(self.v, names), step=self.steps, lr=lr, weight_decay=decay, **more)


def step(block, x, first, end, positions, ids, teacher, temperature=2.0):
    """One forward and backward pass over x [tokens, d_model] (documents given by
    each token's first key and the one behind its last): the mean loss and the
    gradients of x and every weight."""
    b, w, v = block, block.w16, block.weights
    t, h, hk, d = x.shape[0], b.heads, b.heads_kv, b.dim
    new = lambda *s: torch.empty(s, device="cuda")  # noqa: E731
    new16 = lambda *s: torch.empty(s, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    rows = lambda: new(t, b.d_model)  # noqa: E731
    tables = (b.cos, b.sin, positions, b.axis)
    form = dict(cap=b.cap, first_key=first, end_key=end, causal=True)

    # forward
    _, n0 = lin.lin_block_norms(x, None, None, None, v["norm_in"], None, rows())
    qkv = lin.lin_matmul_w16(n0, w["qkv"], new(t, (h + 2 * hk) * d))
    heads = new16(t, h + 2 * hk, d)   # q, k and v of a token in one row
    q, k, val = heads[:, :h], heads[:, h:h + hk], heads[:, h + hk:]
    lin.lin_qk_norm_rope_axes(qkv, v["wq"], v["wk"], *tables, q, k, val)
    o, lse = lin.lin_attention_scores(q, k, val, new16(t, h, d), new(h, t), **form)
    o32 = o.view(t, h * d).float()
    y1 = lin.lin_matmul_w16(o32, w["o"], rows())
    h1, n1 = lin.lin_block_norms(x, y1, v["gate_o"], v["norm_o"], v["norm_mid"], rows(), rows(), **SCALES)
    gate, up = lin.lin_gate_up_w16(n1, w["gate"], w["up"], new(t, w["gate"].shape[1]),
                                   new(t, w["up"].shape[1]))
    zero = torch.zeros(t, b.d_model, device="cuda")   # (the residual is added behind the norm)
    y2 = lin.lin_matmul_residual_swiglu_a_w16(gate, up, w["down"], zero, rows())
    h2, n2 = lin.lin_block_norms(h1, y2, v["gate_down"], v["norm_down"], v["norm_out"], rows(), rows(),
                                 **SCALES)
    logits = lin.lin_matmul_w16(n2, w["lm_head"], new(t, w["lm_head"].shape[1]))
    dlogits, losses, loss = lin.lin_distill_topk(logits, ids, teacher, logits, new(t), new(1),
                                                 temperature, 1.0 / t)

    # backward
    g = {k: torch.empty_like(y) for k, y in v.items()}
    dn = lin.lin_matmul_t_w16(dlogits, w["lm_head"], rows())
    lin.lin_matmul_at(n2, dlogits, g["lm_head"])
    dh, dy2 = rows(), rows()
    lin.lin_block_norms_backward(h2, y2, v["gate_down"], v["norm_down"], v["norm_out"], None, dn, dh, dy2,
                                 g["gate_down"], g["norm_down"], g["norm_out"], **SCALES)
    dgate, dup = lin.lin_matmul_t_swiglu_backward_w16(dy2, w["down"], gate, up, torch.empty_like(gate),
                                                      torch.empty_like(up))
    lin.lin_matmul_at_swiglu_a(gate, up, dy2, g["down"])
    lin.lin_matmul_at(n1, dgate, g["gate"])
    lin.lin_matmul_at(n1, dup, g["up"])
    lin.lin_matmul_t_w16(dgate, w["gate"], dn)
    lin.lin_matmul_t_acc_w16(dup, w["up"], dn)
    dy1 = rows()
    lin.lin_block_norms_backward(h1, y1, v["gate_o"], v["norm_o"], v["norm_mid"], dh, dn, dh, dy1,
                                 g["gate_o"], g["norm_o"], g["norm_mid"], **SCALES)
    do = lin.lin_matmul_t_w16(dy1, w["o"], new(t, h * d))
    lin.lin_matmul_at(o32, dy1, g["o"])
    dheads = new16(t, h + 2 * hk, d)
    dq, dk, dv = dheads[:, :h], dheads[:, h:h + hk], dheads[:, h + hk:]
    lin.lin_attention_scores_backward(q, k, val, o, lse, do.view(t, h, d).bfloat16(), dq, dk, dv, **form)
    dqkv = torch.empty_like(qkv)
    lin.lin_qk_norm_rope_axes_backward(qkv, v["wq"], v["wk"], *tables, dq, dk, dv, dqkv, g["wq"], g["wk"])
    lin.lin_matmul_at(n0, dqkv, g["qkv"])
    lin.lin_matmul_t_w16(dqkv, w["qkv"], dn)
    lin.lin_block_norms_backward(x, None, None, None, v["norm_in"], dh, dn, dh, None, None, None,
                                 g["norm_in"])
    g["x"] = dh
    return loss / t, g


def batch(block, tokens, entries=32, seed=1):
    """Packed documents of patches of uneven sizes, and a random teacher's
    entries."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    cuts = torch.tensor(sorted({0, tokens, tokens // 5, tokens * 3 // 7}), device="cuda")
    i = torch.arange(tokens, device="cuda")
    doc = torch.searchsorted(cuts[1:], i, right=True)
    first, end = cuts[doc].int(), cuts[doc + 1].int()
    at = i - cuts[doc]
    positions = torch.stack([at // 64, at // 8 % 8, at % 8]).int().contiguous()
    x = torch.randn(tokens, block.d_model, generator=g, device="cuda")
    vocab = block.weights["lm_head"].shape[1]
    ids = torch.rand(tokens, vocab, generator=g, device="cuda").topk(entries, dim=1)[1].int()
    teacher = 3 * torch.randn(tokens, entries, generator=g, device="cuda")
    return x, first, end, positions, ids, teacher


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=5)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--rate", type=float, default=1e-3)
    args = ap.parse_args()
    block = Block()
    data = batch(block, args.tokens)
    for i in range(args.steps):
        loss, grads = step(block, *data)
        block.update(grads, lr=args.rate)
        print(f"step {i}: loss {loss.item():.4f}")
    if lin.lin_get_device_status() != lin.LIN_SUCCESS:
        raise SystemExit("a kernel reported a failure")


if __name__ == "__main__":
    main()
