"""The training-step operators around the linear layers: attention and its
gradient, the per-head norm and rotation of queries and keys and its gradient,
and the distillation loss on a teacher's top logits with its gradient.

``run`` computes each of them in its plain form (elementary torch operations
in 32 bits, rounded once at the end), or, with ``own`` true, by the entry
points of ``transformer_linear_layer_tcgen05_gb300.lin``.
"""

import math
import random

import numpy as np
import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one 512-token training sequence of the 768-wide model (12 heads of
        # 64), the smallest attention call of a step: latency counts
        dict(name="attn_fwd_512_f16", op="attn", grad=False, dtype="f16", seqs=1, tq=512, tk=512,
             ragged=0, hq=12, hkv=12, d=64, causal=True),
        # an encoder-decoder batch: seven packed sequences of uneven lengths,
        # queries over another text's keys, heads of 96 shared four to one
        dict(name="attn_fwd_packed_cross_bf16", op="attn", grad=False, dtype="bf16", seqs=7,
             tq=1111, tk=1903, ragged=5, hq=16, hkv=4, d=96, causal=False),
        # the forward pass of a long-context training sequence
        dict(name="attn_fwd_8192_bf16", op="attn", grad=False, dtype="bf16", seqs=1, tq=8192,
             tk=8192, ragged=0, hq=32, hkv=8, d=128, causal=True),
        # the gradient of the first case: the same step's backward pass
        dict(name="attn_bwd_512_f16", op="attn", grad=True, dtype="f16", seqs=1, tq=512, tk=512,
             ragged=0, hq=12, hkv=12, d=64, causal=True),
        # packed documents of uneven lengths over uneven key lengths, causal
        # from the end: where a sequence has fewer keys than queries, its
        # first rows attend to nothing
        dict(name="attn_bwd_packed_f16", op="attn", grad=True, dtype="f16", seqs=9, tq=997,
             tk=1024, ragged=3, hq=12, hkv=6, d=64, causal=True),
        # the gradient of a long-context sequence with shared key heads
        dict(name="attn_bwd_8192_bf16", op="attn", grad=True, dtype="bf16", seqs=1, tq=8192,
             tk=8192, ragged=0, hq=16, hkv=4, d=128, causal=True),
        # queries, keys and values of the 512-token step after the QKV
        # projection
        dict(name="norm_rope_fwd_512_f16", op="rope", grad=False, dtype="f16", t=512, hq=12, hkv=12,
             d=64, rot=64, interleaved=False),
        # its gradient at an odd token count, partial rotation of adjacent
        # pairs
        dict(name="norm_rope_bwd_777_f16", op="rope", grad=True, dtype="f16", t=777, hq=12, hkv=6,
             d=96, rot=48, interleaved=True),
        # a large batch's gradient: 16k tokens of 32 query and 8 key heads
        dict(name="norm_rope_bwd_16k_bf16", op="rope", grad=True, dtype="bf16", t=16384, hq=32,
             hkv=8, d=128, rot=128, interleaved=False),
        # distillation at the lm_head shape of the 768-wide model: 512 tokens,
        # 16384 entries, the teacher's 32 best
        dict(name="distill_512x16384", op="distill", grad=True, m=512, v=16384, k=32, tau=2.0),
        # evaluation: the loss alone, an odd vocabulary
        dict(name="distill_loss_1000x50001", op="distill", grad=False, m=1000, v=50001, k=20,
             tau=1.0),
        # a large vocabulary and batch: logits of 2 GiB
        dict(name="distill_4096x131072", op="distill", grad=True, m=4096, v=131072, k=64, tau=1.5),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["attn_fwd", "attn_bwd", "rope", "distill"])
    if kind.startswith("attn"):
        grad = kind == "attn_bwd"
        hkv = rng.choice([1, 2, 3, 4, 6, 8])
        hq = hkv * rng.choice([1, 2, 3, 4])
        d = rng.choice([32, 40, 64, 64, 80, 96, 128, 128])
        cap = 8192 * 8192 * 16 * 128 * (1.0 if grad else 2.0)
        while True:
            tq = _log_uniform(rng, 16, 8192)
            tk = tq if rng.random() < 0.5 else _log_uniform(rng, 16, 8192)
            seqs = _log_uniform(rng, 1, 32)
            if seqs * tq * tk * hq * max(d, 64) <= cap and seqs * (tq + tk) >= 64:
                break
        return dict(op="attn", grad=grad, dtype=rng.choice(["f16", "bf16"]), seqs=seqs, tq=tq,
                    tk=tk, ragged=rng.choice([0, rng.randrange(1, 1000)]), hq=hq, hkv=hkv, d=d,
                    causal=rng.random() < 0.7)
    if kind == "rope":
        hkv = rng.choice([1, 2, 4, 6, 8, 12])
        hq = hkv * rng.choice([1, 2, 3, 4])
        d = rng.choice([32, 64, 80, 96, 128, 128, 256])
        rot = d if rng.random() < 0.6 else 8 * rng.randrange(1, d // 8 + 1)
        most = min(16384, 16384 * 48 * 128 // ((hq + 2 * hkv) * d))
        return dict(op="rope", grad=rng.random() < 0.6, dtype=rng.choice(["f16", "bf16"]),
                    t=_log_uniform(rng, 1, most), hq=hq, hkv=hkv, d=d, rot=rot,
                    interleaved=rng.random() < 0.4)
    v = _log_uniform(rng, 1000, 131072)
    m = _log_uniform(rng, 8, min(16384, 4096 * 131072 // v))
    return dict(op="distill", grad=rng.random() < 0.75, m=m, v=v, k=_log_uniform(rng, 1, 128),
                tau=rng.choice([1.0, 1.5, 2.0, 4.0]))


def _lengths(case):
    """The sequences' (query, key) lengths: all alike, or (ragged, a seed)
    spread between an eighth of the longest and the longest."""
    if not case["ragged"]:
        return [(case["tq"], case["tk"])] * case["seqs"]
    r = random.Random(case["ragged"])
    some = lambda t: r.randint(max(1, t // 8), t)  # noqa: E731
    got = [(some(case["tq"]), some(case["tk"])) for _ in range(case["seqs"])]
    got[0] = (case["tq"], case["tk"])
    return got


def _pairs(lq, lk, causal):
    """Query-key pairs that the mask leaves."""
    if not causal:
        return lq * lk
    first = lk - lq + 1            # keys that the first query sees (may be negative)
    if first >= 1:
        return lq * (first + lk) // 2
    return lk * (lk + 1) // 2


def work(case):
    if case["op"] == "attn":
        lens = _lengths(case)
        nq, nk = sum(a for a, _ in lens), sum(b for _, b in lens)
        q, kv = nq * case["hq"] * case["d"] * 2, nk * case["hkv"] * case["d"] * 2
        pairs = sum(_pairs(a, b, case["causal"]) for a, b in lens) * case["hq"]
        lse = nq * case["hq"] * 4
        if case["grad"]:   # q, k, v, o, do, lse in; dq, dk, dv out; five products
            return {"bytes": 4 * q + 4 * kv + lse, "flops": 10 * pairs * case["d"]}
        return {"bytes": 2 * q + 2 * kv + lse, "flops": 4 * pairs * case["d"]}
    if case["op"] == "rope":
        n = case["t"] * (case["hq"] + 2 * case["hkv"]) * case["d"]
        table = case["t"] * case["rot"] * 4
        if case["grad"]:
            return {"bytes": 10 * n + table, "flops": 14 * n}
        return {"bytes": 6 * n + table, "flops": 7 * n}
    n = case["m"] * case["v"]
    return {"bytes": n * (8 if case["grad"] else 4) + case["m"] * case["k"] * 8,
            "flops": n * (6 if case["grad"] else 4)}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _cumulative(lengths):
    return torch.tensor([0] + list(np.cumsum(lengths)), dtype=torch.int32, device="cuda")


def _prepare_attn(case, g):
    dt = DTYPES[case["dtype"]]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    lens = _lengths(case)
    nq, nk = sum(a for a, _ in lens), sum(b for _, b in lens)
    st = dict(case=case, scale=1.0 / math.sqrt(d))
    if [a for a, _ in lens] == [b for _, b in lens]:
        # self attention: views of one packed buffer of q, k and v heads, the
        # output of the norm and rotation
        qkv = _randn(g, nq, hq + 2 * hkv, d).to(dt)
        st["q"], st["k"], st["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        dqkv = torch.empty_like(qkv)
        st["dq"], st["dk"], st["dv"] = dqkv[:, :hq], dqkv[:, hq:hq + hkv], dqkv[:, hq + hkv:]
    else:
        st["q"] = _randn(g, nq, hq, d).to(dt)
        kv = _randn(g, nk, 2 * hkv, d).to(dt)
        st["k"], st["v"] = kv[:, :hkv], kv[:, hkv:]
        dkv = torch.empty_like(kv)
        st["dq"], st["dk"], st["dv"] = torch.empty_like(st["q"]), dkv[:, :hkv], dkv[:, hkv:]
    st["cu_q"], st["cu_k"] = _cumulative([a for a, _ in lens]), _cumulative([b for _, b in lens])
    st["max_q"], st["max_k"] = max(a for a, _ in lens), max(b for _, b in lens)
    st["o"] = torch.empty((nq, hq, d), dtype=dt, device="cuda")
    st["lse"] = torch.empty((hq, nq), dtype=torch.float32, device="cuda")
    if case["grad"]:   # the forward pass's results and the gradient that comes back
        o, lse = _plain_attn(st)
        st["o"].copy_(o)
        st["lse"].copy_(lse)
        st["do"] = _randn(g, nq, hq, d).to(dt)
    else:
        del st["dq"], st["dk"], st["dv"]
    return st


def _prepare_rope(case, g):
    dt = DTYPES[case["dtype"]]
    t, hq, hkv, d, rot = case["t"], case["hq"], case["hkv"], case["d"], case["rot"]
    st = dict(case=case, eps=1e-6)
    st["x"] = _randn(g, t, (hq + 2 * hkv) * d) * 1.5
    st["wq"] = 1.0 + 0.2 * _randn(g, d)
    st["wk"] = 1.0 + 0.2 * _randn(g, d)
    # a table of 4096 positions, and documents of up to 4096 tokens packed
    # one after another from a random start
    inv = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64, device="cuda") * 2 / rot)
    ang = torch.arange(4096, dtype=torch.float64, device="cuda")[:, None] * inv
    st["cos"], st["sin"] = ang.cos().float().contiguous(), ang.sin().float().contiguous()
    start = torch.randint(0, 4096, (1,), generator=g, device="cuda")
    st["pos"] = ((torch.arange(t, device="cuda") + start) % 4096).to(torch.int32)
    qkv = torch.empty((t, hq + 2 * hkv, d), dtype=dt, device="cuda")
    if case["grad"]:
        qkv.copy_(_randn(g, t, hq + 2 * hkv, d))
        st["dx"] = torch.empty_like(st["x"])
        st["dwq"] = torch.empty(d, dtype=torch.float32, device="cuda")
        st["dwk"] = torch.empty(d, dtype=torch.float32, device="cuda")
    st["q"], st["k"], st["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    return st


def _prepare_distill(case, g):
    m, v, k = case["m"], case["v"], min(case["k"], case["v"])
    wide = -(-v // 4) * 4          # rows padded to whole 16-byte units
    st = dict(case=case, inv_norm=1.0 / m)
    st["logits"] = (4.0 * _randn(g, m, wide))[:, :v]
    # the teacher agrees in part: its logits are the student's and noise
    teacher = torch.empty((m, k), dtype=torch.float32, device="cuda")
    ids = torch.empty((m, k), dtype=torch.int32, device="cuda")
    for a in range(0, m, 1024):
        z = st["logits"][a:a + 1024]
        best, at = torch.topk(0.7 * z + 2.0 * _randn(g, z.shape[0], v), k, dim=1)
        teacher[a:a + 1024], ids[a:a + 1024] = best, at
    # rows with fewer entries (the rest -1), and padding rows with none
    kept = torch.randint(1, k + 1, (m, 1), generator=g, device="cuda")
    kept[::3] = k
    kept[5::16] = 0
    ids[torch.arange(k, device="cuda")[None] >= kept] = -1
    st["teacher"], st["ids"] = teacher, ids
    st["dlogits"] = torch.empty((m, wide), device="cuda")[:, :v] if case["grad"] else None
    st["losses"] = torch.empty(m, dtype=torch.float32, device="cuda")
    st["loss_sum"] = torch.empty(1, dtype=torch.float32, device="cuda")
    return st


def prepare(case, seed):
    g = _gen(seed)
    return {"attn": _prepare_attn, "rope": _prepare_rope,
            "distill": _prepare_distill}[case["op"]](case, g)


# ------------------------------------------------------------------ plain forms

def _padded(x, cu, most):
    """[tokens, heads, d] as [sequences, heads, most, d] in 32 bits."""
    at = (cu[:-1, None] + torch.arange(most, device=x.device)).clamp(max=max(x.shape[0] - 1, 0))
    return x[at.long()].float().transpose(1, 2)


def _packed(x, cu, tokens):
    """[sequences, heads, most, d] back to [tokens, heads, d]."""
    t = torch.arange(tokens, device=x.device)
    b = torch.searchsorted(cu[1:].long(), t, right=True)
    return x.transpose(1, 2)[b, t - cu[b]]


def _plain_scores(st, q, k):
    """Masked scaled scores [sequences, key heads, group, query, key]."""
    c = st["case"]
    i = torch.arange(st["max_q"], device=q.device)[:, None]
    j = torch.arange(st["max_k"], device=q.device)[None]
    lq, lk = (x.diff()[:, None, None] for x in (st["cu_q"], st["cu_k"]))
    keep = (i < lq) & (j < lk)
    if c["causal"]:
        keep = keep & (j <= i + lk - lq)
    s = torch.matmul(q, k.transpose(-1, -2)).mul_(st["scale"])
    return s.masked_fill_(~keep[:, None, None], -math.inf)


def _plain_operands(st):
    c = st["case"]
    b, g = c["seqs"], c["hq"] // c["hkv"]
    q = _padded(st["q"], st["cu_q"], st["max_q"]).view(b, c["hkv"], g, st["max_q"], c["d"])
    k = _padded(st["k"], st["cu_k"], st["max_k"])[:, :, None]
    v = _padded(st["v"], st["cu_k"], st["max_k"])[:, :, None]
    return q, k, v


def _plain_attn(st):
    q, k, v = _plain_operands(st)
    s = _plain_scores(st, q, k)
    top = s.amax(dim=-1, keepdim=True)
    shift = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = s.sub_(shift).exp_()
    total = p.sum(dim=-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))
    lse = shift + total.log()
    n = st["q"].shape[0]
    o = _packed(o.flatten(1, 2), st["cu_q"], n).to(st["q"].dtype)
    return o, _packed(lse.flatten(1, 2), st["cu_q"], n)[..., 0].t().contiguous()


def _plain_attn_grad(st):
    q, k, v = _plain_operands(st)
    do = _padded(st["do"], st["cu_q"], st["max_q"]).view(q.shape)
    p = _plain_scores(st, q, k)
    top = p.amax(dim=-1, keepdim=True)
    p = p.sub_(torch.where(torch.isinf(top), torch.zeros_like(top), top)).exp_()
    total = p.sum(dim=-1, keepdim=True)
    p = p.div_(torch.where(total > 0, total, torch.ones_like(total)))
    dv = torch.matmul(p.transpose(-1, -2), do).sum(dim=2)
    ds = torch.matmul(do, v.transpose(-1, -2))
    ds = ds.sub_((p * ds).sum(dim=-1, keepdim=True)).mul_(p).mul_(st["scale"])
    dq = torch.matmul(ds, k).flatten(1, 2)
    dk = torch.matmul(ds.transpose(-1, -2), q).sum(dim=2)
    dt, nq, nk = st["q"].dtype, st["q"].shape[0], st["k"].shape[0]
    return (_packed(dq, st["cu_q"], nq).to(dt), _packed(dk, st["cu_k"], nk).to(dt),
            _packed(dv, st["cu_k"], nk).to(dt))


def _rotated(x, cos, sin, rot, interleaved, back=False):
    """x [tokens, heads, d] with the pairs of its first `rot` entries turned
    by the tokens' angles (`back`: by the opposite angles)."""
    c, s = cos[:, None], -sin[:, None] if back else sin[:, None]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * c - b * s, a * s + b * c], dim=-1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * c - b * s, a * s + b * c], dim=-1)
    return torch.cat([turned, x[..., rot:]], dim=-1)


def _plain_rope(st):
    c = st["case"]
    dt, hq, hkv, d = DTYPES[c["dtype"]], c["hq"], c["hkv"], c["d"]
    x = st["x"].view(c["t"], hq + 2 * hkv, d)
    cos, sin = st["cos"][st["pos"].long()], st["sin"][st["pos"].long()]
    outs = []
    for lo, hi, w in ((0, hq, st["wq"]), (hq, hq + hkv, st["wk"])):
        part = x[:, lo:hi]
        r = torch.rsqrt(part.square().mean(dim=-1, keepdim=True) + st["eps"])
        outs.append(_rotated(part * r * w, cos, sin, c["rot"], c["interleaved"]).to(dt))
    return outs[0], outs[1], x[:, hq + hkv:].to(dt)


def _plain_rope_grad(st):
    c = st["case"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    x = st["x"].view(c["t"], hq + 2 * hkv, d)
    cos, sin = st["cos"][st["pos"].long()], st["sin"][st["pos"].long()]
    dxs, dws = [], []
    for lo, hi, w, dy in ((0, hq, st["wq"], st["q"]), (hq, hq + hkv, st["wk"], st["k"])):
        part = x[:, lo:hi]
        r = torch.rsqrt(part.square().mean(dim=-1, keepdim=True) + st["eps"])
        dn = _rotated(dy.float(), cos, sin, c["rot"], c["interleaved"], back=True)
        n = part * r
        dws.append((dn * n).sum(dim=(0, 1)))
        g = dn * w
        dxs.append(r * (g - n * (g * n).mean(dim=-1, keepdim=True)))
    dx = torch.cat([*dxs, st["v"].float()], dim=1).view(c["t"], -1)
    return dx, dws[0], dws[1]


def _plain_distill(st):
    c = st["case"]
    tau = c["tau"]
    has = st["ids"] >= 0
    any_row = has.any(dim=1)
    t = (st["teacher"] / tau).masked_fill(~has, -math.inf)
    top = t.amax(dim=1, keepdim=True)
    e = (t - torch.where(torch.isinf(top), torch.zeros_like(top), top)).exp()
    total = e.sum(dim=1, keepdim=True)
    p = e / torch.where(total > 0, total, torch.ones_like(total))
    log_p = torch.where(has, t - top - total.log(), torch.zeros_like(t))
    z = st["logits"] / tau
    zmax = z.amax(dim=1, keepdim=True)
    ez = (z - zmax).exp_()
    zsum = ez.sum(dim=1, keepdim=True)
    at = st["ids"].clamp(min=0).long()
    log_q = z.gather(1, at) - zmax - zsum.log()
    losses = tau * tau * (p * (log_p - log_q)).sum(dim=1)
    losses = torch.where(any_row, losses, torch.zeros_like(losses))
    if not c["grad"]:
        return losses, losses.sum()[None]
    dz = ez.div_(zsum).scatter_add_(1, at, -p).mul_(any_row[:, None]).mul_(tau * st["inv_norm"])
    return dz, losses, losses.sum()[None]


# ------------------------------------------------------------------ one pass

def run(st):
    c = st["case"]
    if not own:
        if c["op"] == "attn":
            return _plain_attn_grad(st) if c["grad"] else _plain_attn(st)
        if c["op"] == "rope":
            return _plain_rope_grad(st) if c["grad"] else _plain_rope(st)
        return _plain_distill(st)

    from transformer_linear_layer_tcgen05_gb300 import lin
    if c["op"] == "attn":
        how = dict(cu_q=st["cu_q"], cu_k=st["cu_k"], max_q=st["max_q"], max_k=st["max_k"],
                   causal=c["causal"], scale=st["scale"])
        if c["grad"]:
            return lin.lin_attention_backward(st["q"], st["k"], st["v"], st["o"], st["lse"],
                                              st["do"], st["dq"], st["dk"], st["dv"], **how)
        return lin.lin_attention(st["q"], st["k"], st["v"], st["o"], st["lse"], **how)
    if c["op"] == "rope":
        if c["grad"]:
            return lin.lin_qk_norm_rope_backward(
                st["x"], st["wq"], st["wk"], st["cos"], st["sin"], st["pos"], st["q"], st["k"],
                st["v"], st["dx"], st["dwq"], st["dwk"], eps=st["eps"],
                interleaved=c["interleaved"])
        return lin.lin_qk_norm_rope(st["x"], st["wq"], st["wk"], st["cos"], st["sin"], st["pos"],
                                    st["q"], st["k"], st["v"], eps=st["eps"],
                                    interleaved=c["interleaved"])
    got = lin.lin_distill_topk(st["logits"], st["ids"], st["teacher"], st["dlogits"],
                               st["losses"], st["loss_sum"], temperature=c["tau"],
                               inv_norm=st["inv_norm"])
    return got if c["grad"] else got[1:]


# ------------------------------------------------------------------ 64 bits

def _exact_attn(st):
    """Attention and its gradient from the definition, one sequence and head
    at a time."""
    c = st["case"]
    lens = _lengths(c)
    per = c["hq"] // c["hkv"]
    q, k, v = (st[n].double() for n in ("q", "k", "v"))
    out = torch.zeros_like(q)
    lse = torch.full((c["hq"], q.shape[0]), -math.inf, dtype=torch.float64, device="cuda")
    if c["grad"]:
        dout = st["do"].double()
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    q0 = k0 = 0
    for lq, lk in lens:
        rows, cols = slice(q0, q0 + lq), slice(k0, k0 + lk)
        hidden = None
        if c["causal"]:
            hidden = torch.ones(lq, lk, dtype=torch.bool, device="cuda").triu(1 + lk - lq)
        for h in range(c["hq"]):
            kh, vh = k[cols, h // per], v[cols, h // per]
            s = (q[rows, h] @ kh.T) * st["scale"]
            if hidden is not None:
                s = s.masked_fill_(hidden, -math.inf)
            lse[h, rows] = z = torch.logsumexp(s, dim=1)
            p = (s - z.masked_fill(torch.isinf(z), 0.0)[:, None]).exp_()
            o = p @ vh
            out[rows, h] = o
            if c["grad"]:
                g = dout[rows, h]
                dv[cols, h // per] += p.T @ g
                ds = p * (g @ vh.T - (g * o).sum(dim=1, keepdim=True)) * st["scale"]
                dq[rows, h] = ds @ kh
                dk[cols, h // per] += ds.T @ q[rows, h]
        q0, k0 = q0 + lq, k0 + lk
    return (dq, dk, dv) if c["grad"] else (out, lse)


def _exact_rope(st):
    """The norm, and each pair as a complex number times the angle's."""
    c = st["case"]
    hq, hkv, d, rot = c["hq"], c["hkv"], c["d"], c["rot"]
    x = st["x"].double().view(c["t"], -1, d)
    turn = torch.complex(st["cos"].double(), st["sin"].double())[st["pos"].long()][:, None]

    def times(y, by):
        y = y.clone()
        if c["interleaved"]:
            first, second = slice(0, rot, 2), slice(1, rot, 2)
        else:
            first, second = slice(0, rot // 2), slice(rot // 2, rot)
        z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * by
        y[..., first], y[..., second] = z.real, z.imag
        return y

    res, dws = [], []
    for lo, hi, w, name in ((0, hq, st["wq"], "q"), (hq, hq + hkv, st["wk"], "k")):
        part, w = x[:, lo:hi], w.double()
        rms = (part.pow(2).sum(dim=-1, keepdim=True) / d + st["eps"]).sqrt()
        if not c["grad"]:
            res.append(times(part / rms * w, turn))
            continue
        dn = times(st[name].double(), turn.conj())
        dws.append((dn * part / rms).sum(dim=(0, 1)))
        g = dn * w
        res.append(g / rms - part * (g * part).sum(dim=-1, keepdim=True) / (d * rms ** 3))
    if not c["grad"]:
        return res[0], res[1], x[:, hq + hkv:].clone()
    return torch.cat([*res, st["v"].double()], dim=1).view(c["t"], -1), dws[0], dws[1]


def _exact_distill(st):
    c = st["case"]
    tau, m = c["tau"], c["m"]
    losses = torch.zeros(m, dtype=torch.float64, device="cuda")
    dz = torch.zeros(m, c["v"], dtype=torch.float64, device="cuda") if c["grad"] else None
    for a in range(0, m, 512):
        z = st["logits"][a:a + 512].double() / tau
        log_q = torch.log_softmax(z, dim=1)
        ids = st["ids"][a:a + 512].long()
        has = ids >= 0
        log_p = torch.log_softmax(
            (st["teacher"][a:a + 512].double() / tau).masked_fill(~has, -math.inf), dim=1)
        p = log_p.exp().masked_fill(~has, 0.0)
        terms = p * (log_p - log_q.gather(1, ids.clamp(min=0)))
        losses[a:a + 512] = tau ** 2 * terms.masked_fill(~has, 0.0).sum(dim=1)
        if c["grad"]:
            g = log_q.exp().scatter_add(1, ids.clamp(min=0), -p) * (tau * st["inv_norm"])
            dz[a:a + 512] = g * has.any(dim=1, keepdim=True)
    total = losses.sum()[None]
    return (dz, losses, total) if c["grad"] else (losses, total)


def exact(case, seed):
    st = prepare(case, seed)
    return {"attn": _exact_attn, "rope": _exact_rope, "distill": _exact_distill}[case["op"]](st)
