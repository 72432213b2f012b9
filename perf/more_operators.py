"""The rest of a decoder block's training step around the operators of
``operators.py``: attention whose scores are capped, biased by distance or kept
to a range of keys for each query, and its gradient; the norms before and after
a block with its gate and residual, and their gradient; the norm and rotation
of queries and keys by several position axes, and its gradient; and the AdamW
step over many tensors, with states in 32 bits or in 8.

``run`` computes each of them in its plain form (elementary torch operations
in 32 bits, rounded once at the end), or, with ``own`` true, by the entry
points of ``transformer_linear_layer_tcgen05_gb300.lin``.
"""

import math
import random

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
F8 = torch.float8_e4m3fn
BLOCK = 256                # entries of a tensor that share a scale of 8-bit states


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one 512-token sequence of the 768-wide model (12 heads of 64), scores
        # capped: the smallest attention call of a step, where latency counts
        dict(name="attn_fwd_512_cap_f16", op="attn", grad=False, dtype="f16", seqs=1, tq=512,
             tk=512, ragged=0, hq=12, hkv=12, d=64, causal=True, cap=20.0, bias=False,
             mask="none", empty=False),
        # the forward pass of 8192 tokens of several documents in one sequence,
        # scores capped, shared key heads
        dict(name="attn_fwd_8192_cap_docs_bf16", op="attn", grad=False, dtype="bf16", seqs=1,
             tq=8192, tk=8192, ragged=0, hq=32, hkv=8, d=128, causal=True, cap=50.0, bias=False,
             mask="docs", empty=False),
        # the gradient of packed prompts of uneven lengths: a prefix that all
        # queries see, causal behind it, distance bias, padding rows that see
        # nothing
        dict(name="attn_bwd_packed_prefix_bias_f16", op="attn", grad=True, dtype="f16", seqs=9,
             tq=997, tk=997, ragged=3, hq=12, hkv=6, d=64, causal=False, cap=0.0, bias=True,
             mask="prefix", empty=True),
        # the gradient of a long sequence, capped scores
        dict(name="attn_bwd_8192_cap_bf16", op="attn", grad=True, dtype="bf16", seqs=1, tq=8192,
             tk=8192, ragged=0, hq=16, hkv=4, d=128, causal=True, cap=50.0, bias=False,
             mask="none", empty=False),
        # between two blocks of the 768-wide model at 512 tokens: latency
        dict(name="norms_fwd_512x768_f32", op="norms", grad=False, dtype="f32", m=512, width=768,
             post=True, gate="channel"),
        # the gradient at an odd token count, 16-bit block outputs, a gate for
        # each token
        dict(name="norms_bwd_3001x1152_bf16", op="norms", grad=True, dtype="bf16", m=3001,
             width=1152, post=True, gate="token"),
        # the gradient at 16k tokens of the 2048-wide model
        dict(name="norms_bwd_16384x2048_f32", op="norms", grad=True, dtype="f32", m=16384,
             width=2048, post=True, gate="channel"),
        # a still image's patches after the QKV projection, 768-wide model
        dict(name="rope_axes_fwd_576_f16", op="rope", grad=False, dtype="f16", frames=1, rows=24,
             cols=24, hq=12, hkv=12, d=64, rot=64, interleaved=False, layout="sections"),
        # the gradient for a video's patches, pairs dealt to the axes in turn
        dict(name="rope_axes_bwd_video_bf16", op="rope", grad=True, dtype="bf16", frames=17,
             rows=28, cols=34, hq=32, hkv=8, d=128, rot=128, interleaved=False, layout="turns"),
        # the norm weights of many blocks (the group without decay): tensors of
        # 64 to 768 entries, where launches count
        dict(name="adamw_f32_norm_weights", op="adamw", bits=32, layers=32, width=768, ff=0,
             heads=64, vocab=0, scaled=False),
        # two blocks of the 768-wide model with binary16 copies of the matrices
        dict(name="adamw_f32_two_blocks", op="adamw", bits=32, layers=2, width=768, ff=2048,
             heads=64, vocab=0, scaled=True),
        # a large model's share of a card, 8-bit states
        dict(name="adamw_8bit_large", op="adamw", bits=8, layers=8, width=2048, ff=8192,
             heads=128, vocab=16384, scaled=True),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["attn_fwd", "attn_bwd", "norms", "rope", "adamw"])
    if kind.startswith("attn"):
        grad = kind == "attn_bwd"
        hkv = rng.choice([1, 2, 3, 4, 6, 8])
        hq = hkv * rng.choice([1, 2, 3, 4])
        d = rng.choice([32, 40, 64, 64, 80, 96, 128, 128])
        mask = rng.choice(["none", "docs", "prefix", "window"])
        cap = 8192 * 8192 * 16 * 128 * (1.0 if grad else 2.0)
        while True:
            tq = _log_uniform(rng, 1, 8192)
            tk = tq if rng.random() < 0.6 else _log_uniform(rng, 16, 8192)
            seqs = _log_uniform(rng, 1, 32)
            if seqs * tq * tk * hq * max(d, 64) <= cap and seqs * (tq + tk) >= 64:
                break
        return dict(op="attn", grad=grad, dtype=rng.choice(["f16", "bf16"]), seqs=seqs, tq=tq,
                    tk=tk, ragged=rng.choice([0, rng.randrange(1, 1000)]), hq=hq, hkv=hkv, d=d,
                    causal=mask != "prefix" and rng.random() < 0.75,
                    cap=rng.choice([0.0, 15.0, 30.0, 50.0]), bias=rng.random() < 0.5, mask=mask,
                    empty=rng.random() < 0.3)
    if kind == "norms":
        width = 4 * _log_uniform(rng, 16, 2048)
        m = _log_uniform(rng, 1, min(32768, 16384 * 2048 // width))
        return dict(op="norms", grad=rng.random() < 0.6, dtype=rng.choice(["f32", "f16", "bf16"]),
                    m=m, width=width, post=rng.random() < 0.7,
                    gate=rng.choice(["none", "channel", "token", "full"]))
    if kind == "rope":
        hkv = rng.choice([1, 2, 4, 6, 8, 12])
        hq = hkv * rng.choice([1, 2, 3, 4])
        d = rng.choice([32, 64, 80, 96, 128, 128, 256])
        rot = d if rng.random() < 0.6 else 8 * rng.randrange(1, d // 8 + 1)
        while True:
            frames, rows, cols = _log_uniform(rng, 1, 32), _log_uniform(rng, 1, 64), \
                _log_uniform(rng, 1, 64)
            if frames * rows * cols * (hq + 2 * hkv) * d <= 16384 * 48 * 128:
                break
        return dict(op="rope", grad=rng.random() < 0.6, dtype=rng.choice(["f16", "bf16"]),
                    frames=frames, rows=rows, cols=cols, hq=hq, hkv=hkv, d=d, rot=rot,
                    interleaved=rng.random() < 0.4, layout=rng.choice(["sections", "turns"]))
    while True:
        width = _log_uniform(rng, 64, 2048)
        ff = 0 if rng.random() < 0.2 else _log_uniform(rng, 128, 8192)
        layers = _log_uniform(rng, 1, 32)
        vocab = 0 if rng.random() < 0.5 else _log_uniform(rng, 100, 16384)
        case = dict(op="adamw", bits=rng.choice([8, 32]), layers=layers, width=width, ff=ff,
                    heads=rng.choice([64, 80, 128]), vocab=vocab, scaled=rng.random() < 0.5)
        if sum(math.prod(s) for s in _shapes(case)) <= 300_000_000:
            return case


def _lengths(case):
    """The sequences' (query, key) lengths: all alike, or (ragged, a seed)
    spread between an eighth of the longest and the longest."""
    if not case["ragged"]:
        return [(case["tq"], case["tk"])] * case["seqs"]
    r = random.Random(case["ragged"])
    some = lambda t: r.randint(max(1, t // 8), t)  # noqa: E731
    got = []
    for _ in range(case["seqs"]):
        a = some(case["tq"])
        got.append((a, a if case["tq"] == case["tk"] else some(case["tk"])))
    got[0] = (case["tq"], case["tk"])
    return got


def _key_ranges(case):
    """Per sequence the first key and the one behind the last that each query
    sees (numpy; the causal limit apart), by the case alone."""
    out = []
    r = np.random.RandomState(case["tq"] * 7 + case["tk"] + case["seqs"])
    for lq, lk in _lengths(case):
        at = np.arange(lq) + lk - lq          # the query's own place among the keys
        first, end = np.zeros(lq, np.int64), np.full(lq, lk, np.int64)
        if case["mask"] == "docs":            # documents of the sequence, one after another
            cuts = np.unique(np.concatenate([[0], r.randint(0, lk + 1, 1 + lk // 1500), [lk]]))
            doc = np.clip(np.searchsorted(cuts, at, side="right") - 1, 0, len(cuts) - 2)
            first, end = cuts[doc], cuts[doc + 1]
        elif case["mask"] == "prefix":        # a prefix for everyone, causal behind it
            end = np.maximum(at + 1, r.randint(0, lk + 1))
        elif case["mask"] == "window":
            first = at - max(1, lk // 3) + 1
        if case["empty"]:                     # padding rows
            none = r.rand(lq) < 0.05
            first, end = np.where(none, 5, first), np.where(none, 5, end)
        out.append((np.clip(first, 0, lk), np.clip(end, 0, lk)))
    return out


def _pairs(case):
    """Query-key pairs that the masks leave."""
    n = 0
    for (lq, lk), (first, end) in zip(_lengths(case), _key_ranges(case)):
        if case["causal"]:
            end = np.minimum(end, np.arange(lq) + lk - lq + 1)
        n += int(np.maximum(end - first, 0).sum())
    return n


def _shapes(case):
    """Tensors of the weights: a block's matrices and norm weights."""
    w, f, h = case["width"], case["ff"], case["heads"]
    kv = max(1, w // h // 4) * h
    block = [(w,), (w,), (h,), (h,)]
    if f:
        block += [(w, w + 2 * kv), (w, w), (w, f), (w, f), (f, w)]
    return block * case["layers"] + ([(w, case["vocab"])] if case["vocab"] else [])


def work(case):
    if case["op"] == "attn":
        lens = _lengths(case)
        nq, nk = sum(a for a, _ in lens), sum(b for _, b in lens)
        q, kv = nq * case["hq"] * case["d"] * 2, nk * case["hkv"] * case["d"] * 2
        pairs = _pairs(case) * case["hq"]
        rows = nq * case["hq"] * 4
        if case["grad"]:   # q, k, v, o, do, lse in; dq, dk, dv out; five products
            return {"bytes": 4 * q + 4 * kv + rows, "flops": 10 * pairs * case["d"]}
        return {"bytes": 2 * q + 2 * kv + rows, "flops": 4 * pairs * case["d"]}
    if case["op"] == "norms":
        n, b = case["m"] * case["width"], 4 if case["dtype"] == "f32" else 2
        full = 4 * n if case["gate"] == "full" else 0
        if case["grad"]:   # h, dh, y, dn (and the gate) in; dx, dy (and its gradient) out
            return {"bytes": n * (12 + 3 * b) + 2 * full, "flops": 30 * n}
        return {"bytes": n * (8 + 2 * b) + full, "flops": 10 * n}
    if case["op"] == "rope":
        t = case["frames"] * case["rows"] * case["cols"]
        n = t * (case["hq"] + 2 * case["hkv"]) * case["d"]
        table = max(case["frames"], case["rows"], case["cols"]) * case["rot"] * 4 + 12 * t
        if case["grad"]:
            return {"bytes": 10 * n + table, "flops": 14 * n}
        return {"bytes": 6 * n + table, "flops": 7 * n}
    n = sum(math.prod(s) for s in _shapes(case))
    n16 = sum(math.prod(s) for s in _shapes(case) if len(s) == 2)
    per = 28 if case["bits"] == 32 else 16 + 16 / BLOCK
    return {"bytes": n * per + 2 * n16, "flops": 15 * n}


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
    # scores of a few units, some of them near the cap
    st["q"] = (3.0 * _randn(g, nq, hq, d)).to(dt)
    kv = _randn(g, nk, 2 * hkv, d).to(dt)
    st["k"], st["v"] = kv[:, :hkv], kv[:, hkv:]
    st["cu_q"], st["cu_k"] = _cumulative([a for a, _ in lens]), _cumulative([b for _, b in lens])
    st["max_q"], st["max_k"] = max(a for a, _ in lens), max(b for _, b in lens)
    st["cap"] = case["cap"] or None
    st["slopes"] = None
    if case["bias"]:
        st["slopes"] = 2.0 ** (-8.0 * (torch.arange(hq, device="cuda") + 1) / hq)
    st["first"] = st["end"] = None
    if case["mask"] != "none" or case["empty"]:
        first, end = zip(*_key_ranges(case))
        st["first"], st["end"] = (torch.from_numpy(np.concatenate(x)).int().cuda()
                                  for x in (first, end))
    st["o"] = torch.empty((nq, hq, d), dtype=dt, device="cuda")
    st["lse"] = torch.empty((hq, nq), dtype=torch.float32, device="cuda")
    if case["grad"]:   # the forward pass's results and the gradient that comes back
        o, lse = _plain_attn(st)
        st["o"].copy_(o)
        st["lse"].copy_(lse)
        st["do"] = _randn(g, nq, hq, d).to(dt)
        st["dq"] = torch.empty_like(st["q"])
        dkv = torch.empty_like(kv)
        st["dk"], st["dv"] = dkv[:, :hkv], dkv[:, hkv:]
    return st


def _prepare_norms(case, g):
    dt, m, w = DTYPES[case["dtype"]], case["m"], case["width"]
    new = lambda dtype=torch.float32: torch.empty((m, w), dtype=dtype, device="cuda")  # noqa: E731
    st = dict(case=case, eps=1e-6, residual_scale=0.9, block_scale=0.7)
    st["y"] = (2.0 * _randn(g, m, w)).to(dt)
    gate = {"none": None, "channel": (w,), "token": (m, 1), "full": (m, w)}[case["gate"]]
    st["gate"] = None if gate is None else 0.5 + 0.3 * _randn(g, *gate)
    st["w_post"] = 1.0 + 0.2 * _randn(g, w) if case["post"] else None
    st["w_pre"] = 1.0 + 0.2 * _randn(g, w)
    if not case["grad"]:
        st["x"] = 1.5 * _randn(g, m, w)
        st["h"], st["n"] = new(), new(dt)
        return st
    st["h"] = 1.5 * _randn(g, m, w)
    st["dh"], st["dn"] = _randn(g, m, w), _randn(g, m, w).to(dt)
    st["dx"], st["dy"] = new(), new(dt)
    st["dgate"] = None if gate is None else torch.empty_like(st["gate"])
    st["dw_post"] = None if st["w_post"] is None else torch.empty_like(st["w_post"])
    st["dw_pre"] = torch.empty_like(st["w_pre"])
    return st


def _prepare_rope(case, g):
    dt = DTYPES[case["dtype"]]
    hq, hkv, d, rot = case["hq"], case["hkv"], case["d"], case["rot"]
    t = case["frames"] * case["rows"] * case["cols"]
    st = dict(case=case, eps=1e-6)
    st["x"] = _randn(g, t, (hq + 2 * hkv) * d) * 1.5
    st["wq"] = 1.0 + 0.2 * _randn(g, d)
    st["wk"] = 1.0 + 0.2 * _randn(g, d)
    # the patches' places in time, height and width, from a random start
    at = torch.cartesian_prod(*(torch.arange(case[k], device="cuda")
                                for k in ("frames", "rows", "cols"))).view(t, 3).t()
    st["pos"] = (at + torch.randint(0, 900, (3, 1), generator=g, device="cuda")).int().contiguous()
    pairs = rot // 2
    inv = 10000.0 ** (-torch.arange(pairs, dtype=torch.float64, device="cuda") / pairs)
    ang = torch.arange(1024, dtype=torch.float64, device="cuda")[:, None] * inv
    st["cos"], st["sin"] = ang.cos().float().contiguous(), ang.sin().float().contiguous()
    # the axis of each pair: a quarter to time and the rest to height and
    # width, or the axes in turn
    i = torch.arange(pairs, device="cuda")
    if case["layout"] == "turns":
        axis = i % 3
    else:
        first = pairs // 4
        axis = (i >= first).int() + (i >= first + (pairs - first + 1) // 2).int()
    st["axis"] = axis.int().contiguous()
    qkv = torch.empty((t, hq + 2 * hkv, d), dtype=dt, device="cuda")
    if case["grad"]:
        qkv.copy_(_randn(g, t, hq + 2 * hkv, d))
        st["dx"] = torch.empty_like(st["x"])
        st["dwq"] = torch.empty(d, dtype=torch.float32, device="cuda")
        st["dwk"] = torch.empty(d, dtype=torch.float32, device="cuda")
    st["q"], st["k"], st["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    return st


def _prepare_adamw(case, g):
    """The weights' tensors as a training program may keep them, one buffer of
    each kind with every tensor at a multiple of 256 entries in it."""
    shapes = _shapes(case)
    sizes = [math.prod(s) for s in shapes]
    starts = np.concatenate([[0], np.cumsum([-(-n // BLOCK) * BLOCK for n in sizes])])
    total = int(starts[-1])
    st = dict(case=case, step=37, lr=3e-4, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.1)
    used = torch.zeros(total, device="cuda")
    for a, n in zip(starts, sizes):
        used[int(a):int(a) + n] = 1.0
    # gradients whose size differs between blocks
    size = 1e-3 * torch.exp(_randn(g, total // BLOCK, 1))
    flat = {"p": 0.02 * _randn(g, total) * used,
            "g": ((_randn(g, total // BLOCK, BLOCK) * size).view(-1) * used)}
    m = (0.3 * _randn(g, total // BLOCK, BLOCK) * size).view(-1) * used
    r = ((0.3 + torch.rand(total // BLOCK, BLOCK, generator=g, device="cuda")) * size).view(-1) * used
    if case["bits"] == 32:
        flat["m"], flat["v"] = m, r * r
    else:
        flat["m"], flat["ms"] = _coded(m)
        flat["v"], flat["vs"] = _coded(r, least=True)
    flat["w16"] = flat["p"].half()
    st["flat"] = flat
    st["matrix"] = torch.zeros(total, dtype=torch.bool, device="cuda")
    per = {k: (BLOCK if k in ("ms", "vs") else 1) for k in flat}
    lists = {k: [] for k in flat}
    for s, a, n in zip(shapes, starts, sizes):
        a = int(a)
        if len(s) == 2:
            st["matrix"][a:a + n] = True
        for k, t in flat.items():
            if per[k] > 1:
                lists[k].append(t[a // BLOCK:a // BLOCK + -(-n // BLOCK)])
            else:
                lists[k].append(t[a:a + n].view(s) if k != "w16" or len(s) == 2 else None)
    st["lists"] = lists
    st["grad_scale"] = torch.full((1,), 0.8, device="cuda") if case["scaled"] else None
    return st


def prepare(case, seed):
    g = _gen(seed)
    return {"attn": _prepare_attn, "norms": _prepare_norms, "rope": _prepare_rope,
            "adamw": _prepare_adamw}[case["op"]](case, g)


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


def _plain_scores(st, q, k, slope=False):
    """Scores [sequences, key heads, group, query, key], capped, biased and
    masked; `slope`: also the cap's derivative (or None)."""
    c = st["case"]
    i = torch.arange(st["max_q"], device=q.device)[:, None]
    j = torch.arange(st["max_k"], device=q.device)[None]
    lq, lk = (x.diff()[:, None, None] for x in (st["cu_q"], st["cu_k"]))
    keep = (i < lq) & (j < lk)
    if c["causal"]:
        keep = keep & (j <= i + lk - lq)
    if st["first"] is not None:
        at = (st["cu_q"][:-1, None] + i[:, 0]).clamp(max=max(st["q"].shape[0] - 1, 0)).long()
        keep = keep & (j >= st["first"][at][..., None]) & (j < st["end"][at][..., None])
    s = torch.matmul(q, k.transpose(-1, -2)).mul_(st["scale"])
    chain = None
    if st["cap"]:
        s = s.div_(st["cap"]).tanh_()
        chain = 1.0 - s * s if slope else None
        s = s.mul_(st["cap"])
    if st["slopes"] is not None:
        far = (i + lk - lq - j).abs().float()[:, None, None]
        s = s.sub_(st["slopes"].view(1, c["hkv"], -1, 1, 1) * far)
    s = s.masked_fill_(~keep[:, None, None], -math.inf)
    return (s, chain) if slope else s


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
    p, chain = _plain_scores(st, q, k, slope=True)
    top = p.amax(dim=-1, keepdim=True)
    p = p.sub_(torch.where(torch.isinf(top), torch.zeros_like(top), top)).exp_()
    total = p.sum(dim=-1, keepdim=True)
    p = p.div_(torch.where(total > 0, total, torch.ones_like(total)))
    dv = torch.matmul(p.transpose(-1, -2), do).sum(dim=2)
    ds = torch.matmul(do, v.transpose(-1, -2))
    ds = ds.sub_((p * ds).sum(dim=-1, keepdim=True)).mul_(p).mul_(st["scale"])
    if chain is not None:
        ds = ds.mul_(chain)
    dq = torch.matmul(ds, k).flatten(1, 2)
    dk = torch.matmul(ds.transpose(-1, -2), q).sum(dim=2)
    dt, nq, nk = st["q"].dtype, st["q"].shape[0], st["k"].shape[0]
    return (_packed(dq, st["cu_q"], nq).to(dt), _packed(dk, st["cu_k"], nk).to(dt),
            _packed(dv, st["cu_k"], nk).to(dt))


def _plain_norms(st):
    y = st["y"].float()
    if st["w_post"] is not None:
        y = y * torch.rsqrt(y.square().mean(dim=-1, keepdim=True) + st["eps"]) * st["w_post"]
    if st["gate"] is not None:
        y = y * st["gate"]
    h = st["x"] * st["residual_scale"] + y * st["block_scale"]
    n = h * torch.rsqrt(h.square().mean(dim=-1, keepdim=True) + st["eps"]) * st["w_pre"]
    return h, n.to(st["y"].dtype)


def _plain_norm_grad(x, w, dn, eps):
    """The gradients of a norm's input and weight, and its normed input."""
    r = torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + eps)
    n = x * r
    g = dn * w
    return r * (g - n * (g * n).mean(dim=-1, keepdim=True)), (dn * n).sum(dim=0), n


def _plain_norms_grad(st):
    gate, dgate, dw_post = st["gate"], None, None
    d, dw_pre, _ = _plain_norm_grad(st["h"], st["w_pre"], st["dn"].float(), st["eps"])
    d = d + st["dh"]
    out = st["y"].float()
    dout = d * st["block_scale"]
    u = dout if gate is None else dout * gate
    if st["w_post"] is not None:
        u, dw_post, n = _plain_norm_grad(out, st["w_post"], u, st["eps"])
        out = n * st["w_post"]
    if gate is not None:
        dgate = dout * out
        if gate.dim() == 1:
            dgate = dgate.sum(dim=0)
        elif gate.shape[1] == 1:
            dgate = dgate.sum(dim=1, keepdim=True)
    return d * st["residual_scale"], u.to(st["y"].dtype), dgate, dw_post, dw_pre


def _angles(st):
    """The tables' entries of each token and pair."""
    pos = st["pos"][st["axis"].long()].long().t()          # [tokens, pairs]
    pair = torch.arange(pos.shape[1], device=pos.device)
    return st["cos"][pos, pair], st["sin"][pos, pair]


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
    x = st["x"].view(-1, hq + 2 * hkv, d)
    cos, sin = _angles(st)

    def part(lo, hi, w):
        y = x[:, lo:hi]
        r = torch.rsqrt(y.square().mean(dim=-1, keepdim=True) + st["eps"])
        return _rotated(y * r * w, cos, sin, c["rot"], c["interleaved"]).to(dt)

    return part(0, hq, st["wq"]), part(hq, hq + hkv, st["wk"]), x[:, hq + hkv:].to(dt)


def _plain_rope_grad(st):
    c = st["case"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    x = st["x"].view(-1, hq + 2 * hkv, d)
    cos, sin = _angles(st)

    def part(lo, hi, w, dy):
        y = x[:, lo:hi]
        r = torch.rsqrt(y.square().mean(dim=-1, keepdim=True) + st["eps"])
        dn = _rotated(dy.float(), cos, sin, c["rot"], c["interleaved"], back=True)
        n = y * r
        g = dn * w
        return r * (g - n * (g * n).mean(dim=-1, keepdim=True)), (dn * n).sum(dim=(0, 1))

    dq, dwq = part(0, hq, st["wq"], st["q"])
    dk, dwk = part(hq, hq + hkv, st["wk"], st["k"])
    return torch.cat([dq, dk, st["v"].float()], dim=1).view(x.shape[0], -1), dwq, dwk


def _coded(x, least=False):
    """x in blocks of 256 as e4m3 codes and a scale for each block: the largest
    magnitude stands at 448 (blocks below 2^-100 are zero). `least`: what is
    above zero has at least the smallest code."""
    b = x.view(-1, BLOCK)
    top = b.abs().amax(dim=1, keepdim=True)
    scale = torch.where(top >= 2.0 ** -100, top * (1.0 / 448.0), torch.zeros_like(top))
    inv = torch.where(scale > 0, scale.reciprocal(), torch.zeros_like(scale))
    c = b * inv
    if least:
        c = torch.where(c > 0, c.clamp(min=2.0 ** -9), c)
    return c.to(F8).view(-1), scale.view(-1)


def _plain_adamw(st):
    c, f = st["case"], st["flat"]
    (b1, b2), t = st["betas"], st["step"]
    g = f["g"] if st["grad_scale"] is None else f["g"] * st["grad_scale"]
    if c["bits"] == 32:
        m, v = f["m"], f["v"]
    else:
        m = (f["m"].float().view(-1, BLOCK) * f["ms"][:, None]).view(-1)
        r = (f["v"].float().view(-1, BLOCK) * f["vs"][:, None]).view(-1)
        v = r * r
    m = m * b1 + g * (1.0 - b1)
    v = v * b2 + (g * g) * (1.0 - b2)
    r = v.sqrt()
    denom = r * (1.0 / math.sqrt(1.0 - b2 ** t)) + st["eps"]
    p = f["p"] * (1.0 - st["lr"] * st["weight_decay"]) - (m / denom) * (st["lr"] / (1.0 - b1 ** t))
    f["p"].copy_(p)
    f["w16"].copy_(torch.where(st["matrix"], p, f["w16"].float()).half())
    if c["bits"] == 32:
        f["m"].copy_(m)
        f["v"].copy_(v)
        return [f[k] for k in ("p", "m", "v", "w16")]
    (mc, ms), (vc, vs) = _coded(m), _coded(r, least=True)
    f["m"].copy_(mc)
    f["ms"].copy_(ms)
    f["v"].copy_(vc)
    f["vs"].copy_(vs)
    return [f[k] for k in ("p", "m", "ms", "v", "vs", "w16")]


# ------------------------------------------------------------------ one pass

def run(st):
    c = st["case"]
    if not own:
        if c["op"] == "attn":
            return _plain_attn_grad(st) if c["grad"] else _plain_attn(st)
        if c["op"] == "norms":
            return _plain_norms_grad(st) if c["grad"] else _plain_norms(st)
        if c["op"] == "rope":
            return _plain_rope_grad(st) if c["grad"] else _plain_rope(st)
        return _plain_adamw(st)

    from transformer_linear_layer_tcgen05_gb300 import lin
    if c["op"] == "attn":
        how = dict(cap=st["cap"], slopes=st["slopes"], first_key=st["first"], end_key=st["end"],
                   cu_q=st["cu_q"], cu_k=st["cu_k"], max_q=st["max_q"], max_k=st["max_k"],
                   causal=c["causal"], scale=st["scale"])
        if c["grad"]:
            return lin.lin_attention_scores_backward(
                st["q"], st["k"], st["v"], st["o"], st["lse"], st["do"], st["dq"], st["dk"],
                st["dv"], **how)
        return lin.lin_attention_scores(st["q"], st["k"], st["v"], st["o"], st["lse"], **how)
    if c["op"] == "norms":
        how = dict(residual_scale=st["residual_scale"], block_scale=st["block_scale"],
                   eps=st["eps"])
        if c["grad"]:
            return lin.lin_block_norms_backward(
                st["h"], st["y"], st["gate"], st["w_post"], st["w_pre"], st["dh"], st["dn"],
                st["dx"], st["dy"], st["dgate"], st["dw_post"], st["dw_pre"], **how)
        return lin.lin_block_norms(st["x"], st["y"], st["gate"], st["w_post"], st["w_pre"],
                                   st["h"], st["n"], **how)
    if c["op"] == "rope":
        if c["grad"]:
            return lin.lin_qk_norm_rope_axes_backward(
                st["x"], st["wq"], st["wk"], st["cos"], st["sin"], st["pos"], st["axis"], st["q"],
                st["k"], st["v"], st["dx"], st["dwq"], st["dwk"], eps=st["eps"],
                interleaved=c["interleaved"])
        return lin.lin_qk_norm_rope_axes(
            st["x"], st["wq"], st["wk"], st["cos"], st["sin"], st["pos"], st["axis"], st["q"],
            st["k"], st["v"], eps=st["eps"], interleaved=c["interleaved"])
    x, f = st["lists"], st["flat"]
    how = dict(step=st["step"], lr=st["lr"], betas=st["betas"], eps=st["eps"],
               weight_decay=st["weight_decay"], grad_scale=st["grad_scale"])
    if c["bits"] == 32:
        lin.lin_adamw(x["p"], x["g"], x["m"], x["v"], w16=x["w16"], **how)
        return [f[k] for k in ("p", "m", "v", "w16")]
    lin.lin_adamw(x["p"], x["g"], x["m"], x["v"], m_scale=x["ms"], v_scale=x["vs"], w16=x["w16"],
                  **how)
    return [f[k] for k in ("p", "m", "ms", "v", "vs", "w16")]


# ------------------------------------------------------------------ 64 bits

def _exact_attn(st):
    """From the definition, one sequence and head at a time."""
    c = st["case"]
    per = c["hq"] // c["hkv"]
    q, k, v = (st[n].double() for n in ("q", "k", "v"))
    out = torch.zeros_like(q)
    lse = torch.full((c["hq"], q.shape[0]), -math.inf, dtype=torch.float64, device="cuda")
    if c["grad"]:
        dout = st["do"].double()
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    q0 = k0 = 0
    for (lq, lk), (first, end) in zip(_lengths(c), _key_ranges(c)):
        rows, cols = slice(q0, q0 + lq), slice(k0, k0 + lk)
        here = torch.arange(lq, device="cuda")[:, None] + (lk - lq)
        key = torch.arange(lk, device="cuda")[None]
        hidden = (key < torch.from_numpy(first).cuda()[:, None]) | \
                 (key >= torch.from_numpy(end).cuda()[:, None])
        if c["causal"]:
            hidden |= key > here
        for h in range(c["hq"]):
            kh, vh = k[cols, h // per], v[cols, h // per]
            s = (q[rows, h] @ kh.T) * st["scale"]
            if st["cap"]:
                s = torch.tanh(s / st["cap"]) * st["cap"]
            chain = 1.0 - (s / st["cap"]) ** 2 if st["cap"] and c["grad"] else None
            if st["slopes"] is not None:
                s = s - st["slopes"][h].double() * (here - key).abs()
            s = s.masked_fill_(hidden, -math.inf)
            lse[h, rows] = z = torch.logsumexp(s, dim=1)
            p = (s - z.masked_fill(torch.isinf(z), 0.0)[:, None]).exp_()
            o = p @ vh
            out[rows, h] = o
            if c["grad"]:
                g = dout[rows, h]
                dv[cols, h // per] += p.T @ g
                ds = p * (g @ vh.T - (g * o).sum(dim=1, keepdim=True)) * st["scale"]
                if chain is not None:
                    ds = ds * chain
                dq[rows, h] = ds @ kh
                dk[cols, h // per] += ds.T @ q[rows, h]
        q0, k0 = q0 + lq, k0 + lk
    return (dq, dk, dv) if c["grad"] else (out, lse)


def _exact_norms(st):
    c = st["case"]
    w = c["width"]
    y = st["y"].double()
    wide = lambda t: None if t is None else t.double()  # noqa: E731
    gate, wpost, wpre = wide(st["gate"]), wide(st["w_post"]), wide(st["w_pre"])
    rms_y = (y.pow(2).sum(dim=1, keepdim=True) / w + st["eps"]).sqrt()
    out = y if wpost is None else y / rms_y * wpost
    gated = out if gate is None else out * gate
    if not c["grad"]:
        h = st["residual_scale"] * st["x"].double() + st["block_scale"] * gated
        return h, h / (h.pow(2).sum(dim=1, keepdim=True) / w + st["eps"]).sqrt() * wpre
    h, dn = st["h"].double(), st["dn"].double()
    rms = (h.pow(2).sum(dim=1, keepdim=True) / w + st["eps"]).sqrt()
    g = dn * wpre
    d = st["dh"].double() + g / rms - h * (g * h).sum(dim=1, keepdim=True) / (w * rms ** 3)
    dw_pre = (dn * h / rms).sum(dim=0)
    db = st["block_scale"] * d
    dgate = None
    if gate is not None:
        dgate = db * out
        dgate = dgate.sum(dim=0) if c["gate"] == "channel" else \
            dgate.sum(dim=1, keepdim=True) if c["gate"] == "token" else dgate
        db = db * gate
    dw_post, dy = None, db
    if wpost is not None:
        dw_post = (db * y / rms_y).sum(dim=0)
        g = db * wpost
        dy = g / rms_y - y * (g * y).sum(dim=1, keepdim=True) / (w * rms_y ** 3)
    return st["residual_scale"] * d, dy, dgate, dw_post, dw_pre


def _exact_rope(st):
    """The norm, and each pair as a complex number times the angle's."""
    c = st["case"]
    hq, hkv, d, rot = c["hq"], c["hkv"], c["d"], c["rot"]
    x = st["x"].double()
    x = x.view(x.shape[0], -1, d)
    pairs = torch.arange(rot // 2, device="cuda")
    place = torch.stack([st["pos"][int(a)] for a in st["axis"].tolist()], dim=1).long()
    turn = torch.complex(st["cos"].double()[place, pairs], st["sin"].double()[place, pairs])[:, None]

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
    return torch.cat([*res, st["v"].double()], dim=1).view(x.shape[0], -1), dws[0], dws[1]


def _exact_adamw(st):
    """The definition in 64 bits; 8-bit states: the scales, and the codes' values
    before they are rounded to one."""
    c, f = st["case"], st["flat"]
    (b1, b2), t = st["betas"], st["step"]
    g = f["g"].double()
    if st["grad_scale"] is not None:
        g = g * st["grad_scale"].double()
    each = lambda k: f[k].double().repeat_interleave(BLOCK)  # noqa: E731
    if c["bits"] == 32:
        m, v = f["m"].double(), f["v"].double()
    else:
        m, v = f["m"].double() * each("ms"), (f["v"].double() * each("vs")).pow(2)
    m, v = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g.pow(2)
    m_hat, v_hat = m / (1 - b1 ** t), v / (1 - b2 ** t)
    p = f["p"].double()
    p = p - st["lr"] * (st["weight_decay"] * p + m_hat / (v_hat.sqrt() + st["eps"]))
    w16 = torch.where(st["matrix"], p, f["w16"].double())
    if c["bits"] == 32:
        return [p, m, v, w16]
    got = []
    for x in (m, v.sqrt()):
        scale = x.abs().view(-1, BLOCK).amax(dim=1) / 448
        one = torch.where(scale > 0, scale, torch.ones_like(scale))
        got += [(x.view(-1, BLOCK) / one[:, None]).view(-1), scale]
    return [p, *got, w16]


def exact(case, seed):
    st = prepare(case, seed)
    return {"attn": _exact_attn, "norms": _exact_norms, "rope": _exact_rope,
            "adamw": _exact_adamw}[case["op"]](st)
