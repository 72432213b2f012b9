"""lin_attention and lin_attention_backward at the edges of their rules. Bounds
as in test_attention_gpu.py unless a test says otherwise.
"""

import numpy as np
import pytest

from oracle import step_oracle as so
from tests.gpu_util import require_gpu
from tests.test_attention_gpu import UNIT, _check, _cu, _host, _run, _setup
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


def _uneven(lens, hq, hk, d, dtype, k, seed):
    """Inputs whose dO falls by 2^k from a sequence's first row to its last."""
    import torch
    t = _setup(dtype, lens, hq, hk, d, seed=seed)
    t["v"].mul_(0.25)
    at = 0
    for n, _ in lens:
        fall = 2.0 ** torch.round(12 - k * torch.arange(n, device="cuda") / max(n - 1, 1))
        t["do"][at:at + n] *= fall.to(t["do"].dtype)[:, None, None]
        at += n
    return t


# One sequence, several with more and with fewer keys than queries, one long
# enough for parts of the queries, and heads that share a tile.
UNEVEN = [([(512, 512)], 2, 2, 64), ([(300, 500), (450, 400)], 4, 2, 128),
          ([(1100, 1100)], 1, 1, 64), ([(640, 640)], 3, 1, 96)]


@pytest.mark.parametrize("shape", UNEVEN, ids=lambda s: f"{s[0]}h{s[1]}x{s[2]}d{s[3]}")
@pytest.mark.parametrize("k", [14, 18])
def test_key_gradients_where_early_rows_are_large(shape, k):
    # A late key of a causal mask meets late rows only, so the scale of its dS
    # in binary16 must come from those. dS carries a scale that brings the
    # largest norm of dO among them to 2^4 or more: an entry's subnormal
    # spacing is then at most 2^-24 2^-4 of that norm, half of it an entry's
    # error; an entry of dK sums them times |q|. (The rows count in tiles of
    # 128, hence the first row of the sum.)
    lens, hq, hk, d = shape
    t = _uneven(lens, hq, hk, d, "float16", k, seed=40 + k)
    _run(t, lens, True)
    q, kk, v, do = (_host(t[n]) for n in ("q", "k", "v", "do"))
    cu_q = np.concatenate([[0], np.cumsum([a for a, _ in lens])])
    cu_k = np.concatenate([[0], np.cumsum([b for _, b in lens])])
    scale, u = d ** -0.5, UNIT["float16"]
    grads, sizes = so.attention_backward(q, kk, v, do, True, scale, cu_q, cu_k)
    spacing = np.zeros_like(kk)
    norms = np.sqrt((do ** 2).sum(-1))
    for b, (lq, lk) in enumerate(lens):
        for j in range(lk):
            first = max(j // 128 * 128 - (lk - lq) - 128, 0)
            rows = slice(cu_q[b] + first, cu_q[b] + lq)
            top = norms[rows].reshape(-1, hk, hq // hk).max(axis=(0, 2))
            mag = np.abs(q[rows]).reshape(-1, hk, hq // hk, d).sum(axis=(0, 2))
            spacing[cu_k[b] + j] = scale * 2.0 ** -29 * top[:, None] * mag
    err = np.abs(_host(t["dk"]) - grads[1])
    assert np.all(err <= u * np.abs(grads[1]) + (u + 2.0 ** -14) * sizes[1] + 2.0 ** -25 + spacing)
    for at, name in ((0, "dq"), (2, "dv")):
        err = np.abs(_host(t[name]) - grads[at])
        # (P carries 2^8 in binary16: an error of 2^-33 of dO's sum)
        far = 2.0 ** -33 * np.abs(do).sum() if name == "dv" else 0.0
        assert np.all(err <= u * np.abs(grads[at]) + (u + 2.0 ** -14) * sizes[at] + 2.0 ** -25 + far)


def test_views_of_heads_outside_tokens_interleaved():
    # q, k and v side by side for each head and token, both orders
    import torch
    lens, h, d = [(90, 90)], 3, 64
    for outer in ("heads", "tokens"):
        t = _setup("float16", lens, h, h, d, seed=70)
        for names in (("q", "k", "v"), ("dq", "dk", "dv")):
            shape = (h, 90, 3, d) if outer == "heads" else (90, h, 3, d)
            buf = torch.full(shape, float("nan"), device="cuda", dtype=torch.float16)
            for i, n in enumerate(names):
                view = buf[:, :, i].transpose(0, 1) if outer == "heads" else buf[:, :, i]
                view.copy_(t[n])
                t[n] = view
        _run(t, lens, True, packed=False)
        _check(t, lens, True, d ** -0.5, UNIT["float16"])


# (lengths, query heads, key heads, dim): more queries than keys, so that a
# causal mask leaves the first rows nothing; as many as a turn of 64 rows has,
# fewer and more, heads that share a tile, parts of the queries, and a sequence
# with every row seen beside one without
HIDDEN = [([(200, 90)], 2, 2, 64), ([(130, 70)], 4, 2, 128), ([(192, 128)], 1, 1, 96),
          ([(70, 3), (40, 40), (300, 299)], 6, 2, 64), ([(1700, 90)], 2, 1, 64), ([(90, 25)], 3, 1, 72)]


@pytest.mark.parametrize("shape", HIDDEN, ids=lambda s: f"{s[0]}h{s[1]}x{s[2]}d{s[3]}")
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_rows_without_a_key_give_no_gradient(shape, dtype):
    # Rows that the mask leaves nothing hold NaN and infinities (in Q and dO):
    # they reach nothing, and do not set the scale of the other rows' dS
    # (binary16 alone would lose a dO of 2^-14).
    import torch
    lens, hq, hk, d = shape
    t = _setup(dtype, lens, hq, hk, d, seed=50)
    t["do"].mul_(2.0 ** -14)
    clean = {n: t[n].clone() for n in ("q", "do")}
    at, nothing = 0, []
    for lq, lk in lens:
        hidden = slice(at, at + max(lq - lk, 0))
        nothing.append(hidden)
        for n, odd in (("q", float("inf")), ("do", float("-inf"))):
            t[n][hidden] = float("nan")
            t[n][hidden][::3] = odd
            clean[n][hidden] = 0
        at += lq
    _run(t, lens, True)
    for rows in nothing:
        assert torch.all(t["o"][rows] == 0) and torch.all(t["dq"][rows] == 0)
        assert torch.all(t["lse"][:, rows] == -float("inf"))
    q, do = (_host(clean[n]) for n in ("q", "do"))
    k, v = _host(t["k"]), _host(t["v"])
    cu_q = np.concatenate([[0], np.cumsum([a for a, _ in lens])])
    cu_k = np.concatenate([[0], np.cumsum([b for _, b in lens])])
    u = UNIT[dtype]
    grads, sizes = so.attention_backward(q, k, v, do, True, d ** -0.5, cu_q, cu_k)
    for name, g, size in zip(("dq", "dk", "dv"), grads, sizes):
        err = np.abs(_host(t[name]) - g)
        # (the result itself may be subnormal: half its spacing of 2^-24)
        assert np.all(err <= u * np.abs(g) + (u + 2.0 ** -14) * size + 2.0 ** -25), name


def test_parts_are_held_for_the_sequences_rows_only():
    # one short sequence in tensors of many rows: the parts' float32 results
    # are those of the sequence's rows, whatever else the tensors hold
    import torch
    n, lq, lk, h, d = 100_000, 70, 2000, 2, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(60)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").half()  # noqa: E731
    big = lambda: torch.full((n, h, d), float("nan"), device="cuda", dtype=torch.float16)  # noqa: E731
    q0, k0 = 31_000, 90_001
    for lq, lk in ((70, 2000), (2000, 70)):
        t = dict(q=big(), k=big(), v=big(), do=big(), o=big(), dq=big(), dk=big(), dv=big(),
                 lse=torch.full((h, n), float("nan"), device="cuda"))
        for name, at, m in (("q", q0, lq), ("do", q0, lq), ("k", k0, lk), ("v", k0, lk)):
            t[name][at:at + m] = rnd(m, h, d)
        how = dict(cu_q=torch.tensor([q0, q0 + lq], dtype=torch.int32, device="cuda"),
                   cu_k=torch.tensor([k0, k0 + lk], dtype=torch.int32, device="cuda"), max_q=lq,
                   max_k=lk, causal=False)
        lin.lin_attention(t["q"], t["k"], t["v"], t["o"], t["lse"], **how)
        kernels, workspace = lin.lin_last_launch_info()
        if lk == 2000:
            assert kernels == 2   # (at most 16 parts)
            assert 0 < workspace <= 16 * lq * h * (d + 1) * 4
        lin.lin_attention_backward(t["q"], t["k"], t["v"], t["o"], t["lse"], t["do"], t["dq"],
                                   t["dk"], t["dv"], **how)
        kernels, workspace = lin.lin_last_launch_info()
        assert kernels == 3
        assert 0 < workspace <= (n * h + 16 * h + 16 * 2 * 70 * h * d) * 4   # (delta: as LSE)
        torch.cuda.synchronize()
        assert lin.lin_get_device_status() == lin.LIN_SUCCESS
        inner = {x: (y[:, q0:q0 + lq] if x == "lse" else
                     y[k0:k0 + lk] if x in ("k", "v", "dk", "dv") else y[q0:q0 + lq])
                 for x, y in t.items()}
        _check(inner, [(lq, lk)], False, d ** -0.5, UNIT["float16"])
        for x in ("o", "dq"):
            assert t[x][:q0].isnan().all() and t[x][q0 + lq:].isnan().all()
        for x in ("dk", "dv"):
            assert t[x][:k0].isnan().all() and t[x][k0 + lk:].isnan().all()
