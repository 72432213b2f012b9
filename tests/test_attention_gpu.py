"""lin_attention and lin_attention_backward on the GPU against the fp64
oracle.

Bounds, with u the unit rounding of the tensors' type (2^-11 for binary16,
2^-8 for bfloat16): the result is rounded once (u of itself); P (dS) is
rounded once before its product, which moves a sum by at most u times the sum
of magnitudes; O inside delta carries its own rounding. The f32 parts
(exponentials, statistics, accumulation over the lengths here) stay below
2^-14 of those magnitudes; binary16's subnormal spacing adds a constant far
below 1e-6.
"""

import numpy as np
import pytest

from oracle import step_oracle as so
from tests.gpu_util import require_gpu
from transformer_linear_layer_tcgen05_gb300 import lin

pytestmark = pytest.mark.gpu

UNIT = {"float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _cu(lengths):
    import torch
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")


def _host(t):
    return t.double().cpu().numpy()


def _setup(dtype, lens, hq, hk, d, seed, layout="packed"):
    """Random q, k, v, do and NaN-filled results. Layouts: "packed" (views of
    one buffer of heads, tokens first), "heads" (heads first)."""
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = getattr(torch, dtype)
    nq, nk = sum(a for a, _ in lens), sum(b for _, b in lens)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dt)  # noqa: E731
    nan = lambda *s: torch.full(s, float("nan"), device="cuda", dtype=dt)  # noqa: E731
    if layout == "heads":
        make = lambda f, n, h: f(h, n, d).transpose(0, 1)  # noqa: E731
        t = dict(q=make(rnd, nq, hq), k=make(rnd, nk, hk), v=make(rnd, nk, hk),
                 dq=make(nan, nq, hq), dk=make(nan, nk, hk), dv=make(nan, nk, hk),
                 o=make(nan, nq, hq), do=make(rnd, nq, hq))
    else:
        kv, dkv = rnd(nk, 2 * hk, d), nan(nk, 2 * hk, d)
        q, dq = rnd(nq, hq + 1, d), nan(nq, hq + 1, d)   # (a head's room between tokens)
        t = dict(q=q[:, 1:], k=kv[:, :hk], v=kv[:, hk:], dq=dq[:, 1:], dk=dkv[:, :hk],
                 dv=dkv[:, hk:], o=nan(nq, hq, d), do=rnd(nq, hq, d))
    t["lse"] = torch.full((hq, nq), float("nan"), device="cuda")
    return t


def _run(t, lens, causal, scale=None, packed=True):
    import torch
    how = dict(causal=causal, scale=scale)
    if packed:
        how.update(cu_q=_cu([a for a, _ in lens]), cu_k=_cu([b for _, b in lens]),
                   max_q=max(a for a, _ in lens), max_k=max(b for _, b in lens))
    lin.lin_attention(t["q"], t["k"], t["v"], t["o"], t["lse"], **how)
    lin.lin_attention_backward(t["q"], t["k"], t["v"], t["o"], t["lse"], t["do"], t["dq"],
                               t["dk"], t["dv"], **how)
    torch.cuda.synchronize()
    assert lin.lin_get_device_status() == lin.LIN_SUCCESS


def _check(t, lens, causal, scale, u):
    q, k, v, do = (_host(t[n]) for n in ("q", "k", "v", "do"))
    cu_q = np.concatenate([[0], np.cumsum([a for a, _ in lens])])
    cu_k = np.concatenate([[0], np.cumsum([b for _, b in lens])])
    o, lse, w = so.attention(q, k, v, causal, scale, cu_q, cu_k)
    e = 2.0 ** -14
    got = _host(t["lse"])
    assert np.array_equal(np.isinf(got), np.isinf(lse))
    fin = np.isfinite(lse)
    np.testing.assert_allclose(got[fin], lse[fin], rtol=2e-6, atol=2e-6)
    assert np.all(np.abs(_host(t["o"]) - o) <= u * np.abs(o) + (u + e) * w + 1e-6)
    grads, sizes = so.attention_backward(q, k, v, do, causal, scale, cu_q, cu_k)
    for name, g, size in zip(("dq", "dk", "dv"), grads, sizes):
        err = np.abs(_host(t[name]) - g)
        assert np.all(err <= u * np.abs(g) + (u + e) * size + 1e-6), name


# (lengths of queries and keys, query heads, key heads, dim): one token, odd
# lengths, tiles' edges (127, 128, 129, 256, 257), empty sequences, more
# queries than keys and the reverse, shared heads, sizes between the tiles'
SHAPES = [
    ([(1, 1)], 1, 1, 64),
    ([(1, 300)], 2, 1, 128),
    ([(127, 129), (128, 128), (129, 127)], 2, 2, 64),
    ([(256, 257), (0, 40), (257, 255), (3, 0), (5, 5)], 4, 2, 128),
    ([(300, 20), (1, 1), (2, 130)], 3, 3, 32),
    ([(70, 333), (400, 140)], 6, 2, 96),
    ([(33, 47)], 5, 5, 8),
    ([(131, 131), (1, 2)], 8, 1, 72),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}x{s[1]}h{s[2]}d{s[3]}")
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_against_the_oracle(shape, causal, dtype):
    lens, hq, hk, d = shape
    t = _setup(dtype, lens, hq, hk, d, seed=hq * 100 + d)
    _run(t, lens, causal)
    _check(t, lens, causal, d ** -0.5, UNIT[dtype])


@pytest.mark.parametrize("causal", [False, True])
def test_heads_first_and_without_offsets(causal):
    lens = [(150, 150)]
    t = _setup("bfloat16", lens, 4, 2, 64, seed=9, layout="heads")
    _run(t, lens, causal, scale=0.3, packed=False)
    _check(t, lens, causal, 0.3, UNIT["bfloat16"])


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_sharp_scores(dtype):
    # scores of tens: the running maximum moves by far more than the 8 (in
    # base 2) below which it is left in place
    lens = [(200, 500)]
    t = _setup(dtype, lens, 2, 2, 64, seed=11)
    _run(t, lens, False, scale=2.0)
    _check(t, lens, False, 2.0, UNIT[dtype])


def test_a_rising_maximum():
    # every tile's scores above the last one's: the sums are scaled down each
    # time (q one-hot, so that S is k's first entry)
    import torch
    lens = [(130, 640)]
    t = _setup("float16", lens, 1, 1, 64, seed=12)
    t["q"].zero_()
    t["q"][..., 0] = 1
    t["k"][:, 0, 0] = torch.arange(640, device="cuda").half() / 8
    _run(t, lens, True, scale=1.0)
    _check(t, lens, True, 1.0, UNIT["float16"])


@pytest.mark.parametrize("size", [1e-6, 1e-3, 300.0])
def test_small_and_large_gradients_in_binary16(size):
    # dS scales with dO; binary16 alone would lose it below 6e-8
    lens = [(513, 513)]
    t = _setup("float16", lens, 2, 1, 64, seed=13)
    big = {n: t[n].clone() for n in ("q", "k", "v", "do")}
    _run(t, lens, True)
    ref = {n: _host(t[n]) for n in ("dq", "dk", "dv")}
    import torch
    t2 = _setup("float16", lens, 2, 1, 64, seed=13)
    exact2 = 2.0 ** np.round(np.log2(size))   # a power of two: dO's own rounding does not change
    t2["do"].copy_((big["do"].double() * exact2).to(torch.float16))
    if exact2 < 2.0 ** -10:   # (entries that binary16 keeps as subnormals: compare with the oracle)
        _run(t2, lens, True)
        q, k, v, do = (_host(t2[n]) for n in ("q", "k", "v", "do"))
        grads, sizes = so.attention_backward(q, k, v, do, True, 64 ** -0.5)
        for name, g, s in zip(("dq", "dk", "dv"), grads, sizes):
            # (the result itself is subnormal: half its spacing of 2^-24)
            assert np.all(np.abs(_host(t2[name]) - g) <=
                          2.0 ** -25 + UNIT["float16"] * np.abs(g) + (2.0 ** -11 + 2.0 ** -14) * s), name
        return
    _run(t2, lens, True)
    for name, r in ref.items():
        got = _host(t2[name]) / exact2
        # the same dS up to where single rows' scales were rounded: identical roundings
        np.testing.assert_allclose(got, r, rtol=2.0 ** -9, atol=2.0 ** -9 * np.abs(r).max())


@pytest.mark.parametrize("causal", [False, True])
def test_rows_outside_the_sequences(causal):
    # packed tensors with room before, between (none) and behind: NaN and
    # infinities there reach nothing, and nothing is written there
    import torch
    lens = [(100, 90), (77, 140)]
    big = [(40, 33)] + lens + [(150, 60)]
    t = _setup("float16", big, 2, 2, 64, seed=14)
    cq, ck = np.cumsum([0] + [a for a, _ in big]), np.cumsum([0] + [b for _, b in big])
    for n in ("q", "do"):
        t[n][:cq[1]] = float("nan")
        t[n][cq[3]:] = float("inf")
    for n in ("k", "v"):
        t[n][:ck[1]] = float("inf")
        t[n][ck[3]:] = float("nan")
    how = dict(cu_q=torch.tensor(cq[1:4], dtype=torch.int32, device="cuda"),
               cu_k=torch.tensor(ck[1:4], dtype=torch.int32, device="cuda"),
               max_q=100, max_k=140, causal=causal)
    lin.lin_attention(t["q"], t["k"], t["v"], t["o"], t["lse"], **how)
    lin.lin_attention_backward(t["q"], t["k"], t["v"], t["o"], t["lse"], t["do"], t["dq"],
                               t["dk"], t["dv"], **how)
    torch.cuda.synchronize()
    assert lin.lin_get_device_status() == lin.LIN_SUCCESS
    for n in ("o", "dq"):
        assert t[n][:cq[1]].isnan().all() and t[n][cq[3]:].isnan().all()
    for n in ("dk", "dv"):
        assert t[n][:ck[1]].isnan().all() and t[n][ck[3]:].isnan().all()
    inner = {n: (x[:, cq[1]:cq[3]] if n == "lse" else
                 x[ck[1]:ck[3]] if n in ("k", "v", "dk", "dv") else x[cq[1]:cq[3]])
             for n, x in t.items()}
    _check(inner, lens, causal, 64 ** -0.5, UNIT["float16"])


def test_gradient_is_the_difference_of_the_forward():
    # <grad, direction> of the kernel's gradients against central differences
    # of the oracle's forward loss, at bfloat16's accuracy of the sum
    lens = [(60, 90)]
    t = _setup("bfloat16", lens, 4, 2, 64, seed=15)
    _run(t, lens, True)
    q, k, v, do = (_host(t[n]) for n in ("q", "k", "v", "do"))
    rng = np.random.default_rng(15)
    loss = lambda *x: (so.attention(*x, True, 0.125)[0] * do).sum()  # noqa: E731
    for at, name in enumerate(("dq", "dk", "dv")):
        xs = [q, k, v]
        d = rng.standard_normal(xs[at].shape)
        h = 1e-5
        up, dn = list(xs), list(xs)
        up[at], dn[at] = xs[at] + h * d, xs[at] - h * d
        diff = (loss(*up) - loss(*dn)) / (2 * h)
        g = _host(t[name])
        # each entry of the gradient is off by about u of the entries' size,
        # independently: the inner product by that times the vectors' norms
        bound = 4 * UNIT["bfloat16"] * np.linalg.norm(g) * np.linalg.norm(d) / np.sqrt(g.size) * 4
        assert abs((g * d).sum() - diff) <= bound, name


def test_same_call_same_bits_and_other_streams():
    import torch
    lens = [(300, 300), (41, 41)]
    t = _setup("bfloat16", lens, 4, 2, 128, seed=16)
    _run(t, lens, True)
    first = {n: t[n].clone() for n in ("o", "lse", "dq", "dk", "dv")}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for n in first:
            t[n].fill_(float("nan"))
        _run(t, lens, True)
    side.synchronize()
    for n, x in first.items():
        assert torch.equal(t[n].nan_to_num(7.0), x.nan_to_num(7.0)), n


def test_in_a_graph():
    import torch
    lens = [(140, 140)]
    t = _setup("float16", lens, 2, 2, 64, seed=17)
    _run(t, lens, True, packed=False)
    first = {n: t[n].clone() for n in ("o", "dq", "dk", "dv")}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lin.lin_attention(t["q"], t["k"], t["v"], t["o"], t["lse"])
        lin.lin_attention_backward(t["q"], t["k"], t["v"], t["o"], t["lse"], t["do"], t["dq"],
                                   t["dk"], t["dv"])
    for n in first:
        t[n].zero_()
    g.replay()
    torch.cuda.synchronize()
    assert lin.lin_get_device_status() == lin.LIN_SUCCESS
    for n, x in first.items():
        assert torch.equal(t[n], x), n


def test_offsets_past_32_bits():
    # a token stride that puts the last rows more than 2^31 entries behind the first
    import torch
    n, stride = 300, 8 * 1024 * 1024
    base = torch.zeros(n * stride, dtype=torch.float16, device="cuda")
    big = base.as_strided((n, 1, 64), (stride, 64, 1))
    t = _setup("float16", [(n, n)], 1, 1, 64, seed=18)
    big.copy_(t["k"])
    t["k"] = big
    _run(t, [(n, n)], True, packed=False)
    _check(t, [(n, n)], True, 0.125, UNIT["float16"])


def test_nothing_to_do():
    import torch
    t = _setup("float16", [(40, 40)], 1, 1, 64, seed=19)
    empty = torch.empty((0, 1, 64), dtype=torch.float16, device="cuda")
    lse0 = torch.empty((1, 0), device="cuda")
    lin.lin_attention(empty, t["k"], t["v"], empty.clone(), lse0)
    # no keys: every row is empty
    lin.lin_attention(t["q"], empty, empty, t["o"], t["lse"])
    torch.cuda.synchronize()
    assert torch.all(t["o"] == 0) and torch.all(t["lse"] == -float("inf"))
    lin.lin_attention_backward(t["q"], empty, empty, t["o"], t["lse"], t["do"], t["dq"],
                               empty.clone(), empty.clone())
    # no queries: the keys' gradients are zero
    lin.lin_attention_backward(empty, t["k"], t["v"], empty, lse0, empty, empty.clone(), t["dk"],
                               t["dv"])
    torch.cuda.synchronize()
    assert torch.all(t["dq"] == 0) and torch.all(t["dk"] == 0) and torch.all(t["dv"] == 0)
    assert lin.lin_get_device_status() == lin.LIN_SUCCESS


def test_refusals():
    import torch
    t = _setup("float16", [(40, 40)], 4, 2, 64, seed=20)
    call = lambda **kw: lin.lin_attention(*({**t, **kw}[n] for n in ("q", "k", "v", "o", "lse")))  # noqa: E731
    before = t["o"].clone()

    def refused(status, **kw):
        with pytest.raises(lin.LinError) as e:
            call(**kw)
        assert e.value.status == status

    wide = torch.zeros((40, 4, 136), dtype=torch.float16, device="cuda")
    with pytest.raises(lin.LinError) as e:
        lin.lin_attention(wide, wide, wide, wide.clone(), t["lse"])
    assert e.value.status == lin.LIN_ERROR_UNSUPPORTED_SHAPE
    refused(lin.LIN_ERROR_ALIASING, o=t["q"])
    three = torch.zeros((40, 3, 64), dtype=torch.float16, device="cuda")
    refused(lin.LIN_ERROR_UNSUPPORTED_SHAPE, k=three, v=three)   # 4 heads over 3
    odd = torch.zeros(40 * 4 * 64 + 1, dtype=torch.float16, device="cuda")[1:].view(40, 4, 64)
    refused(lin.LIN_ERROR_MISALIGNED, q=odd)
    refused(lin.LIN_ERROR_INVALID_VALUE, q=t["q"][:1].expand(40, 4, 64))   # a stride of 0
    with pytest.raises(lin.LinError) as e:
        lin.lin_attention(t["q"], t["k"], t["v"], t["o"], t["lse"], scale=-1.0)
    assert e.value.status == lin.LIN_ERROR_INVALID_VALUE
    with pytest.raises(TypeError):
        call(k=t["k"].bfloat16())
    with pytest.raises(TypeError):
        call(q=t["q"].float())
    with pytest.raises(ValueError):
        call(v=t["v"][:39])
    with pytest.raises(ValueError):
        lin.lin_attention(t["q"], t["k"], t["v"], t["o"], t["lse"], cu_q=_cu([40]), cu_k=_cu([40]))
    with pytest.raises(lin.LinError) as e:
        lin.lin_attention_backward(t["q"], t["k"], t["v"], t["o"], t["lse"], t["do"], t["dq"],
                                   t["dk"], t["dk"])
    assert e.value.status == lin.LIN_ERROR_ALIASING
    torch.cuda.synchronize()
    assert torch.equal(t["o"].isnan(), before.isnan())


# (lengths, query heads, key heads, dim): few CTAs and a long other side, so
# that it is cut into parts (keys for O and dQ, queries for dK and dV), with
# sequences of other lengths beside the long one, shared heads (whose queries
# count as one long side), and rows that a causal mask leaves to the first
# part alone, or nothing
PARTS = [([(70, 2000)], 1, 1, 64), ([(1700, 90)], 2, 1, 128), ([(1600, 1600), (3, 1), (40, 200)], 1, 1, 64),
         ([(600, 600)], 4, 1, 40), ([(1900, 1550)], 1, 1, 96)]


@pytest.mark.parametrize("shape", PARTS, ids=lambda s: f"{s[0]}x{s[1]}h{s[2]}d{s[3]}")
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_long_and_few(shape, causal, dtype):
    lens, hq, hk, d = shape
    t = _setup(dtype, lens, hq, hk, d, seed=21)
    _run(t, lens, causal)
    kernels, workspace = lin.lin_last_launch_info()
    assert kernels >= 2 and workspace > 0
    _check(t, lens, causal, d ** -0.5, UNIT[dtype])
    first = {n: t[n].clone() for n in ("o", "lse", "dq", "dk", "dv")}
    _run(t, lens, causal)   # the parts are added in order: the same bits
    import torch
    for n, x in first.items():
        assert torch.equal(t[n].nan_to_num(7.0), x.nan_to_num(7.0)), n


def test_one_launch_each_where_there_is_no_need_for_parts():
    import torch
    t = _setup("float16", [(300, 300)], 2, 2, 64, seed=22)
    lin.lin_attention(t["q"], t["k"], t["v"], t["o"], t["lse"])
    assert lin.lin_last_launch_info() == (1, 0)
    lin.lin_attention_backward(t["q"], t["k"], t["v"], t["o"], t["lse"], t["do"], t["dq"], t["dk"],
                               t["dv"])
    kernels, workspace = lin.lin_last_launch_info()
    # delta of each row and head, and the norm of each query tile
    assert kernels == 2 and workspace == (300 * 2 + 3 * 2) * 4
    torch.cuda.synchronize()


def test_many_heads_and_sequences():
    # more CTAs than the SMs hold at once, most of them of short sequences
    lens = [(1 + 7 * i % 150, 1 + 11 * i % 130) for i in range(60)]
    t = _setup("bfloat16", lens, 6, 3, 64, seed=23)
    _run(t, lens, True)
    _check(t, lens, True, 0.125, UNIT["bfloat16"])


# (lengths, query heads, key heads, dim): the query heads of a key head as rows
# of one tile. Numbers of heads that divide a tile and that do not (3, 5, 48:
# rows of a tile that are nobody's, and the heads apart in the gradient), all
# rows of one token (128), more heads than rows (130: apart), one query on many
# keys, sequences that end inside a tile of the packed rows, and enough of them
# for two tiles to a CTA
SHARED = [([(1, 700)], 32, 8, 128), ([(5, 40), (1, 1), (43, 129), (0, 7), (86, 300)], 9, 3, 64),
          ([(31, 31), (33, 200), (2, 0)], 10, 2, 96), ([(3, 260), (1, 9)], 48, 1, 64),
          ([(2, 150)], 128, 1, 40), ([(2, 90)], 130, 1, 64), ([(70, 70), (9, 130)], 64, 1, 80),
          ([(17 + 3 * i, 60 + 5 * i) for i in range(24)], 16, 4, 64),
          ([(1, 2100), (3, 40)], 12, 3, 128)]


@pytest.mark.parametrize("shape", SHARED, ids=lambda s: f"{len(s[0])}h{s[1]}x{s[2]}d{s[3]}")
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("layout", ["packed", "heads"])
def test_shared_heads_of_short_queries(shape, causal, layout):
    lens, hq, hk, d = shape
    dtype = "bfloat16" if layout == "heads" else "float16"
    t = _setup(dtype, lens, hq, hk, d, seed=hq + d, layout=layout)
    _run(t, lens, causal)
    _check(t, lens, causal, d ** -0.5, UNIT[dtype])


@pytest.mark.parametrize("dim", [72, 96, 104])
def test_head_sizes_between_the_products(dim):
    # a long one of each width that the products run over, with parts and
    # without, beside one that ends inside a turn of 64 rows
    lens = [(1100, 1100), (65, 190)]
    t = _setup("bfloat16", lens, 2, 1, dim, seed=dim)
    _run(t, lens, True)
    _check(t, lens, True, dim ** -0.5, UNIT["bfloat16"])


@pytest.mark.parametrize("hq", [64, 128])
def test_more_queries_than_a_grid_has_packed_tiles(hq):
    # tiles of one or two queries would be more than the 65535 of a grid
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(31)
    n, d, tk = 132_000, 8, 5
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").half()  # noqa: E731
    q, k, v, do = rnd(n, hq, d), rnd(tk, 1, d), rnd(tk, 1, d), rnd(n, hq, d)
    o, dq = torch.empty_like(q), torch.empty_like(q)
    dk, dv = torch.empty_like(k), torch.empty_like(v)
    lse = torch.empty(hq, n, device="cuda")
    lin.lin_attention(q, k, v, o, lse, causal=False)
    lin.lin_attention_backward(q, k, v, o, lse, do, dq, dk, dv, causal=False)
    torch.cuda.synchronize()
    assert lin.lin_get_device_status() == lin.LIN_SUCCESS
    u, e = UNIT["float16"], 2.0 ** -14
    k64, v64 = k[:, 0].double(), v[:, 0].double()
    for at in (slice(0, 300), slice(65_400, 65_700), slice(n - 300, n)):
        p = torch.softmax(q[at].double() @ k64.T * d ** -0.5, -1)
        want = p @ v64
        assert torch.all((o[at] - want).abs() <= u * want.abs() + (u + e) * (p @ v64.abs()) + 1e-6)
        dp = do[at].double() @ v64.T
        ds = p * (dp - (p * dp).sum(-1, keepdim=True))
        want = ds @ k64 * d ** -0.5
        size = (p * (dp.abs() + (do[at].double() * o[at].double()).abs().sum(-1, keepdim=True))) \
            @ k64.abs() * d ** -0.5
        assert torch.all((dq[at] - want).abs() <= u * want.abs() + (u + e) * size + 1e-6)
