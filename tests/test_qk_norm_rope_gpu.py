"""lin_qk_norm_rope and its gradient on the GPU against the fp64 oracle.

Bounds: the 16-bit heads are rounded once (u of themselves), everything else
is f32: a handful of roundings of 2^-24 each on terms whose magnitudes are
bounded entry by entry (the two products of a rotation; g and n mean|g n| of
the norm's gradient), taken as 2^-20 of them; a weight's gradient is a sum
over the tokens and heads, off by at most 2^-20 of its terms' magnitudes.
"""

import numpy as np
import pytest

from oracle import step_oracle as so
from tests.gpu_util import require_gpu
from transformer_linear_layer_tcgen05_gb300 import lin

pytestmark = pytest.mark.gpu

UNIT = {"float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}
E = 2.0 ** -20


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _host(t):
    return t.double().cpu().numpy()


def _setup(t, hq, hk, d, rot, dtype, seed, rows=50):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    dt = getattr(torch, dtype)
    st = dict(x=rnd(t, (hq + 2 * hk) * d), wq=1 + 0.3 * rnd(d), wk=1 + 0.3 * rnd(d))
    ang = 3 * rnd(rows, rot // 2)
    st["cos"], st["sin"] = (ang.cos().contiguous(), ang.sin().contiguous()) if rot else (None, None)
    st["pos"] = torch.randint(0, rows, (t,), generator=g, device="cuda", dtype=torch.int32)
    heads = torch.full((t, hq + 2 * hk, d), float("nan"), device="cuda", dtype=dt)
    grads = rnd(t, hq + 2 * hk, d).to(dt)
    cut = lambda y: (y[:, :hq], y[:, hq:hq + hk], y[:, hq + hk:])  # noqa: E731
    st["out"], st["dout"] = cut(heads), cut(grads)
    return st


def _tables(st, rows):
    if st["cos"] is None:
        return np.zeros((rows, 0)), np.zeros((rows, 0))
    return _host(st["cos"]), _host(st["sin"])


# (tokens, heads, key heads, dim, rot): one token; counts that leave groups
# and turns of heads part full; every group size; partial and no rotation
SHAPES = [(1, 1, 1, 64, 64), (5, 3, 1, 8, 8), (37, 4, 2, 32, 16), (129, 12, 12, 64, 64),
          (33, 7, 1, 96, 40), (70, 8, 2, 128, 128), (19, 5, 5, 80, 0), (21, 3, 2, 256, 256),
          (11, 2, 1, 200, 64)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_forward(shape, interleaved, dtype):
    import torch
    t, hq, hk, d, rot = shape
    st = _setup(*shape, dtype, seed=t + d)
    lin.lin_qk_norm_rope(st["x"], st["wq"], st["wk"], st["cos"], st["sin"], st["pos"], *st["out"],
                         eps=1e-5, interleaved=interleaved)
    torch.cuda.synchronize()
    assert lin.lin_get_device_status() == lin.LIN_SUCCESS
    cos, sin = _tables(st, 50)
    pos = st["pos"].cpu().numpy()
    want = so.qk_norm_rope(_host(st["x"]), _host(st["wq"]), _host(st["wk"]), cos, sin, pos, hq, hk,
                           1e-5, interleaved)
    for got, w in zip(st["out"], want):
        size = np.abs(w).max(axis=-1, keepdims=True) * 2   # both products of a pair
        assert np.all(np.abs(_host(got) - w) <= UNIT[dtype] * np.abs(w) + E * size + 2.0 ** -25)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_backward(shape, interleaved, dtype):
    import torch
    t, hq, hk, d, rot = shape
    st = _setup(*shape, dtype, seed=2 * t + d)
    dx = torch.full_like(st["x"], float("nan"))
    dwq, dwk = (torch.full((d,), float("nan"), device="cuda") for _ in range(2))
    args = (st["x"], st["wq"], st["wk"], st["cos"], st["sin"], st["pos"], *st["dout"])
    lin.lin_qk_norm_rope_backward(*args, dx, dwq, dwk, eps=1e-5, interleaved=interleaved)
    torch.cuda.synchronize()
    assert lin.lin_get_device_status() == lin.LIN_SUCCESS
    cos, sin = _tables(st, 50)
    pos = st["pos"].cpu().numpy()
    x, wq, wk = _host(st["x"]), _host(st["wq"]), _host(st["wk"])
    dy = [_host(y) for y in st["dout"]]
    want = so.qk_norm_rope_backward(x, wq, wk, cos, sin, pos, *dy, 1e-5, interleaved)
    # magnitudes: every product's absolute value
    xh = np.abs(x.reshape(t, -1, d))
    r = 1 / np.sqrt((xh ** 2).mean(-1, keepdims=True) + 1e-5)
    big = np.concatenate([np.abs(y).max(-1, keepdims=True) * 2 for y in dy], axis=1)
    w = max(np.abs(wq).max(), np.abs(wk).max())
    size = r * big * w * (1 + xh * r * (xh * r).mean(-1, keepdims=True)) + big
    assert np.all(np.abs(_host(dx) - want[0]).reshape(t, -1, d) <= E * size)
    terms = big * xh * r
    for got, ref, part in ((dwq, want[1], terms[:, :hq]), (dwk, want[2], terms[:, hq:hq + hk])):
        assert np.all(np.abs(_host(got) - ref) <= E * part.sum(axis=(0, 1)))
    # the same call gives the same bits
    again = torch.empty_like(dwq), torch.empty_like(dwk)
    lin.lin_qk_norm_rope_backward(*args, torch.empty_like(dx), *again, eps=1e-5,
                                  interleaved=interleaved)
    assert torch.equal(again[0], dwq) and torch.equal(again[1], dwk)


def test_gradient_is_the_difference_of_the_forward():
    import torch
    st = _setup(17, 3, 2, 64, 32, "bfloat16", seed=4)
    dx, dwq, dwk = torch.empty_like(st["x"]), *(torch.empty(64, device="cuda") for _ in range(2))
    lin.lin_qk_norm_rope_backward(st["x"], st["wq"], st["wk"], st["cos"], st["sin"], st["pos"],
                                  *st["dout"], dx, dwq, dwk, interleaved=True)
    cos, sin = _tables(st, 50)
    pos = st["pos"].cpu().numpy()
    args = [_host(st[n]) for n in ("x", "wq", "wk")]
    dys = [_host(y) for y in st["dout"]]
    f = lambda *a: sum((y * d).sum() for y, d in zip(  # noqa: E731
        so.qk_norm_rope(*a, cos, sin, pos, 3, 2, 1e-6, True), dys))
    rng = np.random.default_rng(4)
    for at, g in enumerate((dx, dwq, dwk)):
        d = rng.standard_normal(args[at].shape)
        up, dn = list(args), list(args)
        up[at], dn[at] = args[at] + 1e-5 * d, args[at] - 1e-5 * d
        diff = (f(*up) - f(*dn)) / 2e-5
        bound = 1e-5 * np.linalg.norm(_host(g)) * np.linalg.norm(d)
        assert abs((_host(g) * d).sum() - diff) <= bound


def test_default_positions_long_tables_and_held_positions():
    import torch
    st = _setup(40, 2, 1, 64, 64, "bfloat16", seed=6)
    how = (st["x"], st["wq"], st["wk"], st["cos"], st["sin"])
    lin.lin_qk_norm_rope(*how, None, *st["out"])
    a = [y.clone() for y in st["out"]]
    lin.lin_qk_norm_rope(*how, torch.arange(40, dtype=torch.int32, device="cuda"), *st["out"])
    assert all(torch.equal(x, y) for x, y in zip(a, st["out"]))
    # positions outside the table are held to its ends
    wild = torch.full((40,), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    wild[::2] = -5
    lin.lin_qk_norm_rope(*how, wild, *st["out"])
    b = [y.clone() for y in st["out"]]
    held = torch.full((40,), 49, dtype=torch.int32, device="cuda")
    held[::2] = 0
    lin.lin_qk_norm_rope(*how, held, *st["out"])
    assert all(torch.equal(x, y) for x, y in zip(b, st["out"]))


def test_a_zero_head_and_eps():
    # a head of zeros: norm sqrt(eps), output 0, gradient g / sqrt(eps)
    import torch
    st = _setup(3, 1, 1, 64, 0, "float16", seed=7)
    st["x"].zero_()
    lin.lin_qk_norm_rope(st["x"], st["wq"], st["wk"], None, None, None, *st["out"], eps=1e-4)
    assert all(torch.all(y == 0) for y in st["out"])
    dx, dwq, dwk = torch.empty_like(st["x"]), *(torch.empty(64, device="cuda") for _ in range(2))
    lin.lin_qk_norm_rope_backward(st["x"], st["wq"], st["wk"], None, None, None, *st["dout"], dx,
                                  dwq, dwk, eps=1e-4)
    want = _host(st["dout"][0])[:, 0] * _host(st["wq"]) * 100
    np.testing.assert_allclose(_host(dx)[:, :64], want, rtol=1e-5)
    assert torch.all(dwq == 0) and torch.all(dwk == 0)


def test_nothing_to_do():
    import torch
    z = lambda *s: torch.empty(s, device="cuda", dtype=torch.float16)  # noqa: E731
    w = torch.ones(64, device="cuda")
    x = torch.empty((0, 3 * 64), device="cuda")
    lin.lin_qk_norm_rope(x, w, w, None, None, None, z(0, 1, 64), z(0, 1, 64), z(0, 1, 64))
    dwq, dwk = torch.ones(64, device="cuda"), torch.ones(64, device="cuda")
    lin.lin_qk_norm_rope_backward(x, w, w, None, None, None, z(0, 1, 64), z(0, 1, 64),
                                  z(0, 1, 64), x.clone(), dwq, dwk)
    assert torch.all(dwq == 0) and torch.all(dwk == 0)


def test_refusals():
    import torch
    st = _setup(9, 2, 1, 64, 64, "float16", seed=8)

    def call(status, **kw):
        a = {**st, **kw}
        with pytest.raises(lin.LinError) as e:
            lin.lin_qk_norm_rope(a["x"], a["wq"], a["wk"], a["cos"], a["sin"], a["pos"], *a["out"],
                                 eps=a.get("eps", 1e-6))
        assert e.value.status == status

    odd = torch.ones(9, 30, device="cuda")
    call(lin.LIN_ERROR_UNSUPPORTED_SHAPE, cos=odd, sin=odd)           # rot 60
    call(lin.LIN_ERROR_INVALID_VALUE, cos=torch.ones(9, 40, device="cuda"),
         sin=torch.ones(9, 40, device="cuda"))                        # rot 80 > 64
    call(lin.LIN_ERROR_INVALID_VALUE, eps=-1.0)
    call(lin.LIN_ERROR_MISALIGNED, wq=torch.ones(65, device="cuda")[1:])
    call(lin.LIN_ERROR_ALIASING, out=(st["out"][0], st["out"][1], st["out"][1]))
    q = st["out"][0]
    with pytest.raises(ValueError):
        lin.lin_qk_norm_rope(st["x"][:, 1:], st["wq"], st["wk"], None, None, None, *st["out"])
    with pytest.raises(TypeError):
        lin.lin_qk_norm_rope(st["x"], st["wq"], st["wk"], st["cos"], st["sin"], st["pos"].long(),
                             *st["out"])
    with pytest.raises(TypeError):
        lin.lin_qk_norm_rope(st["x"], st["wq"], st["wk"], st["cos"], None, st["pos"], *st["out"])
    with pytest.raises(TypeError):
        lin.lin_qk_norm_rope(st["x"], st["wq"], st["wk"], None, None, None, q.float(),
                             *st["out"][1:])
