"""lin_block_norms and its gradient on the GPU against the fp64 oracle.

Bounds: everything is float32 until the results of 16-bit type, which are
rounded once (half a step of themselves). A row's sums are trees of at most 16
terms in a thread and 16 warps, the sums over the tokens of at most some
dozens of terms in a row: below 2^6 roundings of 2^-24 each on terms whose
magnitudes the oracle gives; the gradient stands on two such sums behind each
other. Taken as 2^-17 of the magnitudes.
"""

import numpy as np
import pytest

from oracle import train_oracle as to
from tests.gpu_util import require_gpu
from transformer_linear_layer_tcgen05_gb300 import lin

pytestmark = pytest.mark.gpu

UNIT = {"float32": 2.0 ** -24, "float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}
E = 2.0 ** -17
TINY = 2.0 ** -24   # (binary16's subnormal steps are 2^-24)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _host(t):
    return None if t is None else t.double().cpu().numpy()


def _gate_shape(form, m, w):
    return {"none": None, "channel": (w,), "token": (m, 1), "full": (m, w)}[form]


def _setup(m, w, dtype, gate, post, seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    dt = getattr(torch, dtype)
    shape = _gate_shape(gate, m, w)
    st = dict(x=rnd(m, w), y=(2 * rnd(m, w)).to(dt), dh=rnd(m, w), dn=rnd(m, w).to(dt),
              gate=None if shape is None else rnd(*shape), w_post=1 + rnd(w) if post else None,
              w_pre=1 + rnd(w))
    return st


HOW = dict(residual_scale=0.75, block_scale=1.25, eps=1e-5)


def _nan(t, dtype=None):
    import torch
    return torch.full_like(t, float("nan"), dtype=dtype)


def _ok():
    import torch
    torch.cuda.synchronize()
    assert lin.lin_get_device_status() == lin.LIN_SUCCESS


def _near(got, want, size, unit):
    err = np.abs(_host(got) - want)
    assert np.all(err <= unit * np.abs(want) + E * size + TINY * (unit > 2.0 ** -20))


def _check_forward(st, dtype):
    h, n = _nan(st["x"]), _nan(st["y"])
    lin.lin_block_norms(st["x"], st["y"], st["gate"], st["w_post"], st["w_pre"], h, n, **HOW)
    _ok()
    (wh, wn), (sh, sn) = to.block_norms(*(_host(st[k]) for k in ("x", "y", "gate", "w_post", "w_pre")),
                                        *HOW.values())
    _near(h, wh, sh, UNIT["float32"])
    _near(n, wn, sn, UNIT[dtype])


def _check_backward(st, dtype):
    outs = dict(dx=_nan(st["x"]), dy=_nan(st["y"]),
                **{"d" + k: None if st[k] is None else _nan(st[k]) for k in ("gate", "w_post", "w_pre")})
    args = [st[k] for k in ("x", "y", "gate", "w_post", "w_pre", "dh", "dn")]
    call = lambda o: lin.lin_block_norms_backward(  # noqa: E731
        *args, *(o[k] for k in ("dx", "dy", "dgate", "dw_post", "dw_pre")), **HOW)
    call(outs)
    _ok()
    want, size = to.block_norms_backward(*(_host(t) for t in args), *HOW.values())
    for k, t in outs.items():
        if t is not None:
            _near(t, want[k], size[k], UNIT[dtype] if k == "dy" else UNIT["float32"])
    # the same call gives the same bits
    again = {k: None if t is None else _nan(t) for k, t in outs.items()}
    call(again)
    assert all(t is None or t.equal(again[k]) for k, t in outs.items())


# (tokens, width): one row; rows that leave teams, warps and units part full;
# the borders between one, two and four units to a thread; the widest
SHAPES = [(1, 4), (5, 12), (37, 64), (130, 132), (3, 516), (129, 768), (33, 1024), (50, 1028),
          (700, 1152), (9, 4096), (7, 4100), (3, 8188), (2, 8192)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", ["float32", "float16", "bfloat16"])
def test_shapes(shape, dtype):
    m, w = shape
    st = _setup(m, w, dtype, ("channel", "token", "full", "none")[(m + w // 4) % 4], w % 8 == 4 or m % 2 == 0,
                seed=m + w)
    _check_forward(st, dtype)
    _check_backward(st, dtype)


@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("shape", [(19, 260), (401, 64)])
def test_gates(gate, post, shape):
    st = _setup(*shape, "bfloat16", gate, post, seed=5)
    _check_forward(st, "bfloat16")
    _check_backward(st, "bfloat16")


def test_a_norm_alone():
    import torch
    st = _setup(23, 320, "float32", "none", False, seed=1)
    n = _nan(st["x"])
    lin.lin_block_norms(st["x"], None, None, None, st["w_pre"], None, n, eps=1e-5)
    _ok()
    (_, want), (_, size) = to.block_norms(_host(st["x"]), None, None, None, _host(st["w_pre"]), 1, 1, 1e-5)
    _near(n, want, size, UNIT["float32"])
    dx, dw = _nan(st["x"]), _nan(st["w_pre"])
    lin.lin_block_norms_backward(st["x"], None, None, None, st["w_pre"], None, st["dn"], dx, None,
                                 None, None, dw, eps=1e-5)
    _ok()
    want, size = to.block_norms_backward(_host(st["x"]), None, None, None, _host(st["w_pre"]), None,
                                         _host(st["dn"]), 1, 1, 1e-5)
    _near(dx, want["dx"], size["dx"], UNIT["float32"])
    _near(dw, want["dw_pre"], size["dw_pre"], UNIT["float32"])
    assert torch.isfinite(dx).all()


@pytest.mark.parametrize("post", [False, True])
def test_no_norm_behind(post):
    st = _setup(40, 96, "float16", "channel", post, seed=2)
    h = _nan(st["x"])
    lin.lin_block_norms(st["x"], st["y"], st["gate"], st["w_post"], None, h, None, **HOW)
    _ok()
    (want, _), (size, _) = to.block_norms(*(_host(st[k]) for k in ("x", "y", "gate", "w_post")), None,
                                          *HOW.values())
    _near(h, want, size, UNIT["float32"])
    dx, dy, dg = _nan(st["x"]), _nan(st["y"]), _nan(st["gate"])
    dp = _nan(st["w_post"]) if post else None
    lin.lin_block_norms_backward(None, st["y"], st["gate"], st["w_post"], None, st["dh"], None, dx,
                                 dy, dg, dp, None, **HOW)
    _ok()
    want, size = to.block_norms_backward(None, *(_host(st[k]) for k in ("y", "gate", "w_post")), None,
                                         _host(st["dh"]), None, *HOW.values())
    for k, t, u in (("dx", dx, "float32"), ("dy", dy, "float16"), ("dgate", dg, "float32"),
                    ("dw_post", dp, "float32")):
        if t is not None:
            _near(t, want[k], size[k], UNIT[u])


def test_in_place():
    import torch
    st = _setup(300, 768, "float32", "channel", True, seed=3)
    h, n, n2 = (_nan(st["x"]) for _ in range(3))
    args = [st[k] for k in ("y", "gate", "w_post", "w_pre")]
    lin.lin_block_norms(st["x"], *args, h, n, **HOW)
    x = st["x"].clone()
    lin.lin_block_norms(x, *args, x, n2, **HOW)
    _ok()
    assert torch.equal(x, h) and torch.equal(n2, n)
    outs = lambda: [_nan(st[k]) for k in ("y", "gate", "w_post", "w_pre")]  # noqa: E731
    a, b, dx, dh = outs(), outs(), _nan(h), st["dh"].clone()
    lin.lin_block_norms_backward(h, *args, st["dh"], st["dn"], dx, *a, **HOW)
    lin.lin_block_norms_backward(h, *args, dh, st["dn"], dh, *b, **HOW)
    _ok()
    assert torch.equal(dh, dx) and all(torch.equal(s, t) for s, t in zip(a, b))


def test_no_tokens():
    import torch
    new = lambda *s: torch.full(s, float("nan"), device="cuda")  # noqa: E731
    x, w = new(0, 64), new(64)
    lin.lin_block_norms(x, new(0, 64), w, w, w, new(0, 64), new(0, 64))
    dg, dp, dw = new(64), new(64), new(64)
    lin.lin_block_norms_backward(x, new(0, 64), w, w, w, new(0, 64), new(0, 64), new(0, 64), new(0, 64),
                                 dg, dp, dw)
    _ok()
    assert not dg.any() and not dp.any() and not dw.any()


def test_zero_rows_and_numbers_that_are_none():
    import torch
    st = _setup(6, 128, "float32", "none", True, seed=4)
    st["x"][1], st["y"][1] = 0, 0
    st["y"][3, 5] = float("inf")
    st["x"][4, 7] = float("nan")
    h, n = _nan(st["x"]), _nan(st["x"])
    lin.lin_block_norms(st["x"], st["y"], None, st["w_post"], st["w_pre"], h, n, eps=1e-5)
    _ok()
    rows = torch.isfinite(n).all(dim=1).tolist()
    assert rows == [True, True, True, False, False, True] and not n[1].any() and not h[1].any()


def test_gradient_is_the_difference_of_the_forward():
    import torch
    m, w = 13, 96
    st = _setup(m, w, "float32", "token", True, seed=6)
    ch, cn = st["dh"], st["dn"]
    h, n = _nan(ch), _nan(ch)

    def loss(**new):
        a = {**st, **new}
        lin.lin_block_norms(a["x"], a["y"], a["gate"], a["w_post"], a["w_pre"], h, n, **HOW)
        return (h.double() * ch + n.double() * cn).sum().item()

    loss()
    outs = dict(dx=_nan(ch), dy=_nan(ch), dgate=_nan(st["gate"]), dw_post=_nan(st["w_post"]),
                dw_pre=_nan(st["w_pre"]))
    lin.lin_block_norms_backward(h.clone(), *(st[k] for k in ("y", "gate", "w_post", "w_pre")), ch, cn,
                                 *outs.values(), **HOW)
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    for k in ("x", "y", "gate", "w_post", "w_pre"):
        d = torch.randn(st[k].shape, generator=g, device="cuda")
        step = 2.0 ** -7
        got = (outs["d" + k].double() * d).sum().item()
        want = (loss(**{k: st[k] + step * d}) - loss(**{k: st[k] - step * d})) / (2 * step)
        # the difference's own error: third derivatives times step^2 (some 2^-14
        # of the size of the gradient along d), and f32 results over the step
        size = (outs["d" + k].double().abs() * d.abs()).sum().item()
        assert abs(got - want) <= 2.0 ** -9 * size + 2.0 ** -10


def test_captured_and_on_another_stream():
    import torch
    st = _setup(513, 768, "bfloat16", "channel", True, seed=7)
    args = [st[k] for k in ("x", "y", "gate", "w_post", "w_pre", "dh", "dn")]
    outs = lambda: [_nan(st[k]) for k in ("x", "y", "gate", "w_post", "w_pre")]  # noqa: E731
    want, got = outs(), outs()
    lin.lin_block_norms_backward(*args, *want, **HOW)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        lin.lin_block_norms_backward(*args, *got, **HOW)
    for _ in range(2):
        for t in got:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    for t in got:
        t.fill_(float("nan"))
    torch.cuda.synchronize()
    lin.lin_block_norms_backward(*args, *got, **HOW, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_large_tensor():
    # offsets beyond 2^31 bytes and entries
    import torch
    m, w = 300000, 8192
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    x = torch.zeros(m, w, device="cuda", dtype=torch.float32)
    y = torch.zeros(m, w, device="cuda", dtype=torch.bfloat16)
    n = torch.empty_like(y)
    wt = torch.ones(w, device="cuda")
    x[-1], y[-1] = 3.0, 5.0
    lin.lin_block_norms(x, y, None, wt, wt, x, n, eps=0.25)
    _ok()
    b = 5 / 25.25 ** 0.5
    assert abs(x[-1].double() - 3 - b).max().item() < 1e-5
    assert abs(n[-1].double() - (3 + b) / ((3 + b) ** 2 + 0.25) ** 0.5).max().item() < 2.0 ** -8
    assert not n[:-1].any()
