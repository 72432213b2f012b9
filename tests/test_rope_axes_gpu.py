"""lin_qk_norm_rope_axes and its gradient on the GPU against the fp64 oracle of
the rotation, whose tables are gathered pair by pair. Bounds as in
test_qk_norm_rope_gpu.py: the 16-bit heads are rounded once, the rest is a
handful of float32 roundings, taken as 2^-20 of the terms' magnitudes."""

import numpy as np
import pytest

from oracle import step_oracle as so
from tests.gpu_util import require_gpu
from transformer_linear_layer_tcgen05_gb300 import lin

pytestmark = pytest.mark.gpu

UNIT = {"float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}
E = 2.0 ** -20
ROWS = 50


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _host(t):
    return t.double().cpu().numpy()


def _setup(t, hq, hk, d, rot, axes, layout, dtype, seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    st = dict(x=rnd(t, (hq + 2 * hk) * d), wq=1 + 0.3 * rnd(d), wk=1 + 0.3 * rnd(d))
    ang = 3 * rnd(ROWS, rot // 2)
    st["cos"], st["sin"] = ang.cos().contiguous(), ang.sin().contiguous()
    # (some positions outside the table: held to it)
    st["pos"] = torch.randint(-3, ROWS + 3, (axes, t), generator=g, device="cuda", dtype=torch.int32)
    i = torch.arange(rot // 2, device="cuda", dtype=torch.int32)
    st["axis"] = {"turns": i % axes, "sections": i * axes // (rot // 2),
                  "uneven": (i + 3) * axes // (rot // 2 + 3),
                  "outside": i % (axes + 2) - 1}[layout].int().contiguous()
    heads = torch.full((t, hq + 2 * hk, d), float("nan"), device="cuda", dtype=getattr(torch, dtype))
    grads = rnd(t, hq + 2 * hk, d).to(heads.dtype)
    cut = lambda y: (y[:, :hq], y[:, hq:hq + hk], y[:, hq + hk:])  # noqa: E731
    st["out"], st["dout"] = cut(heads), cut(grads)
    return st


def _tables(st):
    """Each token's own table row, gathered by its pairs' axes."""
    pos = np.clip(st["pos"].cpu().numpy(), 0, ROWS - 1)
    axis = np.clip(st["axis"].cpu().numpy(), 0, len(pos) - 1)
    rows = pos[axis].T                      # [tokens, pairs]
    pair = np.arange(len(axis))
    return _host(st["cos"])[rows, pair], _host(st["sin"])[rows, pair], np.arange(rows.shape[0])


CASES = [(1, 1, 1, 64, 64, 3, "sections"), (37, 4, 2, 32, 16, 3, "turns"), (129, 12, 12, 64, 64, 2, "turns"),
         (33, 7, 1, 96, 40, 3, "uneven"), (70, 8, 2, 128, 128, 4, "sections"), (70, 8, 2, 128, 128, 3, "turns"),
         (21, 3, 2, 256, 256, 3, "uneven"), (11, 2, 1, 200, 64, 1, "turns"), (50, 2, 2, 64, 48, 3, "outside"),
         (1300, 12, 4, 128, 96, 3, "turns"), (1300, 12, 4, 128, 128, 4, "outside")]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_forward_and_backward(case, interleaved, dtype):
    import torch
    t, hq, hk, d = case[:4]
    st = _setup(*case, dtype, seed=t + d)
    how = dict(eps=1e-5, interleaved=interleaved)
    tables = (st["cos"], st["sin"], st["pos"], st["axis"])
    lin.lin_qk_norm_rope_axes(st["x"], st["wq"], st["wk"], *tables, *st["out"], **how)
    torch.cuda.synchronize()
    assert lin.lin_get_device_status() == lin.LIN_SUCCESS
    cos, sin, rows = _tables(st)
    x, wq, wk = _host(st["x"]), _host(st["wq"]), _host(st["wk"])
    want = so.qk_norm_rope(x, wq, wk, cos, sin, rows, hq, hk, 1e-5, interleaved)
    for got, w in zip(st["out"], want):
        size = np.abs(w).max(axis=-1, keepdims=True) * 2
        assert np.all(np.abs(_host(got) - w) <= UNIT[dtype] * np.abs(w) + E * size + 2.0 ** -25)
    dx = torch.full_like(st["x"], float("nan"))
    dwq, dwk = (torch.full((d,), float("nan"), device="cuda") for _ in range(2))
    lin.lin_qk_norm_rope_axes_backward(st["x"], st["wq"], st["wk"], *tables, *st["dout"], dx, dwq, dwk,
                                       **how)
    torch.cuda.synchronize()
    assert lin.lin_get_device_status() == lin.LIN_SUCCESS
    dy = [_host(y) for y in st["dout"]]
    want = so.qk_norm_rope_backward(x, wq, wk, cos, sin, rows, *dy, 1e-5, interleaved)
    xh = np.abs(x.reshape(t, -1, d))
    r = 1 / np.sqrt((xh ** 2).mean(-1, keepdims=True) + 1e-5)
    big = np.concatenate([np.abs(y).max(-1, keepdims=True) * 2 for y in dy], axis=1)
    w = max(np.abs(wq).max(), np.abs(wk).max())
    size = r * big * w * (1 + xh * r * (xh * r).mean(-1, keepdims=True)) + big
    assert np.all(np.abs(_host(dx) - want[0]).reshape(t, -1, d) <= E * size)
    terms = big * xh * r
    for got, ref, part in ((dwq, want[1], terms[:, :hq]), (dwk, want[2], terms[:, hq:hq + hk])):
        assert np.all(np.abs(_host(got) - ref) <= E * part.sum(axis=(0, 1)))


@pytest.mark.parametrize("interleaved", [False, True])
def test_one_position_is_the_plain_form(interleaved):
    import torch
    st = _setup(65, 6, 2, 128, 96, 3, "turns", "bfloat16", seed=8)
    one = st["pos"][1].clamp(0, ROWS - 1).contiguous()
    same = one.expand(3, -1).contiguous()
    how = dict(eps=1e-5, interleaved=interleaved)
    want = [t.clone() for t in st["out"]]
    lin.lin_qk_norm_rope(st["x"], st["wq"], st["wk"], st["cos"], st["sin"], one, *want, **how)
    lin.lin_qk_norm_rope_axes(st["x"], st["wq"], st["wk"], st["cos"], st["sin"], same, st["axis"],
                              *st["out"], **how)
    assert all(torch.equal(a, b) for a, b in zip(want, st["out"]))


def test_large_calls_gather_the_angles():
    # (whose results the cases of 1300 tokens above compare)
    for t, kernels in ((500, 1), (1300, 2)):
        st = _setup(t, 12, 4, 128, 96, 3, "turns", "float16", seed=12)
        lin.lin_qk_norm_rope_axes(st["x"], st["wq"], st["wk"], st["cos"], st["sin"], st["pos"], st["axis"],
                                  *st["out"])
        got, room = lin.lin_last_launch_info()
        assert got == kernels and room == (t * 96 * 4 if kernels == 2 else 0)


def test_no_tokens_and_no_rotation():
    import torch
    st = _setup(0, 2, 1, 64, 64, 3, "turns", "float16", seed=9)
    lin.lin_qk_norm_rope_axes(st["x"], st["wq"], st["wk"], st["cos"], st["sin"], st["pos"], st["axis"],
                              *st["out"])
    st = _setup(9, 2, 1, 64, 64, 3, "turns", "float16", seed=9)
    want = [t.clone() for t in st["out"]]
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    lin.lin_qk_norm_rope_axes(st["x"], st["wq"], st["wk"], None, None, st["pos"], none, *st["out"])
    lin.lin_qk_norm_rope(st["x"], st["wq"], st["wk"], None, None, None, *want)
    torch.cuda.synchronize()
    assert lin.lin_get_device_status() == lin.LIN_SUCCESS
    assert all(torch.equal(a, b) for a, b in zip(want, st["out"]))


def test_captured():
    import torch
    st = _setup(200, 4, 2, 64, 64, 3, "turns", "float16", seed=10)
    args = (st["x"], st["wq"], st["wk"], st["cos"], st["sin"], st["pos"], st["axis"])
    new = lambda: [torch.full_like(t, float("nan")) for t in (st["x"], st["wq"], st["wk"])]  # noqa: E731
    want, got = new(), new()
    lin.lin_qk_norm_rope_axes_backward(*args, *st["dout"], *want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lin.lin_qk_norm_rope_axes_backward(*args, *st["dout"], *got)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
