"""lin_adamw on the GPU against the fp64 oracle.

Bounds: the states in float32 are those of the formula with one rounding to an
operation, bit for bit, and so are the codes and scales of 8-bit states. The
weights come from them by a root, a division and two sums (and, with the step
on the device, float32 corrections): fewer than 2^4 roundings of 2^-24 on the
weight and on the terms of its change, taken as 2^-20 of their magnitudes. The
change's terms are lr decay |p| and lr / (1 - b1^t) / denominator times |b1 m|
and |(1 - b1) g|: m is their sum, rounded with an error of the size of its
larger term (2^-24 of it for each product and the sum, 2^-25 for each factor's
own rounding to float32), however small the sum of the two comes out.
"""

import numpy as np
import pytest

from oracle import train_oracle as to
from tests.gpu_util import require_gpu
from transformer_linear_layer_tcgen05_gb300 import lin

pytestmark = pytest.mark.gpu

SIZES = [1, 7, 8, 255, 256, 257, 1000, 0, 4099, 70000]
HOW = dict(lr=3e-3, betas=(0.9, 0.99), eps=1e-6, weight_decay=0.2)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _np(t):
    return t.detach().cpu().numpy()


def _at(n, off, dtype, width=512):
    """n entries of a tensor that begins `off` entries behind an allocation's
    start, fenced by NaN (or 0xff)."""
    import torch
    size = torch.empty(0, dtype=dtype).element_size()
    buf = torch.full(((n + 64) * size,), 255, dtype=torch.uint8, device="cuda").view(dtype)
    return buf, buf[off:off + n]


def _tensors(sizes, bits, off=0, w16=True, seed=0, zero=False):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rnd = lambda n: torch.randn(n, generator=g, device="cuda")  # noqa: E731
    st = {k: [] for k in ("p", "g", "m", "v", "ms", "vs", "w16", "fences")}
    for n in sizes:
        def put(name, x):
            buf, t = _at(n if name not in ("ms", "vs") else len(x), off, x.dtype)
            t.copy_(x)
            st[name].append(t)
            st["fences"].append((buf, t, buf.clone(), off))
        size = torch.exp(2 * rnd(n))
        put("p", rnd(n))
        put("g", size * rnd(n))
        m, r = (0 * size, 0 * size) if zero else (0.3 * size * rnd(n), size * (rnd(n).abs() + 0.1))
        if bits == 32:
            put("m", m)
            put("v", r * r)
        else:
            for a, b, x, least in (("m", "ms", m, False), ("v", "vs", r, True)):
                c, s = to.coded(_np(x), least)
                put(a, torch.from_numpy(c).cuda().view(torch.float8_e4m3fn))
                put(b, torch.from_numpy(s).cuda())
        if w16:
            put("w16", torch.zeros(n, device="cuda", dtype=torch.float16))
        else:
            st["w16"].append(None)
    return st


def _states(st, i, bits):
    """m and v of tensor i before the step, float32."""
    if bits == 32:
        return _np(st["m"][i]), _np(st["v"][i])
    import torch
    got = []
    for a, b in (("m", "ms"), ("v", "vs")):
        x = to.e4m3_values(_np(st[a][i].view(torch.uint8))).astype(np.float32)
        got.append(x * np.repeat(_np(st[b][i]), 256)[:x.size])
    return got[0], got[1] * got[1]


def _call(st, bits, **how):
    scales = dict(m_scale=st["ms"], v_scale=st["vs"]) if bits == 8 else {}
    w16 = st["w16"] if any(t is not None for t in st["w16"]) else None
    lin.lin_adamw(st["p"], st["g"], st["m"], st["v"], **scales, w16=w16, **{**HOW, **how})


def _check(st, bits, step, how=None, lr=None, scale=None, rel=2.0 ** -20):
    import torch
    before = [(_np(st["p"][i]).copy(), _np(st["g"][i]), *(x.copy() for x in _states(st, i, bits)))
              for i in range(len(st["p"]))]
    _call(st, bits, **(how or dict(step=step)))
    torch.cuda.synchronize()
    assert lin.lin_get_device_status() == lin.LIN_SUCCESS
    lr = HOW["lr"] if lr is None else lr
    for i, (p, g, m, v) in enumerate(before):
        wm, wv, wr = to.adamw_states_f32(g, m, v, *HOW["betas"], scale)
        if bits == 32:
            assert np.array_equal(_np(st["m"][i]), wm, equal_nan=True)
            assert np.array_equal(_np(st["v"][i]), wv, equal_nan=True)
        else:
            for a, b, x, least in (("m", "ms", wm, False), ("v", "vs", wr, True)):
                c, s = to.coded(x, least)
                got = _np(st[a][i].view(torch.uint8))
                # (the sign of a zero or of a NaN is not looked at)
                same = (got == c) | ((got & 127 == c & 127) & ((c & 127 == 0) | (c & 127 == 127)))
                assert np.all(same) and np.array_equal(_np(st[b][i]), s)
        want, _, _ = to.adamw(p, g, m, v, step, lr, *HOW["betas"], HOW["eps"], HOW["weight_decay"],
                              1.0 if scale is None else float(np.float32(scale)))
        got = _np(st["p"][i]).astype(np.float64)
        fine = np.isfinite(want)
        assert np.array_equal(fine, np.isfinite(got))
        b1, b2 = HOW["betas"]
        x = np.abs(g.astype(np.float64)) * (1.0 if scale is None else scale)
        terms = (b1 * np.abs(m.astype(np.float64)) + (1 - b1) * x) / (1 - b1 ** step)
        root = np.sqrt((b2 * v.astype(np.float64) + (1 - b2) * x * x) / (1 - b2 ** step))
        size = np.abs(p) * (1 + lr * HOW["weight_decay"]) + lr * terms / (root + HOW["eps"])
        assert np.all(np.abs(got - want)[fine] <= rel * size[fine])
        if st["w16"][i] is not None:
            assert torch.allclose(st["w16"][i], st["p"][i].half(), rtol=0, atol=0, equal_nan=True)
    # nothing beside the tensors is written
    for buf, t, was, off in st["fences"]:
        was[off:off + t.numel()].copy_(t)
        assert torch.equal(buf.view(torch.uint8), was.view(torch.uint8))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("w16", [False, True])
@pytest.mark.parametrize("off", [0, 1, 8])
def test_steps(bits, w16, off):
    # three steps on: each from what the one before left
    st = _tensors(SIZES, bits, off, w16, seed=off)
    for step in (1, 2, 50000):
        _check(st, bits, step)


@pytest.mark.parametrize("bits", [32, 8])
def test_from_zero_states(bits):
    st = _tensors([300, 64], bits, zero=True, seed=3)
    for step in (1, 2):
        _check(st, bits, step)


@pytest.mark.parametrize("bits", [32, 8])
def test_zero_gradients(bits):
    # (the root of v must not fall to zero before m does)
    import torch
    st = _tensors([520], bits, seed=4)
    st["g"][0].zero_()
    st["g"][0][::3] = 1e-9
    for step in (10, 11, 12):
        _check(st, bits, step)
    assert torch.isfinite(st["p"][0]).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_numbers_that_are_none_stay_where_they_are(bits):
    import torch
    st = _tensors([700], bits, seed=5)
    st["g"][0][3], st["g"][0][300], st["g"][0][301] = float("nan"), float("inf"), float("-inf")
    _check(st, bits, 4)
    bad = ~torch.isfinite(st["p"][0])
    assert bad.nonzero().flatten().tolist() in ([3, 300, 301], [3])
    _check(st, bits, 5)


@pytest.mark.parametrize("bits", [32, 8])
def test_values_on_the_device(bits):
    import torch
    st = _tensors([1000, 513], bits, seed=6)
    step = torch.tensor([7], dtype=torch.int32, device="cuda")
    lr = torch.tensor([5e-3], device="cuda")
    scale = torch.tensor([0.37], device="cuda")
    how = dict(step=step, lr=lr, grad_scale=scale)
    _check(st, bits, 7, how, lr=float(np.float32(5e-3)), scale=0.37)
    step.fill_(1)
    _check(st, bits, 1, dict(step=step), rel=2.0 ** -19)
    _check(st, bits, 3, dict(step=3, lr=lr), lr=float(np.float32(5e-3)))


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_with_a_schedule(bits):
    import torch
    sizes = [2000, 77, 256]
    st, other = _tensors(sizes, bits, seed=7), _tensors(sizes, bits, seed=7)
    step = torch.ones(1, dtype=torch.int32, device="cuda")
    lr = torch.full((1,), 1e-2, device="cuda")
    saved = [[None if t is None else t.clone() for t in st[k]] for k in ("p", "m", "v", "ms", "vs")]
    _call(st, bits, step=step, lr=lr)   # (the library is loaded before the capture)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _call(st, bits, step=step, lr=lr)
    for k, ts in zip(("p", "m", "v", "ms", "vs"), saved):
        for t, s in zip(st[k], ts):
            t.copy_(s)
    for i in range(3):
        step.fill_(i + 1)
        lr.fill_(1e-2 / (i + 1))
        graph.replay()
        _call(other, bits, step=step, lr=lr)
    torch.cuda.synchronize()
    for k in ("p", "m", "v", "ms", "vs", "w16"):
        for a, b in zip(st[k], other[k]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("count", [16, 17, 129, 1000])
def test_many_tensors(bits, count):
    # the launches' list sizes, and several launches
    st = _tensors([(i * 37) % 600 for i in range(count)], bits, seed=8)
    _check(st, bits, 9)
    assert lin.lin_last_launch_info()[0] == -(-sum(1 for i in range(count) if (i * 37) % 600) // 384)


def test_blocks_shared_out_over_long_and_short_tensors():
    st = _tensors([5, 3_000_001, 300, 2_000_000, 1], 8, seed=10)
    _check(st, 8, 2)


def test_a_large_tensor():
    # more than 2^31 entries, 8-bit states
    import torch
    n = (1 << 31) + 777
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    p, g = torch.ones(n, device="cuda"), torch.zeros(n, device="cuda")
    m, v = (torch.zeros(n, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn) for _ in range(2))
    ms, vs = (torch.zeros(-(-n // 256), device="cuda") for _ in range(2))
    g[-1], g[5] = 2.0, -3.0
    lin.lin_adamw([p], [g], [m], [v], [ms], [vs], step=1, lr=0.125, eps=0.0, weight_decay=0.0)
    torch.cuda.synchronize()
    assert lin.lin_get_device_status() == lin.LIN_SUCCESS
    # (0 / 0 where there is no gradient: the step with eps = 0)
    assert abs(p[-1].item() - 0.875) < 1e-6 and abs(p[5].item() - 1.125) < 1e-6
    assert abs(ms[-1].item() * 448 - 0.2) < 1e-6 and torch.isnan(p[n // 2])
