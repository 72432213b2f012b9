"""lin_attention_scores and its gradient on the GPU against the fp64 oracle.

Bounds, with u the unit rounding of the tensors' type: as for attention the
result is rounded once (u of itself), P (dS) once before its product (u of the
sum of magnitudes), and the f32 parts stay below 2^-14 of those magnitudes.
The form of the scores adds: a capped score is cap (1 - 2 r) with r = 1 / (1 +
2^x) from approximations of a few units of 2^-23 of themselves, an error of at
most cap 2^-20 of the score and so of each P relative to itself; a bias is
rounded to 2^-24 of itself, twice (2^-22 of the largest one that counts).
"""

import numpy as np
import pytest

from oracle import train_oracle as to
from tests.gpu_util import require_gpu
from transformer_linear_layer_tcgen05_gb300 import lin

pytestmark = pytest.mark.gpu

UNIT = {"float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _cuts(lengths):
    return np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)


def _host(t):
    return None if t is None else t.double().cpu().numpy()


def _setup(dtype, lens, hq, hk, d, seed, gain=1.0):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = getattr(torch, dtype)
    nq, nk = sum(a for a, _ in lens), sum(b for _, b in lens)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    nan = lambda *s: torch.full(s, float("nan"), device="cuda", dtype=dt)  # noqa: E731
    kv, dkv, q, dq = rnd(nk, 2 * hk, d).to(dt), nan(nk, 2 * hk, d), (gain * rnd(nq, hq + 1, d)).to(dt), \
        nan(nq, hq + 1, d)
    t = dict(q=q[:, 1:], k=kv[:, :hk], v=kv[:, hk:], dq=dq[:, 1:], dk=dkv[:, :hk], dv=dkv[:, hk:],
             o=nan(nq, hq, d), do=rnd(nq, hq, d).to(dt))
    t["lse"] = torch.full((hq, nq), float("nan"), device="cuda")
    return t


def _ranges(kind, lens, seed):
    """first_key, end_key (numpy int32 over all queries)."""
    r = np.random.default_rng(seed)
    first, end = [], []
    for lq, lk in lens:
        at = np.arange(lq) + lk - lq
        f, e = np.zeros(lq, int), np.full(lq, lk)
        if kind == "docs":
            cuts = np.unique(np.concatenate([[0, lk], r.integers(0, lk + 1, 3)]))
            doc = np.clip(np.searchsorted(cuts, at, side="right") - 1, 0, max(len(cuts) - 2, 0))
            if len(cuts) > 1:
                f, e = cuts[doc], cuts[doc + 1]
        elif kind == "prefix":
            e = np.maximum(at + 1, lk // 3)
        elif kind == "window":
            f, e = at - 70, at + 40
        elif kind == "any":     # anywhere, also outside the sequence, also empty
            f = r.integers(-20, lk + 20, lq)
            e = f + r.integers(-10, lk + 1, lq)
        first.append(f)
        end.append(e)
    return np.concatenate(first).astype(np.int32), np.concatenate(end).astype(np.int32)


def _run(t, lens, causal, scale, form, stream=None):
    import torch
    cu = [torch.from_numpy(_cuts(x)).cuda() for x in zip(*lens)]
    how = dict(causal=causal, scale=scale, cu_q=cu[0], cu_k=cu[1], max_q=max(a for a, _ in lens),
               max_k=max(b for _, b in lens), **form)
    lin.lin_attention_scores(t["q"], t["k"], t["v"], t["o"], t["lse"], **how)
    lin.lin_attention_scores_backward(t["q"], t["k"], t["v"], t["o"], t["lse"], t["do"], t["dq"], t["dk"],
                                      t["dv"], **how)
    torch.cuda.synchronize()
    assert lin.lin_get_device_status() == lin.LIN_SUCCESS


def _check(t, lens, causal, scale, form, u):
    q, k, v, do = (_host(t[n]) for n in ("q", "k", "v", "do"))
    cut = dict(cu_q=_cuts([a for a, _ in lens]), cu_k=_cuts([b for _, b in lens]))
    slopes, cap = _host(form.get("slopes")), form.get("cap")
    spec = dict(cap=cap, slopes=slopes, first=_host(form.get("first_key")), end=_host(form.get("end_key")))
    o, lse, w = to.attention_scores(q, k, v, causal, scale, **spec, **cut)
    moved = (cap or 0) * 2.0 ** -20
    if slopes is not None:   # (a key further than 30 / slope below the row's best counts for nothing)
        far = max(max(a, b) for a, b in lens)
        moved += np.minimum(np.abs(slopes).max() * far, 40 + 2 * (cap or 40)) * 2.0 ** -22
    e = 2.0 ** -14 + moved
    got = _host(t["lse"])
    assert np.array_equal(np.isinf(got), np.isinf(lse))
    fin = np.isfinite(lse)
    np.testing.assert_allclose(got[fin], lse[fin], rtol=2e-6, atol=2e-6 + moved)
    assert np.all(np.abs(_host(t["o"]) - o) <= u * np.abs(o) + (u + e) * w + 1e-6)
    grads, sizes = to.attention_scores_backward(q, k, v, do, causal, scale, **spec, **cut)
    for name, g, size in zip(("dq", "dk", "dv"), grads, sizes):
        err = np.abs(_host(t[name]) - g)
        assert np.all(err <= u * np.abs(g) + (u + e) * size + 1e-6), name


def _form(kind, lens, hq, seed):
    import torch
    f = {}
    if "cap" in kind:
        f["cap"] = 5.0
    if "bias" in kind:
        f["slopes"] = 2.0 ** (-1.0 - 4.0 * torch.arange(hq, device="cuda") / hq)
    for mask in ("docs", "prefix", "window", "any"):
        if mask in kind:
            f["first_key"], f["end_key"] = (torch.from_numpy(x).cuda() for x in _ranges(mask, lens, seed))
    return f


# (lengths of queries and keys, query heads, key heads, dim)
SHAPES = [
    ([(1, 1)], 1, 1, 64),
    ([(1, 300)], 2, 1, 128),
    ([(127, 129), (128, 128), (129, 127)], 2, 2, 64),
    ([(256, 257), (0, 40), (257, 255), (3, 0), (5, 5)], 4, 2, 128),
    ([(300, 20), (1, 1), (2, 130)], 3, 3, 32),
    ([(70, 333), (400, 140)], 6, 2, 96),
    ([(131, 700), (1, 2)], 8, 1, 72),
]
KINDS = ["cap", "bias", "docs", "prefix", "window", "any", "cap bias", "cap any", "bias any", "cap bias docs"]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}x{s[1]}h{s[2]}d{s[3]}")
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("causal", [False, True])
def test_against_the_oracle(shape, kind, causal):
    lens, hq, hk, d = shape
    dtype = "float16" if (hq + len(kind)) % 2 else "bfloat16"
    t = _setup(dtype, lens, hq, hk, d, seed=hq * 100 + d, gain=3.0)
    form = _form(kind, lens, hq, seed=d)
    _run(t, lens, causal, d ** -0.5, form)
    _check(t, lens, causal, d ** -0.5, form, UNIT[dtype])


@pytest.mark.parametrize("kind", ["cap bias", "cap any", "docs", "bias window"])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_long_sides_in_parts(kind, dtype):
    # few tiles on one side: the other one is cut into parts
    for lens in ([(64, 2600)], [(1500, 40)]):
        t = _setup(dtype, lens, 2, 1, 64, seed=3)
        form = _form(kind, lens, 2, seed=4)
        _run(t, lens, False, 0.125, form)
        _check(t, lens, False, 0.125, form, UNIT[dtype])


@pytest.mark.parametrize("kind", ["cap bias docs", "any", "cap window", "bias prefix"])
@pytest.mark.parametrize("d, heads", [(64, (36, 18)), (128, (33, 11)), (96, (24, 24))])
def test_many_tiles(kind, d, heads):
    # more tiles of queries than SMs: two of them to a CTA
    lens = [(700, 700), (40, 300)]
    t = _setup("bfloat16", lens, *heads, d, seed=15, gain=2.0)
    form = _form(kind, lens, heads[0], seed=16)
    _run(t, lens, "window" in kind, 0.1, form)
    _check(t, lens, "window" in kind, 0.1, form, UNIT["bfloat16"])


@pytest.mark.parametrize("scale", [0.02, 0.5, 8.0])
def test_scores_far_below_and_above_the_cap(scale):
    lens = [(150, 200)]
    t = _setup("float16", lens, 2, 2, 64, seed=5)
    form = dict(cap=12.0)
    _run(t, lens, True, scale, form)
    _check(t, lens, True, scale, form, UNIT["float16"])


def test_negative_slopes_and_none():
    import torch
    lens = [(90, 170)]
    t = _setup("bfloat16", lens, 4, 2, 64, seed=6)
    form = dict(slopes=torch.tensor([-0.03, 0.0, 0.5, -0.01], device="cuda"))
    _run(t, lens, False, 0.2, form)
    _check(t, lens, False, 0.2, form, UNIT["bfloat16"])


@pytest.mark.parametrize("d", [64, 128])
def test_without_a_form_and_with_the_causal_mask_as_ranges(d):
    import torch
    lens = [(200, 333), (400, 140), (7, 900)]
    a, b, c = (_setup("bfloat16", lens, 4, 2, d, seed=7) for _ in range(3))
    cu = [torch.from_numpy(_cuts(x)).cuda() for x in zip(*lens)]
    how = dict(cu_q=cu[0], cu_k=cu[1], max_q=400, max_k=900, causal=True)
    lin.lin_attention(a["q"], a["k"], a["v"], a["o"], a["lse"], **how)
    lin.lin_attention_backward(*(a[k] for k in ("q", "k", "v", "o", "lse", "do", "dq", "dk", "dv")), **how)
    _run(b, lens, True, None, {})
    end = np.concatenate([np.arange(x) + y - x + 1 for x, y in lens]).astype(np.int32)
    _run(c, lens, False, None, dict(end_key=torch.from_numpy(end).cuda()))
    for k in ("o", "lse", "dq", "dk", "dv"):
        assert torch.equal(a[k], b[k]) and torch.equal(a[k], c[k]), k


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads", [(2, 2), (4, 1)])
def test_rows_without_keys_give_nothing_whatever_they_hold(d, heads):
    import torch
    lens = [(300, 300), (50, 80)]
    nan, inf = float("nan"), float("inf")
    t = _setup("float16", lens, *heads, d, seed=8)
    first, end = _ranges("docs", lens, 2)
    none = np.concatenate([np.arange(0, 5), np.arange(100, 233, 7), [299], np.arange(310, 315)])
    end[none] = first[none]
    form = dict(cap=6.0, first_key=torch.from_numpy(first).cuda(), end_key=torch.from_numpy(end).cuda())
    _run(t, lens, True, 0.1, form)
    want = {k: t[k].clone() for k in ("o", "lse", "dq", "dk", "dv")}
    rows = torch.from_numpy(none).cuda()
    assert not want["o"][rows].any() and not want["dq"][rows].any()
    assert torch.isinf(want["lse"][:, rows]).all()
    t["q"][rows[::2]], t["do"][rows[::3]], t["q"][rows[1]] = nan, inf, -inf
    _run(t, lens, True, 0.1, form)
    for k in want:
        assert torch.equal(t[k], want[k]), k
    # (one entry of the last head alone)
    t["q"][rows], t["do"][rows] = 0, 0
    t["do"][rows[7], -1, d - 1] = nan
    _run(t, lens, True, 0.1, form)
    for k in want:
        assert torch.equal(t[k], want[k]), k


def test_rows_without_keys_that_hold_the_largest_numbers():
    # (finite ones, whose products are not)
    import torch
    lens = [(300, 300)]
    t = _setup("bfloat16", lens, 2, 1, 64, seed=13)
    t["k"][:], t["v"][:] = 100 * t["k"], 100 * t["v"]
    end = np.arange(1, 301).astype(np.int32)
    none = np.arange(3, 300, 17)
    end[none] = 0
    form = dict(end_key=torch.from_numpy(end).cuda())
    _run(t, lens, True, 0.1, form)
    want = {k: t[k].clone() for k in ("o", "lse", "dq", "dk", "dv")}
    assert all(torch.isfinite(t[k]).all() for k in ("o", "dq", "dk", "dv"))
    rows = torch.from_numpy(none).cuda()
    for q, do in ((3e38, 1.0), (1.0, -3e38), (1e20, 1e20)):
        t["q"][rows], t["do"][rows] = q, do
        _run(t, lens, True, 0.1, form)
        for k in want:
            assert torch.equal(t[k], want[k]), (k, q, do)


@pytest.mark.parametrize("cap", [1e-3, 300.0, 4096.0])
def test_small_and_large_caps(cap):
    lens = [(140, 260)]
    t = _setup("float16", lens, 2, 2, 64, seed=14, gain=2.0)
    form = dict(cap=cap)
    _run(t, lens, True, 0.2, form)
    _check(t, lens, True, 0.2, form, UNIT["float16"])


@pytest.mark.parametrize("kind", ["cap", "bias", "cap bias", "ranges"])
def test_pairs_that_the_mask_parts_and_whose_products_are_not_finite(kind):
    # two documents in a tile: large V and small dO in one, the other way in the
    # other, so that dO V is infinite between them, and finite in each
    import torch
    lens = [(100, 100)]
    first = torch.tensor([0] * 40 + [40] * 60, dtype=torch.int32, device="cuda")
    end = torch.tensor([40] * 40 + [100] * 60, dtype=torch.int32, device="cuda")
    form = dict(_form(kind, lens, 2, seed=17), first_key=first, end_key=end)
    for causal in (False, True):
        t = _setup("bfloat16", lens, 2, 1, 64, seed=17)
        _run(t, lens, causal, 0.2, form)
        want = {k: t[k].clone() for k in ("o", "dq", "dk", "dv")}
        t["v"][:40] *= 2.0 ** 75
        t["do"][:40] *= 2.0 ** -75
        t["v"][40:] *= 2.0 ** -60
        t["do"][40:] *= 2.0 ** 60
        _run(t, lens, causal, 0.2, form)
        # (powers of two: dO V, dS, dQ and dK of each document are what they were,
        # but that dK's tile scales by its largest dO, 2^60 of the second document:
        # in bfloat16, whose exponents are float32's, the first one's dS and sums
        # of 2^-135 or more of them would have to stay above 2^-126)
        for k in ("dq", "dk"):
            assert torch.isfinite(t[k]).all(), k
            assert torch.equal(t[k][40:], want[k][40:]), k
        assert torch.equal(t["dq"], want["dq"])
        assert torch.equal(t["o"][:40] * 2.0 ** -75, want["o"][:40])
        assert torch.equal(t["dv"][40:] * 2.0 ** -60, want["dv"][40:])


@pytest.mark.parametrize("d, heads", [(64, (2, 1)), (64, (36, 18)), (128, (33, 11))])
@pytest.mark.parametrize("kind", ["cap", "cap bias", "bias"])
def test_what_the_mask_hides_does_not_show(kind, d, heads):
    # one document's queries, keys and values changed: the others' results are
    # the same bits (scores of a cap are computed four at a time)
    import torch
    lens = [(390, 390)]
    at = torch.arange(390, dtype=torch.int32, device="cuda")
    cuts = torch.tensor([0, 61, 130, 199, 390], dtype=torch.int32, device="cuda")
    doc = torch.searchsorted(cuts, at, right=True)
    form = dict(_form(kind, lens, heads[0], seed=18), first_key=cuts[doc - 1].contiguous(),
                end_key=cuts[doc].contiguous())
    t = _setup("float16", lens, *heads, d, seed=18, gain=3.0)
    rest = torch.cat([at[:130], at[199:]]).long()
    want = None
    for gain in (1.0, 7.0, 0.0):
        for name in ("q", "k", "v"):
            t[name][130:199] = gain * t[name][130:199].flip(0)
        _run(t, lens, True, d ** -0.5, form)
        got = {k: t[k][rest].clone() for k in ("o", "dq", "dk", "dv")}
        got["lse"] = t["lse"][:, rest].clone()
        want = want or got
        for k in want:
            assert torch.equal(got[k], want[k]), (k, gain)


def test_no_row_sees_anything():
    import torch
    for lens in ([(200, 300)], [(3, 2000)]):
        t = _setup("bfloat16", lens, 2, 1, 128, seed=9)
        zero = torch.zeros(lens[0][0], dtype=torch.int32, device="cuda")
        _run(t, lens, False, None, dict(end_key=zero))
        assert not t["o"].any() and torch.isinf(t["lse"]).all()
        assert not t["dq"].any() and not t["dk"].any() and not t["dv"].any()


def test_rows_outside_every_sequence_stay():
    import torch
    t = _setup("float16", [(300, 300)], 2, 2, 64, seed=10)
    first, end = (torch.from_numpy(x).cuda() for x in _ranges("any", [(300, 300)], 3))
    cu = torch.tensor([20, 150, 260], dtype=torch.int32, device="cuda")
    how = dict(cu_q=cu, cu_k=cu, max_q=130, max_k=130, cap=9.0, first_key=first, end_key=end)
    lin.lin_attention_scores(t["q"], t["k"], t["v"], t["o"], t["lse"], **how)
    lin.lin_attention_scores_backward(*(t[k] for k in ("q", "k", "v", "o", "lse", "do", "dq", "dk", "dv")),
                                      **how)
    torch.cuda.synchronize()
    assert lin.lin_get_device_status() == lin.LIN_SUCCESS
    for k in ("o", "dq", "dk", "dv"):
        assert torch.isnan(t[k][:20]).all() and torch.isnan(t[k][260:]).all()
        assert torch.isfinite(t[k][20:260]).all()


def test_captured_and_two_streams():
    import torch
    lens = [(700, 700), (90, 90)]
    form = _form("cap bias docs", lens, 4, seed=11)
    want, got, other = (_setup("bfloat16", lens, 4, 2, 64, seed=11) for _ in range(3))
    _run(want, lens, True, None, form)
    cu = [torch.from_numpy(_cuts(x)).cuda() for x in zip(*lens)]
    how = dict(cu_q=cu[0], cu_k=cu[1], max_q=700, max_k=700, **form)

    def both(t, stream=None):
        lin.lin_attention_scores(t["q"], t["k"], t["v"], t["o"], t["lse"], **how, stream=stream)
        lin.lin_attention_scores_backward(*(t[k] for k in ("q", "k", "v", "o", "lse", "do", "dq", "dk", "dv")),
                                          **how, stream=stream)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(got)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        graph.replay()
        both(other, side)
    torch.cuda.synchronize()
    for k in ("o", "lse", "dq", "dk", "dv"):
        assert torch.equal(got[k], want[k]) and torch.equal(other[k], want[k])


def test_gradient_is_the_difference_of_the_forward():
    import torch
    lens = [(96, 130)]
    t = _setup("float16", lens, 2, 1, 32, seed=12, gain=2.0)
    form = _form("cap bias window", lens, 2, seed=12)
    _run(t, lens, False, 0.3, form)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    spec = dict(cap=form["cap"], slopes=_host(form["slopes"]), first=_host(form["first_key"]),
                end=_host(form["end_key"]))
    args = {k: _host(t[k]) for k in ("q", "k", "v")}
    do = _host(t["do"])

    def loss(**new):
        a = {**args, **new}
        return (to.attention_scores(a["q"], a["k"], a["v"], False, 0.3, **spec)[0] * do).sum()

    for k in ("q", "k", "v"):
        d = torch.randn(t[k].shape, generator=g, device="cuda").double().cpu().numpy()
        got = (_host(t["d" + k]) * d).sum()
        want = (loss(**{k: args[k] + 1e-5 * d}) - loss(**{k: args[k] - 1e-5 * d})) / 2e-5
        # each entry is off by some 2^-10 of its terms (test_against_the_oracle)
        assert abs(got - want) <= 2.0 ** -9 * (np.abs(_host(t["d" + k])) * np.abs(d)).sum() * 2
