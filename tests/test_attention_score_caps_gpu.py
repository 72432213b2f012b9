"""Capped scores on every way that the forward kernel of two tiles to a CTA has
for them (polynomials of three and of five terms, and the exponential), at caps
over the whole range, against the fp64 oracle with the bounds of
test_attention_scores_gpu.py. Here scale reaches cap / 8 (6) where it is 0.1
there, so that one term of dK counts that the 1e-6 of those bounds holds there: dS
is a binary16 number times a power of two by which the largest row of dO that the
tile meets counts as having a norm of 2^4 to 2^5. Its smallest step is 2^-24, so
dS is off by up to 2^-25 2^-4 of that norm and dK by scale times that times the
sum of the |Q| that the key meets (dQ: by the row's own norm, and the |K|).
"""

import numpy as np
import pytest

from oracle import train_oracle as to
from tests.gpu_util import require_gpu
from tests.test_attention_score_tiles_gpu import _some, _two_tiles
from tests.test_attention_scores_gpu import UNIT, _form, _host, _run, _setup

pytestmark = pytest.mark.gpu

# Sizes of the scores beside the cap, of a row's largest in a tile: nothing,
# below 3/10, between that and 3/4, beyond
SIZES = [0.0, 0.05, 0.16, 1.0, 0.1, 0.2, 4.0]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _sized(t, cap, scale):
    """Rows of Q of which each has scores of the next of the sizes."""
    import torch
    d = t["q"].shape[2]
    size = torch.tensor(SIZES, device="cuda")[torch.arange(len(t["q"]), device="cuda") * 5 // 4 % len(SIZES)]
    # (k's entries are normal, so are q's: q k is some sqrt(d))
    t["q"].copy_(t["q"].float() * size[:, None, None] * (cap / scale / d ** 0.5))


def _check(t, causal, scale, form, u):
    """test_attention_scores_gpu._check for one sequence, with the steps of dS."""
    q, k, v, do = (_host(t[n]) for n in ("q", "k", "v", "do"))
    cap, slopes = form.get("cap"), _host(form.get("slopes"))
    spec = dict(cap=cap, slopes=slopes, first=_host(form.get("first_key")), end=_host(form.get("end_key")))
    o, lse, w = to.attention_scores(q, k, v, causal, scale, **spec)
    moved = (cap or 0) * 2.0 ** -20
    if slopes is not None:
        moved += np.minimum(np.abs(slopes).max() * len(k), 40 + 2 * (cap or 40)) * 2.0 ** -22
    e = 2.0 ** -14 + moved
    got = _host(t["lse"])
    assert np.array_equal(np.isinf(got), np.isinf(lse))
    fin = np.isfinite(lse)
    np.testing.assert_allclose(got[fin], lse[fin], rtol=2e-6, atol=2e-6 + moved)
    assert np.all(np.abs(_host(t["o"]) - o) <= u * np.abs(o) + (u + e) * w + 1e-6)
    grads, sizes = to.attention_scores_backward(q, k, v, do, causal, scale, **spec)
    step = 0.0
    if u == UNIT["float16"]:
        group = q.shape[1] // k.shape[1]
        norm = np.sqrt((do * do).sum(-1, keepdims=True))            # [tokens, heads, 1]
        step = 2.0 ** -29 * scale
        of_k = np.repeat(np.abs(k).sum(0), group, 0)[None] * norm   # (all keys, more than it meets)
        of_q = (np.abs(q).sum(0).reshape(k.shape[1], group, -1).sum(1) * norm.max())[None]
    for name, g, size in zip(("dq", "dk", "dv"), grads, sizes):
        err = np.abs(_host(t[name]) - g)
        steps = 0.0 if not step or name == "dv" else step * (of_k if name == "dq" else of_q)
        assert np.all(err <= u * np.abs(g) + (u + e) * size + steps + 1e-6), name


@pytest.mark.parametrize("kind", ["cap", "cap docs", "cap bias window"])
@pytest.mark.parametrize("cap", [1e-3, 15.0, 30.0, 50.0])
@pytest.mark.parametrize("d, heads", [(64, (40, 40)), (96, (60, 30)), (128, (40, 40))])
def test_scores_on_both_sides_of_where_a_way_ends(d, heads, cap, kind):
    lens = [(390, 390)]
    _two_tiles(lens, *heads)
    for dtype in ("float16", "bfloat16"):
        t = _setup(dtype, lens, *heads, d, seed=30 + d)
        # (a scale with which Q of either type holds these scores)
        scale = cap / 8
        _sized(t, cap, scale)
        form = dict(_form(kind, lens, heads[0], seed=31), cap=cap)
        _run(t, lens, "bias" not in kind, scale, form)
        part, how = _some(t, form, [0, heads[1] // 2, heads[1] - 1])
        _check(part, "bias" not in kind, scale, how, UNIT[dtype])
        assert all(np.isfinite(_host(t[k])).all() for k in ("o", "dq", "dk", "dv"))


@pytest.mark.parametrize("cap, scale", [(2.0 ** -20, 1.0), (2.0 ** -18, 1.0), (1.0, 40000.0),
                                        (2.0 ** -20, 4096.0), (2.0 ** -16, 2.0 ** 30)])
@pytest.mark.parametrize("causal", [False, True])
def test_caps_far_below_the_scale(cap, scale, causal):
    # (the polynomials' coefficients grow with the powers of scale / cap)
    lens, heads = [(300, 300)], (54, 54)
    _two_tiles(lens, *heads)
    t = _setup("bfloat16", lens, *heads, 64, seed=33)
    _sized(t, cap, scale)
    _run(t, lens, causal, scale, dict(cap=cap))
    for _ in range(2):
        part, form = _some(t, dict(cap=cap), [0, 30, 53])
        _check(part, causal, scale, form, UNIT["bfloat16"])
        assert all(np.isfinite(_host(t[k])).all() for k in ("o", "lse", "dq", "dk", "dv"))
        t["q"].zero_()
        _run(t, lens, causal, scale, dict(cap=cap))
