"""The fp64 oracle of the training-step operators: closed forms, and every
gradient against central differences of its forward form."""

import math

import numpy as np
import pytest

from oracle import step_oracle as so


def _directional(f, x, dx, h=1e-5):
    return (f(x + h * dx) - f(x - h * dx)) / (2 * h)


def test_attention_closed_forms():
    rng = np.random.default_rng(1)
    v = rng.standard_normal((5, 2, 3))
    # equal scores: the mean over the keys that the row sees
    o, lse, _ = so.attention(np.zeros((5, 4, 3)), rng.standard_normal((5, 2, 3)), v, True, 0.7)
    for i in range(5):
        np.testing.assert_allclose(o[i, 3], v[:i + 1, 1].mean(axis=0), rtol=1e-13)
        assert math.isclose(lse[2, i], math.log(i + 1), abs_tol=1e-13)
    # fewer keys than queries, causal from the end: the first rows see nothing
    o, lse, _ = so.attention(np.ones((5, 2, 3)), np.ones((2, 2, 3)), v[:2], True, 1.0)
    assert np.all(o[:3] == 0) and np.all(lse[:, :3] == -np.inf)
    np.testing.assert_allclose(o[3], v[0], rtol=1e-15)


def test_attention_sequences_do_not_mix():
    rng = np.random.default_rng(2)
    q, k, v = (rng.standard_normal((7, 2, 4)) for _ in range(3))
    cu = np.array([0, 3, 3, 7])
    o, lse, _ = so.attention(q, k, v, False, 0.5, cu, cu)
    o2, lse2, _ = so.attention(q[3:], k[3:], v[3:], False, 0.5)
    np.testing.assert_array_equal(o[3:], o2)
    np.testing.assert_array_equal(lse[:, 3:], lse2)


@pytest.mark.parametrize("causal,lk", [(False, 5), (True, 5), (True, 3), (True, 9)])
def test_attention_gradient_is_the_difference(causal, lk):
    rng = np.random.default_rng(3 + lk)
    q, do = (rng.standard_normal((5, 4, 6)) for _ in range(2))
    k, v = (rng.standard_normal((lk, 2, 6)) for _ in range(2))
    grads, sizes = so.attention_backward(q, k, v, do, causal, 0.4)
    loss = lambda q, k, v: (so.attention(q, k, v, causal, 0.4)[0] * do).sum()  # noqa: E731
    for g, size, at in zip(grads, sizes, range(3)):
        d = rng.standard_normal(g.shape)
        xs = [q, k, v]
        diff = _directional(lambda x: loss(*(xs[:at] + [x] + xs[at + 1:])), xs[at], d)  # noqa: B023
        assert math.isclose((g * d).sum(), diff, rel_tol=1e-7, abs_tol=1e-8)
        assert np.all(size >= np.abs(g) - 1e-12)


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope_gradient_is_the_difference(interleaved):
    rng = np.random.default_rng(5)
    x = rng.standard_normal((3, 4 * 8))
    w = [rng.standard_normal(8) for _ in range(2)]
    ang = rng.standard_normal((6, 3))
    pos = np.array([5, 0, 2])
    dys = [rng.standard_normal((3, h, 8)) for h in (2, 1, 1)]
    f = lambda x, wq, wk: sum(  # noqa: E731
        (y * d).sum() for y, d in zip(so.qk_norm_rope(x, wq, wk, np.cos(ang), np.sin(ang), pos, 2,
                                                      1, 1e-3, interleaved), dys))
    grads = so.qk_norm_rope_backward(x, *w, np.cos(ang), np.sin(ang), pos, *dys, 1e-3, interleaved)
    args = [x, *w]
    for at, g in enumerate(grads):
        d = rng.standard_normal(g.shape)
        diff = _directional(lambda y: f(*(args[:at] + [y] + args[at + 1:])), args[at], d)  # noqa: B023
        assert math.isclose((g * d).sum(), diff, rel_tol=1e-8, abs_tol=1e-8)


def test_norm_rope_keeps_lengths():
    # a rotation keeps the norm of every pair: unit weights give rows of norm sqrt(d)
    rng = np.random.default_rng(6)
    x = rng.standard_normal((4, 3 * 10))
    ang = rng.standard_normal((9, 5))
    for inter in (False, True):
        q, k, v = so.qk_norm_rope(x, np.ones(10), np.ones(10), np.cos(ang), np.sin(ang),
                                  np.array([0, 8, 3, 3]), 1, 1, 0.0, inter)
        np.testing.assert_allclose((q ** 2).sum(-1), 10.0, rtol=1e-12)
        np.testing.assert_allclose((k ** 2).sum(-1), 10.0, rtol=1e-12)
        np.testing.assert_array_equal(v[:, 0], x[:, 20:])


def test_distillation_gradient_is_the_difference():
    rng = np.random.default_rng(7)
    z = rng.standard_normal((4, 11)) * 2
    ids = np.array([[1, 5, 9], [0, -1, 3], [-1, -1, -1], [4, 4, 99]])
    t = rng.standard_normal((4, 3))
    losses, dz = so.distill_topk(z, ids, t, 1.7, 0.25)
    assert losses[2] == 0 and np.all(dz[2] == 0) and np.all(losses[:2] > 0)
    d = rng.standard_normal(z.shape)
    diff = _directional(lambda y: so.distill_topk(y, ids, t, 1.7, 0.25)[0].sum(), z, d)
    assert math.isclose((dz * d).sum(), 0.25 * diff, rel_tol=1e-7, abs_tol=1e-9)
    np.testing.assert_allclose(dz.sum(axis=1), 0, atol=1e-15)


def test_distillation_of_the_same_distribution_is_zero():
    # the teacher's entries are the whole vocabulary and its logits the student's
    rng = np.random.default_rng(8)
    z = rng.standard_normal((3, 6))
    ids = np.tile(rng.permutation(6), (3, 1))
    losses, dz = so.distill_topk(z, ids, np.take_along_axis(z, ids, 1) + 4.0, 2.0, 1.0)
    np.testing.assert_allclose(losses, 0, atol=1e-14)
    np.testing.assert_allclose(dz, 0, atol=1e-15)
