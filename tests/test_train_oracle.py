"""The fp64 oracle of the block norms, scored attention and AdamW, pinned by
closed forms, differences and the codes' own definition (CPU only)."""

import numpy as np
import pytest

from oracle import step_oracle as so
from oracle import train_oracle as to


def _difference(f, x, at, h=1e-6):
    a, b = x.copy(), x.copy()
    a[at] += h
    b[at] -= h
    return (f(a) - f(b)) / (2 * h)


def test_block_norms_closed_form():
    # a row of equal entries c has rms |c|: its norm is the weight
    x, w = np.full((2, 4), 3.0), np.array([1.0, 2.0, -1.0, 0.5])
    (h, n), _ = to.block_norms(x, None, None, None, w, 2.0, 1.0, 0.0)
    assert np.allclose(h, 6.0) and np.allclose(n, w)
    (h, n), _ = to.block_norms(x, -x, np.array([1.0, 0.0, 1.0, 1.0]), w, None, 1.0, 10.0, 0.0)
    assert n is None and np.allclose(h, 3.0 - 10.0 * w * [1, 0, 1, 1])


@pytest.mark.parametrize("gate", [None, (6,), (3, 1), (3, 6)])
@pytest.mark.parametrize("post", [False, True])
def test_block_norms_gradient_is_the_difference(gate, post):
    r = np.random.default_rng(1)
    v = dict(x=r.normal(size=(3, 6)), y=r.normal(size=(3, 6)), w_pre=r.normal(size=6))
    v["gate"] = None if gate is None else r.normal(size=gate)
    v["w_post"] = r.normal(size=6) if post else None
    ch, cn = r.normal(size=(3, 6)), r.normal(size=(3, 6))

    def loss(**new):
        a = {**v, **new}
        (h, n), _ = to.block_norms(a["x"], a["y"], a["gate"], a["w_post"], a["w_pre"], 0.8, 1.3, 1e-3)
        return (h * ch).sum() + (n * cn).sum()

    (h, _), _ = to.block_norms(v["x"], v["y"], v["gate"], v["w_post"], v["w_pre"], 0.8, 1.3, 1e-3)
    got, _ = to.block_norms_backward(h, v["y"], v["gate"], v["w_post"], v["w_pre"], ch, cn, 0.8, 1.3,
                                     1e-3)
    for name in ("x", "y", "gate", "w_post", "w_pre"):
        if v[name] is None:
            continue
        d = got["d" + name]
        assert d.shape == v[name].shape
        for at in np.ndindex(*d.shape):
            assert abs(d[at] - _difference(lambda t: loss(**{name: t}), v[name], at)) < 1e-6


def test_codes():
    every = np.arange(256, dtype=np.uint8)
    values = to.e4m3_values(every)
    assert values[0x7e] == 448 and values[1] == 2.0 ** -9 and np.isnan(values[0x7f])
    keep = ~np.isnan(values)
    assert np.array_equal(to.e4m3_codes(values[keep]), every[keep])
    # between two codes the nearer, in the middle the even one, behind 448 448
    assert np.array_equal(to.e4m3_codes([1.0625, 1.06, 1.1875, 500.0, -1e9]),
                          to.e4m3_codes([1.0, 1.0, 1.25, 448.0, -448.0]))
    torch = pytest.importorskip("torch")
    x = (np.random.default_rng(0).normal(size=4000) * 30).astype(np.float32)
    got = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(got, to.e4m3_codes(x))


def test_coded_blocks():
    x = np.concatenate([np.linspace(-2, 2, 256), np.full(10, 2.0 ** -101), [np.inf, np.nan, 1.0]])
    c, s = to.coded(x.astype(np.float32))
    assert np.isclose(s[0], 2 / 448, rtol=1e-6) and c[0] == 0xfe and c[255] == 0x7e
    assert np.isclose(s[1], 1 / 448, rtol=1e-6) and c[266] == 127 and c[267] == 127 and c[268] == 0x7e
    c, s = to.coded(np.array([1.0, 1e-9, 0.0], np.float32), least=True)
    assert list(c) == [0x7e, 1, 0]


def test_adamw_first_step():
    # the first step from zero states goes by lr along the gradient's sign
    p, m, v = to.adamw([1.0, -2.0], [0.3, -5.0], [0, 0], [0, 0], 1, 0.1, 0.9, 0.99, 0.0, 0.0)
    assert np.allclose(p, [0.9, -1.9]) and np.allclose(m, [0.03, -0.5])


def test_scored_attention_without_scores_is_attention():
    r = np.random.default_rng(2)
    q, k, v, do = (r.normal(size=s) for s in ((7, 4, 8), (9, 2, 8), (9, 2, 8), (7, 4, 8)))
    for a, b in zip(to.attention_scores(q, k, v, True, 0.3), so.attention(q, k, v, True, 0.3)):
        assert np.allclose(a, b)
    a, b = to.attention_scores_backward(q, k, v, do, True, 0.3), so.attention_backward(q, k, v, do, True, 0.3)
    for x, y in zip(a[0], b[0]):
        assert np.allclose(x, y)


def test_scored_attention_gradient_is_the_difference():
    r = np.random.default_rng(3)
    q, k, v = 2 * r.normal(size=(4, 2, 4)), r.normal(size=(5, 1, 4)), r.normal(size=(5, 1, 4))
    do = r.normal(size=q.shape)
    how = dict(causal=False, scale=0.7, cap=1.5, slopes=[0.2, -0.1], first=np.array([0, 1, 3, 2]),
               end=np.array([5, 4, 3, 5]))
    f = lambda q, k, v: (to.attention_scores(q, k, v, **how)[0] * do).sum()  # noqa: E731
    got, _ = to.attention_scores_backward(q, k, v, do, **how)
    for i, x in enumerate((q, k, v)):
        for at in np.ndindex(*x.shape):
            args = lambda t: f(*(t if j == i else y for j, y in enumerate((q, k, v))))  # noqa: E731
            assert abs(got[i][at] - _difference(args, x, at)) < 1e-7
    assert not got[0][2].any()   # (the row without a key)
