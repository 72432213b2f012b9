"""lin_distill_topk on the GPU against the fp64 oracle.

Bounds: an exponential's argument z / tau (tens at most, in base 2) is rounded
at 2^-24 of itself and the exponential to 2^-22, so q is off by less than
2^-17 of itself, and so is p; a loss by the same share of its terms'
magnitudes, sum p (|log p| + |log q|).
"""

import numpy as np
import pytest

from oracle import step_oracle as so
from tests.gpu_util import require_gpu
from transformer_linear_layer_tcgen05_gb300 import lin

pytestmark = pytest.mark.gpu

E = 2.0 ** -17


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _inputs(m, v, k, seed, ld=None):
    rng = np.random.default_rng(seed)
    z = (4 * rng.standard_normal((m, v))).astype(np.float32)
    ids = np.stack([rng.permutation(v)[:k] for _ in range(m)]).astype(np.int32).reshape(m, k)
    t = (3 * rng.standard_normal((m, k))).astype(np.float32)
    if k > 1:
        ids[::3, rng.integers(1, k):] = -1          # rows with fewer entries
    if k > 2:
        ids[1::4, k // 2] = v + 7                   # an id behind the vocabulary
    if m > 2:
        ids[2] = -1                                 # a padding row
    return z, ids, t


def _device(z, ids, t, ld):
    import torch
    buf = torch.full((z.shape[0], ld), float("nan"), device="cuda")
    zd = buf[:, :z.shape[1]]
    zd.copy_(torch.from_numpy(z))
    return zd, torch.from_numpy(ids).cuda(), torch.from_numpy(t).cuda()


def _check(z, ids, t, tau, inv, dz, losses, total):
    want_l, want_d = so.distill_topk(z, ids, t, tau, inv)
    m, v = z.shape
    if dz is not None:
        plain, _ = so.distill_topk(z, np.full((m, 1), -1), np.zeros((m, 1)), tau, inv)
        # q + p bounds both terms: |dz| / (tau inv) + 2 p
        p = np.zeros((m, v))
        for i in range(m):
            has = (ids[i] >= 0) & (ids[i] < v)
            if has.any():
                e = np.exp((t[i, has] - t[i, has].max()) / np.float64(tau))
                np.add.at(p[i], ids[i][has], e / e.sum())
        size = np.abs(want_d) + 2 * p * tau * inv
        assert np.all(np.abs(dz - want_d) <= E * size + 1e-37)
    lse = np.log(np.exp(z.astype(np.float64) / tau - (z / tau).max(1, keepdims=True)).sum(1)) + \
        (z / np.float64(tau)).max(1)
    size = tau ** 2 * (np.abs(lse) + np.abs(z).max(1) / tau + 20)
    assert np.all(np.abs(losses - want_l) <= E * size)
    assert abs(total - losses.sum()) <= 1e-6 * np.abs(losses).sum() + 1e-12
    empty = ~((ids >= 0) & (ids < v)).any(axis=1)
    assert np.all(losses[empty] == 0)
    if dz is not None:
        assert np.all(dz[empty] == 0)


# (rows, vocabulary, entries): a vocabulary of one; sizes of one access, of
# one CTA, of every cluster size, at their edges, and longer than a cluster
# of eight holds
SHAPES = [(1, 1, 1), (3, 5, 3), (7, 1003, 1), (9, 4096, 33), (5, 16384, 32), (5, 16388, 8),
          (4, 32769, 100), (3, 50001, 20), (3, 131072, 64), (3, 131076, 5), (2, 300007, 1024)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("tau,inv", [(1.0, 1.0), (2.5, 1.0 / 3)])
@pytest.mark.parametrize("wide", [False, True], ids=["rows of any stride", "16-byte rows"])
def test_against_the_oracle(shape, tau, inv, wide):
    import torch
    m, v, k = shape
    z, ids, t = _inputs(m, v, min(k, v), seed=v + k)
    ld = -(-v // 4) * 4 if wide else v + 3
    zd, idd, td = _device(z, ids, t, ld)
    out = torch.full((m, ld), 7.0, device="cuda")
    losses, total = torch.full((m,), float("nan"), device="cuda"), torch.ones(1, device="cuda")
    lin.lin_distill_topk(zd, idd, td, out[:, :v], losses, total, tau, inv)
    assert lin.lin_last_launch_info() == (2, 0)
    torch.cuda.synchronize()
    assert lin.lin_get_device_status() == lin.LIN_SUCCESS
    dz = out[:, :v].double().cpu().numpy()
    _check(z, ids, t, tau, inv, dz, losses.double().cpu().numpy(), total.item())
    assert torch.all(out[:, v:] == 7.0)   # nothing behind the vocabulary
    # the losses alone, then in place: the same bits
    l2, s2 = torch.empty_like(losses), torch.empty_like(total)
    lin.lin_distill_topk(zd, idd, td, None, l2, s2, tau, inv)
    assert torch.equal(l2, losses) and torch.equal(s2, total)
    lin.lin_distill_topk(zd, idd, td, zd, l2, s2, tau, inv)
    torch.cuda.synchronize()
    assert torch.equal(zd, out[:, :v]) and torch.equal(l2, losses)


@pytest.mark.parametrize("v", [40, 20000])
def test_an_entry_listed_twice(v):
    import torch
    z, ids, t = _inputs(4, v, 6, seed=3)
    ids[0] = [5, 9, 5, 5, 9, 1]
    ids[3] = v - 1
    zd, idd, td = _device(z, ids, t, v)
    losses, total = torch.empty(4, device="cuda"), torch.empty(1, device="cuda")
    dz = torch.empty_like(zd)
    lin.lin_distill_topk(zd, idd, td, dz, losses, total, 1.5)
    _check(z, ids, t, 1.5, 1.0, dz.double().cpu().numpy(), losses.double().cpu().numpy(),
           total.item())


def test_masked_logits_and_teacher_logits():
    # logits of -inf and of the type's lowest value have no probability; a
    # teacher logit of -inf is an empty place
    import torch
    z, ids, t = _inputs(4, 3001, 5, seed=4)
    ids[:] = np.arange(10, 15)
    z[:, 100:2500] = -np.inf
    z[:, 2500] = np.finfo(np.float32).min
    t[1, 2] = -np.inf
    t[3] = -np.inf
    zd, idd, td = _device(z, ids, t, 3001)
    losses, total = torch.empty(4, device="cuda"), torch.empty(1, device="cuda")
    dz = torch.empty_like(zd)
    lin.lin_distill_topk(zd, idd, td, dz, losses, total, 2.0, 0.5)
    ids2 = ids.copy()
    ids2[1, 2] = -1
    ids2[3] = -1
    t2 = np.where(np.isinf(t), 0, t)
    _check(np.maximum(z, -1e4), ids2, t2, 2.0, 0.5, dz.double().cpu().numpy(),
           losses.double().cpu().numpy(), total.item())
    assert torch.all(dz[:3, 100:2501] == 0)


def test_gradient_is_the_difference_of_the_losses():
    import torch
    z, ids, t = _inputs(5, 777, 9, seed=5)
    zd, idd, td = _device(z, ids, t, 777)
    losses, total = torch.empty(5, device="cuda"), torch.empty(1, device="cuda")
    dz = torch.empty_like(zd)
    lin.lin_distill_topk(zd, idd, td, dz, losses, total, 3.0, 0.2)
    d = np.random.default_rng(5).standard_normal(z.shape)
    f = lambda h: so.distill_topk(z + h * d, ids, t, 3.0, 0.2)[0].sum()  # noqa: E731
    diff = 0.2 * (f(1e-5) - f(-1e-5)) / 2e-5
    g = dz.double().cpu().numpy()
    assert abs((g * d).sum() - diff) <= 1e-5 * np.linalg.norm(g) * np.linalg.norm(d)


def test_nothing_to_do():
    import torch
    e = lambda *s, dt=torch.float32: torch.ones(s, device="cuda", dtype=dt)  # noqa: E731
    total, losses = e(1), e(3)
    lin.lin_distill_topk(e(0, 9), e(0, 2, dt=torch.int32), e(0, 2), e(0, 9), e(0), total)
    assert total.item() == 0
    total.fill_(1)
    lin.lin_distill_topk(e(3, 9), e(3, 0, dt=torch.int32), e(3, 0), None, losses, total)
    assert total.item() == 0 and torch.all(losses == 0)   # no entries: padding rows


def test_refusals():
    import torch
    z, ids, t = _inputs(4, 64, 5, seed=6)
    zd, idd, td = _device(z, ids, t, 64)
    losses, total = torch.empty(4, device="cuda"), torch.empty(1, device="cuda")

    def refused(status, *a, **kw):
        with pytest.raises(lin.LinError) as e:
            lin.lin_distill_topk(*a, **kw)
        assert e.value.status == status

    for tau in (0.0, -1.0, float("inf"), float("nan")):
        refused(lin.LIN_ERROR_INVALID_VALUE, zd, idd, td, None, losses, total, tau)
    wide = torch.zeros((4, 1025), device="cuda")
    refused(lin.LIN_ERROR_UNSUPPORTED_SHAPE, zd, wide.int(), wide, None, losses, total)
    refused(lin.LIN_ERROR_INVALID_VALUE, zd[:1].expand(4, 64), idd, td, None, losses, total)
    buf = torch.zeros((4, 80), device="cuda")
    refused(lin.LIN_ERROR_ALIASING, buf[:, :64], idd, td, buf[:, 8:72], losses, total)
    flat = torch.zeros(4 * 64 + 4, device="cuda")
    refused(lin.LIN_ERROR_ALIASING, zd, idd, td, flat[:256].view(4, 64), flat[200:204], total)
    with pytest.raises(TypeError):
        lin.lin_distill_topk(zd, idd.long(), td, None, losses, total)
    with pytest.raises(TypeError):
        lin.lin_distill_topk(zd, idd, td[:, :4], None, losses, total)
    with pytest.raises(ValueError):
        lin.lin_distill_topk(zd, idd, td, torch.empty(64, 4, device="cuda").t(), losses, total)


# rows of one, two and four warps at the edges between them, and so many rows
# that a CTA walks over several
@pytest.mark.parametrize("m,v,k", [(40, 1020, 9), (40, 1024, 9), (40, 1027, 9), (7000, 1999, 3),
                                   (40, 2044, 40), (40, 2048, 40), (40, 2051, 40), (5000, 1030, 5),
                                   (40, 4100, 3), (2500, 4090, 5)])
def test_widths_of_a_row(m, v, k):
    import torch
    z, ids, t = _inputs(m, v, k, seed=m + v)
    zd, idd, td = _device(z, ids, t, v)
    out = torch.full((m, v), 7.0, device="cuda")
    losses, total = torch.full((m,), float("nan"), device="cuda"), torch.ones(1, device="cuda")
    lin.lin_distill_topk(zd, idd, td, out, losses, total, 1.5, 0.5)
    torch.cuda.synchronize()
    assert lin.lin_get_device_status() == lin.LIN_SUCCESS
    _check(z, ids, t, 1.5, 0.5, out.double().cpu().numpy(), losses.double().cpu().numpy(),
           total.item())
