"""lin_distill_topk over many rows, which a CTA takes one after another, and over
long rows beside many entries, and odd values. Bounds as in test_distill_gpu.py.
"""

import numpy as np
import pytest

from oracle import step_oracle as so
from tests.gpu_util import require_gpu
from tests.test_distill_gpu import E, _check, _device, _inputs
from transformer_linear_layer_tcgen05_gb300 import lin

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _results(m, v, ld):
    import torch
    return (torch.full((m, ld), 7.0, device="cuda")[:, :v],
            torch.full((m,), float("nan"), device="cuda"), torch.ones(1, device="cuda"))


# Rows that one CTA takes one after another, of one, two, four and eight warps:
# the losses alone have no barrier of the gradient's between them.
@pytest.mark.parametrize("m,v,k", [(9000, 1000, 4), (9000, 1030, 4), (6000, 2051, 4), (3000, 4100, 9),
                                   (3000, 8000, 9), (1500, 16384, 33), (1500, 16001, 3)])
def test_the_losses_alone_of_many_rows(m, v, k):
    import torch
    z, ids, t = _inputs(m, v, k, seed=m + v)
    zd, idd, td = _device(z, ids, t, v)
    dz, losses, total = _results(m, v, v)
    lin.lin_distill_topk(zd, idd, td, dz, losses, total, 1.5, 0.5)
    torch.cuda.synchronize()
    some = np.linspace(0, m - 1, 40).astype(int)
    want, _ = so.distill_topk(z[some], ids[some], t[some], 1.5, 0.5)
    got = losses.double().cpu().numpy()
    # (z and p: tens at most, terms of 2^-17 of them)
    assert np.all(np.abs(got[some] - want) <= E * 1.5 ** 2 * 120)
    for _ in range(10):
        _, l2, s2 = _results(m, v, v)
        lin.lin_distill_topk(zd, idd, td, None, l2, s2, 1.5, 0.5)
        assert torch.equal(l2, losses) and torch.equal(s2, total)
    assert lin.lin_get_device_status() == lin.LIN_SUCCESS


# Rows of three parts and more (up to 48 CTA's parts of 4096 units, streamed
# twice beyond that), beside few entries and beside as many as there may be.
@pytest.mark.parametrize("m,v,k", [(2, 786432, 1024), (2, 786430, 970), (3, 1048576, 1024),
                                   (2, 1048573, 5), (2, 800001, 64), (2, 600000, 1024)])
def test_long_rows_and_many_entries(m, v, k):
    import torch
    z, ids, t = _inputs(m, v, k, seed=v + k)
    zd, idd, td = _device(z, ids, t, v)
    dz, losses, total = _results(m, v, v)
    lin.lin_distill_topk(zd, idd, td, dz, losses, total, 2.0, 0.5)
    torch.cuda.synchronize()
    assert lin.lin_get_device_status() == lin.LIN_SUCCESS
    _check(z, ids, t, 2.0, 0.5, dz.double().cpu().numpy(), losses.double().cpu().numpy(),
           total.item())
    _, l2, s2 = _results(m, v, v)
    lin.lin_distill_topk(zd, idd, td, None, l2, s2, 2.0, 0.5)
    assert torch.equal(l2, losses) and torch.equal(s2, total)
    lin.lin_distill_topk(zd, idd, td, zd, l2, s2, 2.0, 0.5)
    assert torch.equal(zd, dz) and torch.equal(l2, losses)
    assert lin.lin_get_device_status() == lin.LIN_SUCCESS


@pytest.mark.parametrize("v", [900, 5000, 40000])
def test_teacher_logits_that_are_no_numbers(v):
    # the softmax over a row's entries is NaN where one of its logits is NaN
    # or infinite: so is the loss, and so are the gradients of its entries;
    # the other rows, and a row's other logits, are not touched by it
    import torch
    z, ids, t = _inputs(6, v, 40, seed=9)
    ids[:] = np.arange(100, 140)
    odd = t.copy()
    odd[0, 3] = np.nan
    odd[1, :] = np.nan
    odd[2, 35] = np.inf
    odd[4, :] = np.nan
    odd[4, 7] = -np.inf          # an empty place in a row of NaN
    odd[5, 1] = np.nan
    ids[5] = -1                  # a padding row, whatever its places hold
    zd, idd, td = _device(z, ids, odd, v)
    dz, losses, total = _results(6, v, v)
    lin.lin_distill_topk(zd, idd, td, dz, losses, total, 1.5)
    torch.cuda.synchronize()
    got = losses.cpu().numpy()
    assert np.isnan(got[[0, 1, 2, 4]]).all() and np.isnan(total.item())
    assert got[5] == 0 and torch.all(dz[5] == 0)
    want_l, want_d = so.distill_topk(z, ids, t, 1.5, 1.0)
    size = 1.5 ** 2 * (np.abs(z).max() + 40)
    assert abs(got[3] - want_l[3]) <= E * size
    g = dz.double().cpu().numpy()
    for row in (0, 1, 2, 4):
        listed = np.zeros(v, dtype=bool)
        listed[100:140] = True
        if row == 4:
            listed[107] = False
        assert np.isnan(g[row, listed]).all()
        # (an entry without probability has tau q)
        q = so.distill_topk(z[row:row + 1], np.array([[v - 1]]), np.zeros((1, 1)), 1.5, 1.0)[1][0]
        others = ~listed
        others[v - 1] = False
        assert np.all(np.abs(g[row] - q)[others] <= E * q[others] + 1e-37)
    assert np.isfinite(g[3]).all()


@pytest.mark.parametrize("v", [700, 3001, 33000])
@pytest.mark.parametrize("tau", [1.0, 2.5])
def test_logits_far_from_zero(v, tau):
    # a softmax does not depend on what its logits have in common: with 2^16
    # added to both sides' (on a grid of 2^-7, so that every sum is exact) the
    # results are those of the logits without it, within the bounds of these
    import torch
    z, ids, t = _inputs(5, v, 12, seed=10)
    z, t = (np.round(x * 128) / 128 for x in (z, t))
    zd, idd, td = _device(z + np.float32(65536), ids, t + np.float32(65536), v)
    dz, losses, total = _results(5, v, v)
    lin.lin_distill_topk(zd, idd, td, dz, losses, total, tau, 0.5)
    torch.cuda.synchronize()
    _check(z, ids, t, tau, 0.5, dz.double().cpu().numpy(), losses.double().cpu().numpy(),
           total.item())
