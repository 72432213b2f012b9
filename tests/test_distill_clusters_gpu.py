"""lin_distill_topk over rows that one cluster of CTAs takes one after another.
Bounds as in test_distill_gpu.py.
"""

import numpy as np
import pytest

from tests.gpu_util import require_gpu
from tests.test_distill_gpu import E, _check
from transformer_linear_layer_tcgen05_gb300 import lin

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _results(m, v, ld):
    import torch
    return (torch.full((m, ld), 7.0, device="cuda")[:, :v],
            torch.full((m,), float("nan"), device="cuda"), torch.ones(1, device="cuda"))


# Rows that one cluster takes one after another, of every cluster size: the
# exchange between its CTAs, the entries' ring, the slots and, in place, rows
# overwritten while a peer is at the next one, all go round several times.
@pytest.mark.parametrize("m,v,k", [(1200, 16388, 40), (800, 32768, 7), (700, 50001, 40),
                                   (400, 65539, 100), (400, 131072, 40), (150, 262144, 40),
                                   (60, 600001, 40), (40, 1048576, 40)])
@pytest.mark.parametrize("pad", [0, 3], ids=["dense rows", "padded rows"])
def test_many_rows_of_clusters(m, v, k, pad):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(m + v)
    buf = torch.full((m, v + pad), float("nan"), device="cuda")
    zd = buf[:, :v]
    for a in range(0, m, 64):
        zd[a:a + 64] = 4 * torch.randn(min(64, m - a), v, generator=g, device="cuda")
    rng = np.random.default_rng(m + v)
    # (a random stride through the vocabulary: different entries)
    ids = (rng.integers(0, v, (m, 1)) + np.arange(k) * 7919) % v
    ids[3::8, k // 2:] = -1
    ids[5::16] = -1
    t = (3 * rng.standard_normal((m, k))).astype(np.float32)
    ids = ids.astype(np.int32)
    idd, td = torch.from_numpy(ids).cuda(), torch.from_numpy(t).cuda()
    some = np.unique(np.linspace(0, m - 1, 12).astype(int))
    z = zd[torch.from_numpy(some).cuda()].cpu().numpy()
    dz, losses, total = _results(m, v, v + pad)
    lin.lin_distill_topk(zd, idd, td, dz, losses, total, 2.0, 0.25)
    torch.cuda.synchronize()
    assert lin.lin_get_device_status() == lin.LIN_SUCCESS
    got = losses.double().cpu().numpy()
    _check(z, ids[some], t[some], 2.0, 0.25, dz[torch.from_numpy(some).cuda()].double().cpu().numpy(),
           got[some], got[some].sum())
    assert abs(total.item() - got.sum()) <= 1e-6 * np.abs(got).sum()
    # every row's gradient sums to nothing (to the rounding of its terms), and
    # those of padding rows are zero
    sums = torch.stack([dz[i].double().sum() for i in range(m)]).cpu().numpy()
    assert np.all(np.abs(sums) <= 2 * E * 2.0 * 0.25 * 2)
    assert torch.all(dz[5::16] == 0)
    for out in (None, zd):
        for _ in range(3 if out is None else 1):
            _, l2, s2 = _results(m, 1, 1)
            lin.lin_distill_topk(zd, idd, td, out, l2, s2, 2.0, 0.25)
            assert torch.equal(l2, losses) and torch.equal(s2, total)
    assert torch.equal(zd, dz)
    assert lin.lin_get_device_status() == lin.LIN_SUCCESS
