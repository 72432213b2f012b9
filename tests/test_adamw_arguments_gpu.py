"""lin_adamw's arguments: tensors that are laid out like the weights, and the
smallest eps."""

import pytest

from tests.gpu_util import require_gpu
from transformer_linear_layer_tcgen05_gb300 import lin

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _group(shape, bits):
    import torch
    st = dict(p=torch.randn(shape, device="cuda"), g=torch.randn(shape, device="cuda"))
    n = st["p"].numel()
    for k in ("m", "v"):
        st[k] = torch.zeros(shape, device="cuda", dtype=torch.uint8 if bits == 8 else torch.float32)
        st[k] = st[k].view(torch.float8_e4m3fn) if bits == 8 else st[k]
        st[k + "_scale"] = torch.zeros(-(-n // 256), device="cuda")
    st["w16"] = torch.zeros(shape, device="cuda", dtype=torch.float16)
    return st


def _step(st, bits, **how):
    import torch
    one = {k: [v] for k, v in st.items()}
    scales = dict(m_scale=one["m_scale"], v_scale=one["v_scale"]) if bits == 8 else {}
    lin.lin_adamw(one["p"], one["g"], one["m"], one["v"], w16=one["w16"], **scales, **how)
    torch.cuda.synchronize()
    assert lin.lin_get_device_status() == lin.LIN_SUCCESS


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("which", ["g", "m", "v", "w16"])
def test_tensors_of_another_shape_are_refused(bits, which):
    # as many entries in another order would scramble the weight
    st = _group((24, 40), bits)
    for shape in ((40, 24), (48, 20), (2, 12, 40)):
        bad = dict(st, **{which: st[which].view(shape)})
        was = st["p"].clone()
        with pytest.raises((TypeError, ValueError)):
            _step(bad, bits)
        assert (st["p"] == was).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_flat_tensors_and_ones_in_a_shape(bits):
    # (buffers of a whole bucket; entries in the weight's own order)
    import torch
    st = _group((24, 40), bits)
    want = {k: t.clone() for k, t in st.items()}
    _step(want, bits)
    for shape in ((960,), (1, 24, 40), (24, 1, 40), (960, 1)):
        got = {k: t.clone() for k, t in st.items()}
        _step({k: t.view(shape) if k in ("g", "m", "v", "w16") else t for k, t in got.items()}, bits)
        for k in want:
            assert torch.equal(got[k].view(torch.uint8), want[k].view(torch.uint8)), (k, shape)
    got = {k: t.clone() for k, t in st.items()}
    _step(dict(got, p=got["p"].view(-1)), bits)
    assert torch.equal(got["p"], want["p"])


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [1e-300, 1e-46, 1e-42, 2e-39, 1e-38, 1e-20])
@pytest.mark.parametrize("on_device", [False, True])
def test_eps_below_what_float32_holds(bits, eps, on_device):
    # entries that have had no gradient yet: 0 / eps
    import torch
    st = _group((700,), bits)
    st["g"][::3] = 0
    want = st["p"][::3] * (1 - 0.01 * 0.1)
    step = torch.ones(1, dtype=torch.int32, device="cuda") if on_device else 1
    _step(st, bits, step=step, lr=0.01, eps=eps, weight_decay=0.1)
    # (the factor rounded to float32, and the product)
    assert (st["p"][::3] - want).abs().le(2.0 ** -22 * want.abs()).all()
    assert torch.isfinite(st["p"]).all()
