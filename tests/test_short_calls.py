"""The extension module behind the short calls refuses what the library must
not see, before anything touches CUDA (CPU only)."""

import pytest

from transformer_linear_layer_tcgen05_gb300 import build, lin

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build_library()


def _heads(*shape, dtype=torch.float16):
    return torch.zeros(*shape, dtype=dtype)


@pytest.mark.parametrize("bad", [None, 3, "q", _heads(4, 2, 8), _heads(4, 2, 8, dtype=torch.int16)])
def test_attention_wants_cuda_heads(bad):
    with pytest.raises(TypeError, match="Q must be a CUDA tensor"):
        lin.lin_attention(bad, bad, bad, bad, bad)
    with pytest.raises(TypeError, match="Q must be a CUDA tensor"):
        lin.lin_attention_backward(bad, bad, bad, bad, bad, bad, bad, bad, bad)


def test_norm_and_rotation_want_cuda_heads():
    x, h = torch.zeros(4, 48), _heads(4, 2, 8)
    with pytest.raises(TypeError, match="Q must be a CUDA tensor"):
        lin.lin_qk_norm_rope(x, None, None, None, None, None, h, h, h)
    with pytest.raises(TypeError, match="dQ must be a CUDA tensor"):
        lin.lin_qk_norm_rope_backward(x, None, None, None, None, None, h, h, h, x, None, None)


def test_distillation_wants_cuda_logits():
    z = torch.zeros(3, 5)
    for bad in (z, None, 1.0, torch.zeros(3, 5, dtype=torch.float64)):
        with pytest.raises(TypeError, match="logits must be a float32 CUDA matrix"):
            lin.lin_distill_topk(bad, z, z, z, z, z)


def test_the_module_counts_its_arguments():
    calls = lin._short_calls()
    for f, n in ((calls.attention, 12), (calls.attention_backward, 16), (calls.qk_norm_rope, 12),
                 (calls.qk_norm_rope_backward, 15), (calls.distill_topk, 9)):
        with pytest.raises(TypeError, match=f"{n} arguments, not 1"):
            f(None)


def test_binding_wants_every_function():
    calls = lin._short_calls()
    with pytest.raises(KeyError):
        calls.bind({"lin_attention": 1})
    with pytest.raises(ValueError):
        calls.bind({n: 0 for n in ("lin_attention", "lin_attention_backward", "lin_qk_norm_rope",
                                   "lin_qk_norm_rope_backward", "lin_distill_topk")})
