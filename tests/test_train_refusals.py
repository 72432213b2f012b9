"""What the block norms, the rotation by axes and the AdamW step refuse before
anything touches CUDA (CPU only: fake, never-dereferenced addresses)."""

import ctypes

import pytest

from transformer_linear_layer_tcgen05_gb300 import build, lin

BASE = 1 << 40
INVALID, SHAPE, ALIGN, ALIAS = (lin.LIN_ERROR_INVALID_VALUE, lin.LIN_ERROR_UNSUPPORTED_SHAPE,
                                lin.LIN_ERROR_MISALIGNED, lin.LIN_ERROR_ALIASING)


class Norms(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("gate", ctypes.c_int32), ("tokens", ctypes.c_int64),
                ("width", ctypes.c_int64), ("residual_scale", ctypes.c_float),
                ("block_scale", ctypes.c_float), ("eps", ctypes.c_float)]


class Tensor(ctypes.Structure):
    _fields_ = [(k, ctypes.c_void_p) for k in ("p", "g", "m", "v", "m_scale", "v_scale", "w16")] + \
        [("n", ctypes.c_int64)]


class Step(ctypes.Structure):
    _fields_ = [("state_bits", ctypes.c_int32), ("step", ctypes.c_int64)] + \
        [(k, ctypes.c_double) for k in ("lr", "beta1", "beta2", "eps", "weight_decay")] + \
        [(k, ctypes.c_void_p) for k in ("lr_device", "step_device", "grad_scale")]


@pytest.fixture(scope="module")
def L():
    build.build_library()
    return lin.lib()


def _at(i):
    return BASE + (i << 32)


# ---------------------------------------------------------------- norms

FORWARD = ("X", "Y", "GATE", "W_POST", "W_PRE", "H", "N")
BACKWARD = ("H", "Y", "GATE", "W_POST", "W_PRE", "DH", "DN", "DX", "DY", "DGATE", "DW_POST", "DW_PRE")


def _norms(L, backward=False, shape=None, **new):
    s = Norms(**{**dict(dtype=2, gate=1, tokens=8, width=64, residual_scale=1, block_scale=1, eps=1e-6),
                 **(shape or {})})
    names = BACKWARD if backward else FORWARD
    p = {k: _at(i + 1) for i, k in enumerate(names)}
    assert set(new) <= set(p)
    p.update(new)
    f = L.lin_block_norms_backward if backward else L.lin_block_norms
    return f(ctypes.byref(s), *(p[k] for k in names), None)



@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("bad, want", [
    (dict(dtype=3), INVALID), (dict(dtype=-1), INVALID), (dict(gate=4), INVALID),
    (dict(gate=0), INVALID),                 # a gate that is none
    (dict(tokens=-1), INVALID), (dict(width=-4), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(residual_scale=float("inf")), INVALID), (dict(block_scale=float("nan")), INVALID),
    (dict(width=66), SHAPE), (dict(width=8196), SHAPE), (dict(tokens=1 << 31), SHAPE),
    (dict(tokens=1 << 28, width=4096), SHAPE)])
def test_norms_shapes(L, backward, bad, want):
    assert _norms(L, backward, bad) == want


@pytest.mark.parametrize("new", [dict(X=None), dict(GATE=None), dict(Y=None), dict(N=None),
                                 dict(W_PRE=None), dict(H=None, N=None, W_PRE=None)])
def test_norms_forward_wants_what_goes_together(L, new):
    assert _norms(L, **new) == INVALID


@pytest.mark.parametrize("new", [dict(DX=None), dict(DGATE=None), dict(DY=None), dict(DW_POST=None),
                                 dict(DW_PRE=None), dict(W_POST=None), dict(W_PRE=None), dict(Y=None),
                                 dict(H=None), dict(DN=None), dict(GATE=None),
                                 dict(DH=None, DN=None, W_PRE=None, DW_PRE=None)])
def test_norms_backward_wants_what_goes_together(L, new):
    assert _norms(L, True, **new) == INVALID


def test_norms_alignment_and_overlap(L):
    for k in FORWARD:
        i = FORWARD.index(k) + 1
        assert _norms(L, **{k: _at(i) + 4}) == ALIGN
    # 16-bit tensors need 8 bytes, a token's gate 4
    assert _norms(L, shape=dict(dtype=1), Y=_at(2) + 8) != ALIGN
    assert _norms(L, shape=dict(dtype=1), Y=_at(2) + 4) == ALIGN
    assert _norms(L, shape=dict(gate=2), GATE=_at(3) + 4) != ALIGN
    rows = 8 * 64 * 4
    for out in ("H", "N"):
        for k in FORWARD:
            if k not in (out, "X"):
                assert _norms(L, **{k: _at(1), out: _at(1), "X": _at(20)}) == ALIAS
    assert _norms(L, H=_at(1)) != ALIAS                       # H over X
    assert _norms(L, H=_at(1) + 16) == ALIAS                  # not beside it
    assert _norms(L, N=_at(1)) == ALIAS
    assert _norms(L, H=_at(1) + rows) != ALIAS
    assert _norms(L, True, DX=_at(BACKWARD.index("DH") + 1)) != ALIAS
    assert _norms(L, True, DX=_at(1)) == ALIAS                # over H
    assert _norms(L, True, DY=_at(2)) == ALIAS
    assert _norms(L, True, DW_PRE=_at(BACKWARD.index("DW_POST") + 1) + 16) == ALIAS


def test_norms_without_entries(L):
    assert _norms(L, shape=dict(tokens=0)) == lin.LIN_SUCCESS
    assert _norms(L, shape=dict(width=0)) == lin.LIN_SUCCESS
    assert _norms(L, True, shape=dict(width=0)) == lin.LIN_SUCCESS
    assert lin.lin_last_launch_info() == (0, 0)


# ---------------------------------------------------------------- AdamW

def _step(L, tensors, count=None, **how):
    s = Step(**{**dict(state_bits=32, step=1, lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1),
                **how})
    list_ = (Tensor * max(1, len(tensors)))(*tensors)
    return L.lin_adamw(ctypes.byref(s), list_, len(tensors) if count is None else count, None)


def _tensor(i=0, n=1000, **new):
    p = {k: _at(10 * i + j + 1) for j, k in enumerate(("p", "g", "m", "v", "m_scale", "v_scale", "w16"))}
    return Tensor(**{**p, "n": n, **new})


@pytest.mark.parametrize("how", [dict(state_bits=16), dict(step=0), dict(step=-3), dict(beta1=1.0),
                                 dict(beta2=-0.1), dict(beta1=float("nan")), dict(eps=-1e-9),
                                 dict(eps=float("inf")), dict(lr=float("nan")),
                                 dict(weight_decay=float("inf"))])
def test_adamw_numbers(L, how):
    assert _step(L, [_tensor()], **how) == INVALID


def test_adamw_tensors(L):
    assert L.lin_adamw(None, None, 0, None) == INVALID
    assert _step(L, [], count=-1) == INVALID
    assert _step(L, []) == lin.LIN_SUCCESS
    assert _step(L, [_tensor(n=0), Tensor(n=0)]) == lin.LIN_SUCCESS   # nothing to do
    assert _step(L, [_tensor(n=-1)]) == INVALID
    assert _step(L, [_tensor(n=1 << 39)]) == SHAPE
    assert _step(L, [_tensor()], count=(1 << 20) + 1) == SHAPE
    for k in ("p", "g", "m", "v"):
        assert _step(L, [_tensor(**{k: None})]) == INVALID
        assert _step(L, [_tensor(**{k: _at(5) + 2})]) == ALIGN
    for k in ("m_scale", "v_scale"):
        assert _step(L, [_tensor(**{k: None})], state_bits=8) == INVALID
        assert _step(L, [_tensor(**{k: _at(50) + 2})], state_bits=8) == ALIGN
    assert _step(L, [_tensor(w16=_at(50) + 1)]) == ALIGN
    assert _step(L, [_tensor()], grad_scale=_at(60) + 1) == ALIGN


def test_adamw_overlap(L):
    a = _tensor()
    for k in ("p", "g", "m", "v", "w16"):
        for j in ("p", "m", "v", "w16"):
            if j != k:
                assert _step(L, [_tensor(**{j: getattr(a, k)})]) == ALIAS
    assert _step(L, [_tensor(), _tensor()]) == ALIAS            # the same tensor twice
    assert _step(L, [_tensor(), _tensor(1, g=_at(2))]) != ALIAS  # a gradient of two tensors
    assert _step(L, [_tensor(), _tensor(1, m=_at(1) + 3996)]) == ALIAS
    assert _step(L, [_tensor(), _tensor(1, m=_at(1) + 4000)]) != ALIAS
    assert _step(L, [_tensor()], grad_scale=_at(1)) == ALIAS
    # codes are one byte an entry, scales one float to 256 of them
    assert _step(L, [_tensor(), _tensor(1, v=_at(3) + 1000)], state_bits=8) != ALIAS
    assert _step(L, [_tensor(), _tensor(1, v=_at(3) + 999)], state_bits=8) == ALIAS
    assert _step(L, [_tensor(), _tensor(1, v=_at(5) + 15)], state_bits=8) == ALIAS
    assert _step(L, [_tensor(), _tensor(1, v=_at(5) + 16)], state_bits=8) != ALIAS


# ---------------------------------------------------------------- axes and Python

def test_axes_count(L):
    for f, n in ((L.lin_qk_norm_rope_axes, 10), (L.lin_qk_norm_rope_axes_backward, 13)):
        assert f(None, 0, *[None] * (n + 1)) == INVALID
        assert f(None, 5, *[None] * (n + 1)) == SHAPE
        assert f(None, 3, *[None] * (n + 1)) == INVALID


def test_python_wants_cuda_tensors():
    torch = pytest.importorskip("torch")
    build.build_library()
    x = torch.zeros(4, 8)
    with pytest.raises(TypeError, match="X must be a CUDA matrix"):
        lin.lin_block_norms(x, x, None, None, None, x, None)
    with pytest.raises(TypeError, match="DX must be a CUDA matrix"):
        lin.lin_block_norms_backward(x, x, None, None, None, x, None, None, x, None, None, None)
    with pytest.raises(TypeError, match="params must be a list of tensors"):
        lin.lin_adamw(None, [], [], [])
    with pytest.raises(TypeError, match="params must be a list of tensors"):
        lin.lin_adamw(3, [], [], [])
    with pytest.raises(TypeError, match="params: contiguous float32 CUDA tensors"):
        lin.lin_adamw([x], [x], [x], [x])
    with pytest.raises(ValueError, match="grads must have 1 entries"):
        lin.lin_adamw([x], [], [x], [x])
    h = torch.zeros(4, 2, 8, dtype=torch.float16)
    with pytest.raises(TypeError, match="Q must be a CUDA tensor"):
        lin.lin_qk_norm_rope_axes(x, None, None, None, None, None, None, h, h, h)


def test_the_module_counts_its_arguments():
    pytest.importorskip("torch")
    build.build_library()
    calls = lin._short_calls()
    for f, n in ((calls.qk_norm_rope_axes, 13), (calls.qk_norm_rope_axes_backward, 16),
                 (calls.block_norms, 11), (calls.block_norms_backward, 16), (calls.adamw, 15)):
        with pytest.raises(TypeError, match=f"{n} arguments, not 1"):
            f(None)


# ---------------------------------------------------------------- scores of attention

class Heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class Shape(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("causal", ctypes.c_int32)] + \
        [(k, ctypes.c_int64) for k in ("tokens_q", "tokens_k", "heads_q", "heads_kv", "dim", "sequences",
                                       "max_q", "max_k")] + \
        [("cu_q", ctypes.c_void_p), ("cu_k", ctypes.c_void_p), ("scale", ctypes.c_float)]


class Form(ctypes.Structure):
    _fields_ = [("cap", ctypes.c_float), ("slopes", ctypes.c_void_p), ("first_key", ctypes.c_void_p),
                ("end_key", ctypes.c_void_p)]


def _scores(L, backward=False, scale=1.0, **form):
    s = Shape(0, 1, 16, 16, 2, 1, 64, 1, 16, 16, None, None, scale)
    t = [Heads(_at(i + 1), 2 * 64, 64) for i in range(8)]
    f = Form(**form)
    if backward:
        args = [*t[:4], _at(30), *t[4:]]
        return L.lin_attention_scores_backward(
            ctypes.byref(s), ctypes.byref(f), *(x if isinstance(x, int) else ctypes.byref(x) for x in args), None)
    return L.lin_attention_scores(ctypes.byref(s), ctypes.byref(f), *(ctypes.byref(x) for x in t[:4]), _at(30),
                                  None)


@pytest.mark.parametrize("backward", [False, True])
def test_scores_numbers(L, backward):
    for cap in (-1.0, float("nan"), float("inf"), float("-inf")):
        assert _scores(L, backward, cap=cap) == INVALID
    for cap, scale in ((4097.0, 1.0), (1e30, 1.0), (1e-38, 10.0), (2.0 ** -21, 1.0), (1e-38, 1e-38)):
        assert _scores(L, backward, scale=scale, cap=cap) == SHAPE
    for cap in (2.0 ** -20, 4096.0):
        assert _scores(L, backward, cap=cap) != SHAPE
    assert _scores(L, backward, scale=0.0, cap=1.0) == INVALID
    f = L.lin_attention_scores_backward if backward else L.lin_attention_scores
    assert f(None, None, *[None] * (10 if backward else 6)) == INVALID


def test_scores_python():
    torch = pytest.importorskip("torch")
    build.build_library()
    h = torch.zeros(4, 2, 8, dtype=torch.float16)
    with pytest.raises(TypeError, match="Q must be a CUDA tensor"):
        lin.lin_attention_scores(h, h, h, h, h, cap=3.0)
    with pytest.raises(TypeError, match="Q must be a CUDA tensor"):
        lin.lin_attention_scores_backward(h, h, h, h, h, h, h, h, h, cap=3.0)
    for f, n in ((lin._short_calls().attention_scores, 16), (lin._short_calls().attention_scores_backward, 20)):
        with pytest.raises(TypeError, match=f"{n} arguments, not 1"):
            f(None)
