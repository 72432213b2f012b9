"""The training operators in captured graphs that run at the same time, and
attention's forms at the ends of what their arguments may be. Bounds as in
test_attention_score_caps_gpu.py."""

import numpy as np
import pytest

from tests.gpu_util import require_gpu
from tests.test_attention_score_caps_gpu import _check
from tests.test_attention_scores_gpu import UNIT, _form, _run, _setup
from transformer_linear_layer_tcgen05_gb300 import lin

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _rope(seed):
    """(the calls, their results): rotation by axes, large enough that the angles
    are gathered into a workspace first."""
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    t, h, hk, d = 2100, 12, 2, 128
    x, w, angle = rnd(t, (h + 2 * hk) * d), 1 + 0.1 * rnd(d), rnd(50, d // 2)
    pos = torch.randint(0, 50, (3, t), generator=g, device="cuda", dtype=torch.int32)
    axis = torch.arange(d // 2, device="cuda", dtype=torch.int32) % 3
    heads = [torch.empty(t, n, d, device="cuda", dtype=torch.bfloat16) for n in (h, hk, hk)]
    out = [torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)]
    cos, sin = angle.cos(), angle.sin()

    def call():
        lin.lin_qk_norm_rope_axes(x, w, w, cos, sin, pos, axis, *heads)
        assert lin.lin_last_launch_info()[0] == 2   # (gathered)
        lin.lin_qk_norm_rope_axes_backward(x, w, w, cos, sin, pos, axis, *heads, *out)

    return call, heads + out


def _norms(seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    m, w = 1500, 1152
    x, y, gate, post, pre = rnd(m, w), rnd(m, w).half(), rnd(w), rnd(w), rnd(w)
    h, n = torch.empty_like(x), torch.empty_like(y)
    out = [torch.empty_like(t) for t in (x, y, gate, post, pre)]
    dh, dn = rnd(m, w), rnd(m, w).half()

    def call():
        lin.lin_block_norms(x, y, gate, post, pre, h, n)
        lin.lin_block_norms_backward(h, y, gate, post, pre, dh, dn, *out)

    return call, [h, n] + out


def _scores(seed):
    lens = [(700, 700)]
    t = _setup("float16", lens, 6, 2, 96, seed=seed)
    form = _form("cap bias docs", lens, 6, seed=seed)

    def call():
        lin.lin_attention_scores(t["q"], t["k"], t["v"], t["o"], t["lse"], **form)
        lin.lin_attention_scores_backward(*(t[k] for k in ("q", "k", "v", "o", "lse", "do", "dq", "dk", "dv")),
                                          **form)

    return call, [t[k] for k in ("o", "lse", "dq", "dk", "dv")]


@pytest.mark.parametrize("make", [_rope, _norms, _scores])
def test_two_captured_calls_at_the_same_time(make):
    # (each graph has workspace of its own)
    import torch
    (one, out1), (two, out2) = make(1), make(2)
    one(), two()
    torch.cuda.synchronize()
    want = [t.clone() for t in out1 + out2]
    graphs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for call in (one, two):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        graphs.append(graph)
    for t in out1 + out2:
        t.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    assert lin.lin_get_device_status() == lin.LIN_SUCCESS
    for got, w in zip(out1 + out2, want):
        assert torch.equal(got, w)


@pytest.mark.parametrize("kind", ["cap", "bias", "cap bias"])
@pytest.mark.parametrize("heads", [(32, 8), (5, 5), (7, 1)])
def test_one_query_on_many_keys(kind, heads):
    import torch
    lens = [(1, 8003)]
    dtype = "float16" if heads[1] == 8 else "bfloat16"
    t = _setup(dtype, lens, *heads, 128, seed=51, gain=3.0)
    form = _form(kind, lens, heads[0], seed=51)
    for first in (None, 7000, 8002, 8003):
        if first is not None:
            form["first_key"] = torch.tensor([first], dtype=torch.int32, device="cuda")
            form["end_key"] = torch.tensor([2 ** 31 - 1], dtype=torch.int32, device="cuda")
        _run(t, lens, True, 128 ** -0.5, form)
        _check(t, True, 128 ** -0.5, form, UNIT[dtype])


def test_ends_of_the_ranges():
    import torch
    lens, big = [(300, 257)], 2 ** 31
    t = _setup("bfloat16", lens, 4, 2, 64, seed=52)
    r = np.random.default_rng(52)
    ends = np.array([-big, -big + 1, -1, 0, 1, 127, 128, 129, 256, 257, 258, big - 2, big - 1], dtype=np.int64)
    for causal in (False, True):
        form = dict(cap=7.0)
        for k in ("first_key", "end_key"):
            form[k] = torch.from_numpy(r.choice(ends, 300).astype(np.int32)).cuda()
        _run(t, lens, causal, 0.125, form)
        _check(t, causal, 0.125, form, UNIT["bfloat16"])


def test_nothing_to_do():
    import torch
    for nq, nk in ((0, 0), (0, 40), (40, 0)):
        t = _setup("float16", [(nq, nk)], 2, 1, 64, seed=53)
        form = dict(cap=3.0, slopes=torch.ones(2, device="cuda"),
                    first_key=torch.zeros(nq, dtype=torch.int32, device="cuda"),
                    end_key=torch.full((nq,), 9, dtype=torch.int32, device="cuda"))
        _run(t, [(nq, nk)], False, 1.0, form)
        assert not t["o"].any() and not t["dq"].any() and not t["dk"].any() and not t["dv"].any()
        assert torch.isinf(t["lse"]).all()
