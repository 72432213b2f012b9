"""Gradients of attention over documents whose dO are of very different sizes:
what other documents hold does not show in a document's results. Bounds as in
test_attention_score_caps_gpu.py, which counts the steps of dS in binary16: the
others' dO has norms of some 2^11 here."""

import pytest

from tests.gpu_util import require_gpu
from tests.test_attention_score_caps_gpu import _check
from tests.test_attention_scores_gpu import UNIT, _form, _run, _setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _documents(layout, n):
    """first_key, end_key of documents that have tiles of 128 of their own, and
    which rows belong to the document that is looked at."""
    import torch
    at = torch.arange(n, dtype=torch.int32, device="cuda")
    if layout == "the first of three":
        cut = torch.where(at < 256, 0, torch.where(at < 640, 256, 640)).int()
        end = torch.where(at < 256, 256, torch.where(at < 640, 640, n)).int()
        return cut, end, at < 256
    if layout == "the last":
        return (at // 512 * 512).int(), torch.where(at < 512, 512, n).int(), at >= 512
    # "apart": its rows are the first and the last tiles, and see the first tile of keys
    own = (at < 128) | (at >= n - 128)
    return torch.where(own, 0, 128).int(), torch.where(own, 128, n).int(), own


@pytest.mark.parametrize("layout", ["the first of three", "the last", "apart"])
@pytest.mark.parametrize("form", ["ranges", "cap", "bias", "cap bias"])
@pytest.mark.parametrize("d, heads", [(64, (2, 1)), (128, (3, 3)), (96, (8, 2))])
def test_sizes_of_other_documents_gradients(d, heads, form, layout):
    # binary16, whose range is short: dO of the other documents 2^16 times as large
    import torch
    n = 768
    lens = [(n, n)]
    first, end, own = _documents(layout, n)
    how = dict(_form(form, lens, heads[0], seed=41), first_key=first, end_key=end)
    keys = own & (torch.arange(n, device="cuda") < 128) if layout == "apart" else own
    for causal in (False, True):
        t = _setup("float16", lens, *heads, d, seed=40 + d)
        t["do"].mul_(2.0 ** -8)
        _run(t, lens, causal, d ** -0.5, how)
        _check(t, causal, d ** -0.5, how, UNIT["float16"])
        want = {k: t[k].clone() for k in ("dq", "dk", "dv")}
        other = t["do"][~own].clone()
        # (infinities: of documents in tiles of their own, which "apart" is not)
        for gain in (2.0 ** 16, float("inf"))[:1 if layout == "apart" else 2]:
            t["do"][~own] = other * gain
            _run(t, lens, causal, d ** -0.5, how)
            assert torch.equal(t["dq"][own], want["dq"][own])
            assert torch.equal(t["dk"][keys], want["dk"][keys])
            assert torch.equal(t["dv"][keys], want["dv"][keys])
            if gain < 2.0 ** 20:
                _check(t, causal, d ** -0.5, how, UNIT["float16"])
