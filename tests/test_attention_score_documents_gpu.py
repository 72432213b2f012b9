"""Gradients of attention over documents whose dO are of very different sizes:
what other documents hold does not show in a document's results. Bounds as in
test_attention_score_caps_gpu.py, which counts the steps of dS in binary16: the
others' dO has norms of some 2^11 here."""

import pytest

from tests.gpu_util import require_gpu
from tests.test_attention_score_caps_gpu import _check
from tests.test_attention_score_tiles_gpu import _two_tiles
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


@pytest.mark.parametrize("kind", ["cap", "cap bias", "bias", "ranges"])
@pytest.mark.parametrize("d, heads", [(64, (45, 45)), (96, (90, 30)), (128, (45, 45))])
@pytest.mark.parametrize("aligned", [True, False])
def test_what_the_mask_hides_does_not_show_in_two_tiles_to_a_cta(aligned, d, heads, kind):
    # one document's queries, keys, values and dO changed: the others' results are
    # the same bits; dK in binary16, whose scale is a tile's, where the documents
    # have tiles of their own
    import torch
    n = 500
    lens = [(n, n)]
    _two_tiles(lens, *heads)
    at = torch.arange(n, dtype=torch.int32, device="cuda")
    cuts = torch.tensor([0, 128, 384, n] if aligned else [0, 61, 130, 199, n], dtype=torch.int32, device="cuda")
    doc = torch.searchsorted(cuts, at, right=True)
    form = dict(_form(kind, lens, heads[0], seed=43), first_key=cuts[doc - 1].contiguous(),
                end_key=cuts[doc].contiguous())
    if "cap" in kind:
        form["cap"] = 20.0
    a, b = (128, 384) if aligned else (130, 199)
    rest = torch.cat([at[:a], at[b:]]).long()
    for dtype in ("float16", "bfloat16"):
        t = _setup(dtype, lens, *heads, d, seed=43, gain=3.0)
        same = ["o", "dq", "dv"] + (["dk"] if aligned or dtype == "bfloat16" else [])
        want = None
        for gain, of_do in ((1.0, 1.0), (7.0, 2.0 ** 10), (0.0, 2.0 ** -12), (1.0, 0.0)):
            for name in ("q", "k", "v"):
                t[name][a:b] = gain * t[name][a:b].flip(0)
            t["do"][a:b] = of_do * t["do"][a:b].flip(0)
            _run(t, lens, True, d ** -0.5, form)
            got = {k: t[k][rest].clone() for k in same}
            got["lse"] = t["lse"][:, rest].clone()
            want = want or got
            for k in want:
                assert torch.equal(got[k], want[k]), (k, dtype, gain)


@pytest.mark.parametrize("kind", ["cap", "cap bias", "bias"])
@pytest.mark.parametrize("d, heads", [(64, (2, 2)), (64, (45, 45)), (96, (90, 30)), (128, (3, 1))])
def test_other_queries_do_not_show(kind, d, heads):
    # later keys of larger scores: a row's running maximum grows, or not, whatever
    # those of the rows beside it do
    import torch
    lens = [(420, 420)]
    form = _form(kind, lens, heads[0], seed=45)
    if "cap" in kind:
        form["cap"] = 100.0
    for dtype in ("float16", "bfloat16"):
        t = _setup(dtype, lens, *heads, d, seed=45, gain=0.5)
        t["k"][128:256] *= 3
        t["k"][256:] *= 9
        want = None
        for gain in (1.0, 30.0, 1 / 64):
            t["q"][::2] *= gain
            _run(t, lens, False, d ** -0.5, form)
            got = {k: t[k][1::2].clone() for k in ("o", "dq")}
            got["lse"] = t["lse"][:, 1::2].clone()
            want = want or got
            for k in want:
                assert torch.equal(got[k], want[k]), (k, dtype, gain)


def test_rows_of_a_tile_that_are_nobodys():
    # (three heads to a tile: two of its 128 rows hold what was in shared memory;
    # calls between bring other contents there)
    import torch
    n, heads = 500, (90, 30)
    lens = [(n, n)]
    _two_tiles(lens, *heads)
    form = _form("docs", lens, heads[0], seed=46)
    other = _setup("bfloat16", lens, *heads, 96, seed=47, gain=100.0)
    t = _setup("bfloat16", lens, *heads, 96, seed=46, gain=3.0)
    t["k"][200:] *= 5
    _run(t, lens, False, 0.1, form)
    want = {k: t[k].clone() for k in ("o", "lse", "dq", "dk", "dv")}
    for _ in range(5):
        _run(other, lens, False, 3.0, form)
        _run(t, lens, False, 0.1, form)
        for k in want:
            assert torch.equal(t[k], want[k]), k
        other["q"].mul_(-1.5)
