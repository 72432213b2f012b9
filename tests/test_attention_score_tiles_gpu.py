"""lin_attention_scores where a CTA of the forward kernel has two tiles of
queries (more tiles than SMs), against the fp64 oracle with the bounds of
test_attention_scores_gpu.py, whose shapes mostly make one tile to a CTA."""

import numpy as np
import pytest

from tests.gpu_util import require_gpu
from tests.test_attention_scores_gpu import UNIT, _check, _form, _run, _setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _two_tiles(lens, hq, hk):
    """Fails unless the call has more tiles of 128 rows than the GPU has SMs (a
    tile holds the query heads of a key head where that makes no more of them)."""
    import torch
    longest = max(a for a, _ in lens)
    apart = -(-longest // 128) * hq * len(lens)
    packed = -(-longest // (128 // (hq // hk))) * hk * len(lens)
    assert min(apart, packed) > torch.cuda.get_device_properties(0).multi_processor_count


def _some(t, how, keep):
    """The tensors and the form of the key heads `keep` and their query heads
    (heads do not mix: the oracle is spared the others)."""
    group = t["q"].shape[1] // t["k"].shape[1]
    of_q = [h * group + i for h in keep for i in range(group)]
    part = {k: x[:, keep] if k in ("k", "v", "dk", "dv") else x[of_q] if k == "lse" else x[:, of_q]
            for k, x in t.items()}
    return part, dict(how, **({"slopes": how["slopes"][of_q]} if "slopes" in how else {}))


def _keys_by_tile(kind, lq, lk):
    """Ranges whose first keys differ from one tile of queries to the next."""
    at = np.arange(lq)
    if kind == "rising":      # a window: the second tile of a CTA begins a tile of keys later
        f = at * (lk - 60) // lq
        return f, f + 60
    if kind == "falling":     # the first tile is the late one
        f = (lk - 60) - at * (lk - 60) // lq
        return f, f + 60
    # one tile of queries at the first keys, the next at the last ones, with
    # tiles of keys between them that neither sees; "none": the early one sees nothing
    early = at // (64 if lq < 400 else 128) % 2 == (0 if kind != "first late" else 1)
    f = np.where(early, at % 5, lk - 100)
    e = np.where(early, 70 if kind != "none" else 0, lk - at % 7)
    return f, e


@pytest.mark.parametrize("kind", ["rising", "falling", "last late", "first late", "none"])
@pytest.mark.parametrize("name", ["ranges", "cap", "bias", "cap bias"])
@pytest.mark.parametrize("d, heads", [(64, (40, 40)), (96, (40, 40)), (128, (40, 40)), (128, (60, 30))])
def test_tiles_of_queries_whose_first_keys_differ(kind, name, d, heads):
    import torch
    lens = [(517, 901)] if heads[0] == heads[1] else [(390, 640)]
    _two_tiles(lens, *heads)
    how = _form(name, lens, heads[0], seed=20)
    how["first_key"], how["end_key"] = (torch.from_numpy(x.astype(np.int32)).cuda()
                                        for x in _keys_by_tile(kind, *lens[0]))
    dtype = "float16" if len(kind) % 2 else "bfloat16"
    t = _setup(dtype, lens, *heads, d, seed=d + heads[1], gain=2.0)
    _run(t, lens, False, d ** -0.5, how)
    part, form = _some(t, how, [0, heads[1] // 2, heads[1] - 1])
    _check(part, lens, False, d ** -0.5, form, UNIT[dtype])
    for k in ("o", "dq", "dk", "dv"):
        assert torch.isfinite(t[k]).all(), k
    want = {k: t[k].clone() for k in ("o", "lse", "dq", "dk", "dv")}
    _run(t, lens, False, d ** -0.5, how)
    for k in want:
        assert torch.equal(t[k], want[k]), k
