"""Which views of shared memory the attention entry points take and which they
refuse as overlapping, against the sets of their entries (CPU only: fake,
never-dereferenced addresses, refused or accepted before any CUDA call; an
accepted call then fails at the device checks)."""

import ctypes
import itertools
import random

import pytest

from transformer_linear_layer_tcgen05_gb300 import build, lin


class Heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class Shape(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("causal", ctypes.c_int32),
                ("tokens_q", ctypes.c_int64), ("tokens_k", ctypes.c_int64),
                ("heads_q", ctypes.c_int64), ("heads_kv", ctypes.c_int64),
                ("dim", ctypes.c_int64), ("sequences", ctypes.c_int64),
                ("max_q", ctypes.c_int64), ("max_k", ctypes.c_int64),
                ("cu_q", ctypes.c_void_p), ("cu_k", ctypes.c_void_p), ("scale", ctypes.c_float)]


BASE = 1 << 40
FAR = [BASE + (i << 30) for i in range(1, 6)]


@pytest.fixture(scope="module")
def L():
    build.build_library()
    return lin.lib()


def _status(L, q, k, tokens_q, tokens_k, heads_q, heads_kv, dim, o):
    """lin_attention's status for O at `o`, Q at `q` and K at `k` (entries from
    BASE, token stride, head stride); V and LSE lie far away."""
    s = Shape(0, 0, tokens_q, tokens_k, heads_q, heads_kv, dim, 1, tokens_q, tokens_k, None, None,
              1.0)
    at = lambda v: ctypes.byref(Heads(BASE + 2 * v[0], v[1], v[2]))  # noqa: E731
    v = Heads(FAR[0], heads_kv * dim, dim)
    return L.lin_attention(ctypes.byref(s), at(q), at(k), ctypes.byref(v), at(o), FAR[1], None)


def _entries(v, tokens, heads, dim):
    """The 8-entry units of a view (starts, strides and dim are multiples of 8)."""
    return {(v[0] + i * v[1] + j * v[2]) // 8 + u
            for i, j, u in itertools.product(range(tokens), range(heads), range(dim // 8))}


def _stride_pair(r, tokens, heads, dim):
    """Strides of a valid view: either side inner, with room or without."""
    room = lambda: 8 * r.choice([0, 0, 1, 3, dim // 8, dim // 4])  # noqa: E731
    if r.random() < 0.5:
        hs = dim * r.choice([1, 1, 2, 3]) + room()
        return hs * (heads - 1) + dim + room(), hs
    ts = dim * r.choice([1, 1, 2, 3]) + room()
    return ts, ts * (tokens - 1) + dim + room()


def test_interleaved_views_of_one_buffer(L):
    t, h, d = 90, 3, 64
    far = (1 << 32, h * d, d)
    for ts, hs in ((h * 3 * d, 3 * d), (3 * d, t * 3 * d)):   # [tokens, heads, 3, dim], heads first
        q, k, o = (0, ts, hs), (d, ts, hs), (2 * d, ts, hs)
        for a, b in itertools.permutations((q, k, o), 2):
            assert _status(L, a, b, t, t, h, h, d, far) != lin.LIN_ERROR_ALIASING
            assert _status(L, a, far, t, t, h, h, d, b) != lin.LIN_ERROR_ALIASING
            assert _status(L, far, a, t, t, h, h, d, b) != lin.LIN_ERROR_ALIASING
        # half a head further they share entries
        assert _status(L, q, far, t, t, h, h, d, (d // 2, ts, hs)) == lin.LIN_ERROR_ALIASING


def test_overlaps_are_the_shared_entries(L):
    # equal strides: refused just where an entry is shared; other strides: at
    # least there
    r = random.Random(7)
    far = (1 << 32, 4096, 256)
    seen = {True: 0, False: 0}
    for _ in range(4000):
        tokens, heads, dim = r.choice([1, 2, 3, 5]), r.choice([1, 2, 3, 4]), r.choice([8, 16, 24])
        ts, hs = _stride_pair(r, tokens, heads, dim)
        q = (8 * r.randrange(0, 60), ts, hs)
        same = r.random() < 0.7
        o = (8 * r.randrange(0, 60), *((ts, hs) if same else _stride_pair(r, tokens, heads, dim)))
        shared = bool(_entries(q, tokens, heads, dim) & _entries(o, tokens, heads, dim))
        refused = _status(L, q, far, tokens, 4, heads, heads, dim, o) == lin.LIN_ERROR_ALIASING
        assert refused or not shared, (tokens, heads, dim, q, o)
        if same:
            assert refused == shared, (tokens, heads, dim, q, o)
            seen[shared] += 1
    assert min(seen.values()) > 300


def test_overlaps_of_tensors_of_other_extents(L):
    # K beside O: other numbers of tokens and heads over the same strides
    r = random.Random(8)
    seen = {True: 0, False: 0}
    for _ in range(4000):
        tokens, heads_kv, dim = r.choice([1, 2, 3, 5]), r.choice([1, 2]), r.choice([8, 16])
        tokens_k, heads = r.choice([1, 2, 4, 6]), heads_kv * r.choice([1, 2, 3])
        ts, hs = _stride_pair(r, max(tokens, tokens_k), heads, dim)
        far = (1 << 32, heads * dim, dim)
        k, o = (8 * r.randrange(0, 60), ts, hs), (8 * r.randrange(0, 60), ts, hs)
        shared = bool(_entries(k, tokens_k, heads_kv, dim) & _entries(o, tokens, heads, dim))
        refused = _status(L, far, k, tokens, tokens_k, heads, heads_kv, dim, o) == \
            lin.LIN_ERROR_ALIASING
        assert refused == shared, (tokens, tokens_k, heads, heads_kv, dim, k, o)
        seen[shared] += 1
    assert min(seen.values()) > 300
