"""Which views ttt_rope takes, at the C boundary and without a GPU: outputs that share
memory with inputs, with each other, with the table or the positions are refused; slices of
one buffer that do not are taken.  The memory that a view touches is enumerated here."""
import ctypes
import itertools
import random

import numpy as np
import pytest
import torch

from test_sequence_layers_gb300 import abi, build

BASE = 1 << 30
TABLE, POS = 1 << 50, 1 << 51
REFUSED, NO_DEVICE = -1, -4


@pytest.fixture(scope="module")
def L():
    build.build()
    return abi.lib()


def _call(L, views, B, T, Hq, Hk, d, table=TABLE, positions=None):
    """views: (element offset, strides) of q, k, v, q_out, k_out, v_out, or None."""
    ptr = [None if v is None else BASE + 2 * v[0] for v in views]
    strides = [s for v in views for s in ((0, 0, 0) if v is None else v[1])]
    desc = abi.RopeDesc(B, T, Hq, Hk, d, d // 2 * 2, 0, 0, abi.TTT_BF16, T, 0, 0, T if positions else 0,
                        (ctypes.c_longlong * 18)(*strides))
    return L.ttt_rope(desc, *ptr[:3], table, positions, *ptr[3:], None)


def _refused(L, *a, **kw):
    assert _call(L, *a, **kw) == REFUSED


def _taken(L, *a, **kw):
    if torch.cuda.is_available():
        pytest.skip("made-up addresses: only where nothing can be launched")
    assert _call(L, *a, **kw) == NO_DEVICE


def _elements(v, B, H, T, d):
    i = np.indices((B, H, T, d)).reshape(4, -1)
    return v[0] + i[0] * v[1][0] + i[1] * v[1][1] + i[2] * v[1][2] + i[3]


FAR = 1 << 24


def test_a_shifted_output_over_another_tensors_input(L):
    """Rows 200 apart: k_out holds features 32 .. 95 of q's rows."""
    st = (200 * 8, 200 * 8, 200)
    _refused(L, [(0, st), (FAR, st), None, (2 * FAR, st), (32, st), None], 2, 8, 1, 1, 64)
    _refused(L, [(32, st), (FAR, st), None, (2 * FAR, st), (0, st), None], 2, 8, 1, 1, 64)
    _taken(L, [(0, st), (FAR, st), None, (2 * FAR, st), (64, st), None], 2, 8, 1, 1, 64)  # features 64 .. 127


def test_outputs_that_share_memory(L):
    st = (3 * 8 * 16, 8 * 16, 16)
    _refused(L, [(0, st), (FAR, st), None, (2 * FAR, st), (2 * FAR, st), None], 2, 8, 3, 3, 16)
    _refused(L, [(0, st), (FAR, st), (3 * FAR, st), (2 * FAR, st), (4 * FAR, st), (4 * FAR + 16, st)], 2, 8, 3, 3, 16)
    _taken(L, [(0, st), (FAR, st), None, (2 * FAR, st), (2 * FAR + 2 * 3 * 8 * 16, st), None], 2, 8, 3, 3, 16)


def test_table_and_positions(L):
    st = (3 * 8 * 16, 8 * 16, 16)
    v = [(0, st), None, None, (FAR, st), None, None]
    _refused(L, v, 2, 8, 3, 1, 16, table=BASE + 2 * FAR + 32)
    _refused(L, v, 2, 8, 3, 1, 16, positions=BASE + 2 * FAR)
    _refused(L, v, 2, 8, 3, 1, 16, positions=BASE + 2 * FAR - 8 * 16 + 8)
    _taken(L, v, 2, 8, 3, 1, 16, positions=POS)


def test_an_output_that_holds_elements_twice(L):
    std = (3 * 8 * 16, 8 * 16, 16)
    for st in ((3 * 8 * 16, 8 * 16, 15), (3 * 8 * 16 - 1, 8 * 16, 16), (16, 16, 3 * 32)):
        _refused(L, [(0, std), None, None, (FAR, st), None, None], 2, 8, 3, 1, 16)


@pytest.mark.parametrize("Hq,Hk", [(3, 3), (4, 1), (6, 2), (1, 1)])
def test_in_place_in_a_projection_buffer(L, Hq, Hk):
    """[B,T,Hq + 2 Hk,d]: every tensor is rotated where it stands."""
    B, T, d = 2, 9, 16
    n = Hq + 2 * Hk
    st = (T * n * d, d, n * d)
    v = [(0, st), (Hq * d, st), ((Hq + Hk) * d, st)]
    _taken(L, v + v, B, T, Hq, Hk, d)
    _refused(L, v + [v[0], v[2], v[1]], B, T, Hq, Hk, d)  # k and v trade places


def test_drawn_views(L):
    rng = random.Random(5)
    seen = {True: 0, False: 0}
    for _ in range(3000):
        B, T, H, d = rng.randint(1, 3), rng.randint(1, 4), rng.randint(1, 3), rng.randint(1, 5)
        order = list(itertools.permutations(range(3)))[rng.randrange(6)]
        n, st, step = (B, H, T), [0, 0, 0], d + rng.choice([0, 0, 1, 4, 7])
        for i in order:
            st[i] = step
            step = step * n[i] + rng.choice([0, 0, 3, 10, 25])
        q, k_out = (rng.randint(0, 2 * step), st), (rng.randint(0, 2 * step), st)
        views = [q, (FAR, st), None, (2 * FAR, st), k_out, None]
        both = bool(np.intersect1d(_elements(q, B, H, T, d), _elements(k_out, B, H, T, d)).size)
        seen[both] += 1
        (_refused if both else _taken)(L, views, B, T, H, H, d)
    assert min(seen.values()) > 500
