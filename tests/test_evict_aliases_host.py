"""Evictions whose arrays share memory are refused: their tokens would be moved twice at once."""
import ctypes

import pytest

from paged_kv_gqa_17_b200 import binding as bd

INVALID = -1
P = 256  # any aligned non-null address: these calls return before they use it


@pytest.fixture(scope="module")
def L():
    from paged_kv_gqa_17_b200 import build

    build.build()
    return bd.lib()


def evict(L, bases, row_bytes=256, positions=None, lens=P, new=2 * P, ws=1 << 20):
    shape = bd.make_shape(2, 8, 2, 128, 16, 4, 9)
    planes = (bd.Plane * len(bases))(*[bd.Plane(b, 16 * 512, 16 * 512, 512, row_bytes, 0) for b in bases])
    return L.pkv_evict_tokens(P, 64, 32, positions, 64, 32, planes, len(bases), P, lens, 4, 2, new, ctypes.byref(shape), P,
                              ws, None)


def test_planes_that_share_memory(L):
    a = 1 << 20
    assert evict(L, [a, a]) == INVALID
    assert evict(L, [a, 4 * a, a]) == INVALID
    assert evict(L, [a, a + 255]) == INVALID
    assert evict(L, [a + 16, a]) == INVALID


def test_scores_given_as_positions(L):
    assert evict(L, [1 << 20], positions=P) == INVALID


def test_new_lengths_over_the_old_ones(L):
    assert evict(L, [1 << 20], lens=P, new=P + 4) == INVALID
    assert evict(L, [1 << 20], lens=P + 4, new=P) == INVALID
    assert evict(L, [1 << 20], lens=P, new=P + 8, ws=100) == -3  # two rows, side by side: on to the workspace's size
