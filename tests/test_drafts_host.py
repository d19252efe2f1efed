"""The drafted-token operators, the parts that need no device: null arguments refused before
any device use, and the masks of trees.  CPU only."""
import ctypes

import numpy as np
import pytest

import paged_kv_cache_split_gb300 as pkv
from paged_kv_cache_split_gb300 import build as pkv_build

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib():
    pkv_build.build()
    return pkv.lib()


def test_null_pools(lib):
    n = ctypes.c_size_t()
    f = ctypes.c_float
    assert lib.pkv_write_rotated(None, 0, 1, None, None, None, 0, 0, None, 0, 0, None, None, 1, 64, 0, None, None, f(0), 0,
                                 None, 0, 0, None, 0, 0, None) == pkv.PKV_ERR_INVALID
    assert lib.pkv_tree_workspace_bytes(None, 1, 1, 1, ctypes.byref(n)) == pkv.PKV_ERR_INVALID
    assert lib.pkv_paged_tree_attention(None, 0, 1, 1, 1, None, None, 0, None, 1, None, 0, f(1), None, None, 0,
                                        None) == pkv.PKV_ERR_INVALID
    assert lib.pkv_accept_drafts(None, 1, 1, 1, None, None, None, 1, None, None, None) == pkv.PKV_ERR_INVALID


def ancestors(parents, i):
    seen = []
    while i >= 0:
        seen.append(i)
        i = parents[i]
    return seen


@pytest.mark.parametrize("n_q", [1, 2, 31, 32, 33, 64, 100])
def test_masks_of_trees(n_q):
    rng = np.random.default_rng(n_q)
    parents = np.array([[int(rng.integers(-1, i)) if i else -1 for i in range(n_q)] for _ in range(3)])
    masks, depths = pkv.tree_masks(parents)
    assert masks.shape == (3, n_q, -(-n_q // 32)) and masks.dtype == np.int32
    assert depths.shape == (3, n_q) and depths.dtype == np.int32
    for b in range(3):
        for i in range(n_q):
            up = ancestors(parents[b], i)
            bits = [j for j in range(32 * masks.shape[2]) if int(masks[b, i, j // 32]) >> (j % 32) & 1]
            assert bits == sorted(up) and depths[b, i] == len(up) - 1


def test_masks_of_one_tree_and_of_none():
    masks, depths = pkv.tree_masks([-1, 0, 0, -5])
    assert masks.tolist() == [[1], [3], [5], [8]] and depths.tolist() == [0, 1, 1, 0]
    masks, depths = pkv.tree_masks(np.zeros((2, 0), int))
    assert masks.shape == (2, 0, 0) and depths.shape == (2, 0)
    for bad in ([0], [-1, 1], [-1, 0, 5]):
        with pytest.raises(ValueError, match="before"):
            pkv.tree_masks(bad)
    with pytest.raises(TypeError):
        pkv.tree_masks([-1.0, 0.0])
