"""Head norms and windows of the paged oracle against something other than itself."""
import numpy as np
import pytest
import torch

from oracle import paged as opg


def test_head_norm_is_torch_rms_norm():
    rng = np.random.default_rng(0)
    x, w = rng.standard_normal((5, 3, 16)), rng.standard_normal(16)
    ref = torch.nn.functional.rms_norm(torch.from_numpy(x), (16,), torch.from_numpy(w), 1e-5)
    np.testing.assert_allclose(opg.head_norm(x, w, 1e-5), ref.numpy(), rtol=1e-13)
    assert opg.head_norm(x, None, 1e-5) is not None and np.array_equal(opg.head_norm(x, None, 1e-5), x)


def test_a_normed_head_has_the_weights_size():
    x = np.array([[[3.0, 4.0, 0.0, 0.0]]])  # mean square 25 / 4
    np.testing.assert_allclose(opg.head_norm(x, [2, 2, 2, 2], 0.0), [[[2.4, 3.2, 0, 0]]])


def _linear(rng, n, d=8, R=4):
    pool = rng.standard_normal((2, -(-n // R), R, 1, d))
    return pool[0], pool[1], [list(range(pool.shape[1]))]


@pytest.mark.parametrize("window,first", [(1, 0), (3, 0), (3, 2), (5, 1), (100, 0), (2, 100)])
def test_windowed_causal_attention_is_masked_torch_attention(window, first):
    rng = np.random.default_rng(window + first)
    L, n, d = 6, 5, 8
    K, V, table = _linear(rng, L + n)
    q = rng.standard_normal((n, 1, d))
    got = opg.attention(q, K, V, table, [L], [0, n], 0.4, window=window, first=first)
    keep = torch.zeros(n, L + n, dtype=torch.bool)
    for i in range(n):
        for r in range(L + i + 1):
            keep[i, r] = L + i - r < window or r < first
    k, v = (torch.from_numpy(x.reshape(-1, d)[:L + n]) for x in (K, V))
    ref = torch.nn.functional.scaled_dot_product_attention(torch.from_numpy(q[:, 0]), k, v, attn_mask=keep, scale=0.4)
    np.testing.assert_allclose(got[:, 0], ref.numpy(), rtol=1e-10)


@pytest.mark.parametrize("window,first", [(1, 0), (2, 0), (3, 1), (4, 8), (50, 0)])
def test_a_chain_tree_sees_what_causal_rows_see(window, first):
    rng = np.random.default_rng(3)
    L, n = 7, 6
    K, V, table = _linear(rng, L + n)
    q = rng.standard_normal((n, 1, 8))
    chain = np.array([(1 << i + 1) - 1 for i in range(n)], np.uint64)
    np.testing.assert_array_equal(opg.attention(q, K, V, table, [L], [0, n], 0.4, chain, window=window, first=first),
                                  opg.attention(q, K, V, table, [L], [0, n], 0.4, window=window, first=first))


def test_a_tree_counts_depths_by_hand():
    # node 2 hangs below node 0, beside node 1: depth 1, position L + 1; window 2: itself and node 0 alone
    rng = np.random.default_rng(4)
    K, V, table = _linear(rng, 8)
    q = rng.standard_normal((3, 1, 8))
    got = opg.attention(q, K, V, table, [4], [0, 3], 0.4, np.array([1, 3, 5], np.uint64), window=2)
    k, v = K.reshape(-1, 8), V.reshape(-1, 8)
    for i, seen in enumerate(([3, 4], [4, 5], [4, 6])):
        s = np.exp(k[seen] @ q[i, 0] * 0.4)
        np.testing.assert_allclose(got[i, 0], s @ v[seen] / s.sum(), rtol=1e-12)
    # a row without a bit stands at position L: its window holds rows 3 and (its own, which it does not see) 4
    none = opg.attention(q[:1], K, V, table, [4], [0, 1], 0.4, np.array([0], np.uint64), window=2)
    np.testing.assert_allclose(none[0, 0], v[3], rtol=1e-12)


def test_a_wide_window_is_none():
    rng = np.random.default_rng(5)
    K, V, table = _linear(rng, 11)
    q = rng.standard_normal((4, 1, 8))
    np.testing.assert_array_equal(opg.attention(q, K, V, table, [7], [0, 4], 0.4, window=11),
                                  opg.attention(q, K, V, table, [7], [0, 4], 0.4))
