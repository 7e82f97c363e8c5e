"""The paged-cache oracle against something other than itself."""
import numpy as np
import pytest
import torch

from oracle import attention as oatt
from oracle import paged as opg


def _paged(rng, rows, R, H, d, spare=2):
    """Contiguous rows [B][n][H][d] laid into shuffled pages."""
    B, n = rows.shape[:2]
    per = -(-n // R)
    ids = rng.permutation(B * per + spare)
    table = ids[:B * per].reshape(B, per)
    pool = rng.standard_normal((B * per + spare, R, H, d))
    for b in range(B):
        for r in range(n):
            pool[table[b, r // R], r % R] = rows[b, r]
    return pool, table


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_is_complex_multiplication(interleaved):
    rng = np.random.default_rng(0)
    x, pos, w = rng.standard_normal((5, 3, 16)), rng.integers(0, 10**6, 5), rng.uniform(0, 1, 4)
    y = opg.rope(x, pos, w, interleaved, 1.25)
    z = np.exp(1j * pos[:, None, None] * w) * 1.25
    pairs = (x[..., 0:8:2] + 1j * x[..., 1:8:2]) if interleaved else (x[..., :4] + 1j * x[..., 4:8])
    r = pairs * z
    got = (y[..., 0:8:2] + 1j * y[..., 1:8:2]) if interleaved else (y[..., :4] + 1j * y[..., 4:8])
    np.testing.assert_allclose(got, r, rtol=1e-9, atol=1e-9)
    np.testing.assert_array_equal(y[..., 8:], x[..., 8:])


def test_rope_scores_depend_on_distance_alone():
    rng = np.random.default_rng(1)
    q, k, w = rng.standard_normal((1, 1, 16)), rng.standard_normal((1, 1, 16)), rng.uniform(0, 1, 8)
    at = lambda i, j: float((opg.rope(q, [i], w, False, 1.0) * opg.rope(k, [j], w, False, 1.0)).sum())  # noqa: E731
    assert abs(at(100, 93) - at(7, 0)) < 1e-9


def test_attention_over_pages_is_tree_attention_over_rows():
    rng = np.random.default_rng(2)
    B, Kmax, Hq, Hkv, d, L = 2, 5, 4, 2, 8, 9
    Q = rng.standard_normal((B, Kmax, Hq, d))
    kv = [rng.standard_normal((B, L + Kmax, Hkv, d)) for _ in range(2)]
    mask = np.array([[1, 3, 5, 11, 16]] * B, np.uint64)
    (K, table), = [_paged(rng, kv[0], 4, Hkv, d)]
    V = np.zeros_like(K)
    for b in range(B):
        for r in range(L + Kmax):
            V[table[b, r // 4], r % 4] = kv[1][b, r]
    got = opg.attention(Q.reshape(-1, Hq, d), K, V, table, [L] * B, [0, Kmax, 2 * Kmax], 0.3, mask.reshape(-1))
    ref = oatt.tree_attention(Q, kv[0][:, :L], kv[1][:, :L], kv[0][:, L:], kv[1][:, L:], [L] * B, mask, 0.3)
    # sums of L + Kmax = 14 terms of order one, in 64 bits: each off by up to 14 * 2^-53 = 1.6e-15 absolutely,
    # however far the terms cancel
    np.testing.assert_allclose(got.reshape(ref.shape), ref, rtol=1e-12, atol=1e-14)


def test_causal_attention_is_torch_attention():
    rng = np.random.default_rng(3)
    n, Hq, Hkv, d = 7, 4, 2, 8
    q, k, v = rng.standard_normal((n, Hq, d)), rng.standard_normal((1, n, Hkv, d)), rng.standard_normal((1, n, Hkv, d))
    K, table = _paged(rng, k, 4, Hkv, d)
    V = np.zeros_like(K)
    for r in range(n):
        V[table[0, r // 4], r % 4] = v[0, r]
    got = opg.attention(q, K, V, table, [0], [0, n], d ** -0.5)
    t = lambda x: torch.from_numpy(x).transpose(0, 1)  # noqa: E731
    ref = torch.nn.functional.scaled_dot_product_attention(
        t(q), t(k[0]).repeat_interleave(2, 0), t(v[0]).repeat_interleave(2, 0), is_causal=True).transpose(0, 1)
    np.testing.assert_allclose(got, ref.numpy(), rtol=1e-10)


def test_a_row_that_sees_nothing_is_zero():
    out = opg.attention(np.ones((2, 1, 4)), np.ones((1, 16, 1, 4)), np.ones((1, 16, 1, 4)), [[0]], [0], [0, 2], 1.0,
                        np.array([0, 3], np.uint64))
    assert (out[0] == 0).all() and (out[1] == 1).all()


def test_pages_by_hand():
    # two sequences of 5 and 4 rows, pages of 4 rows, 8 pages
    P = opg.Pages([[3, 5] + [-1] * 4, [1] + [-1] * 5, [-1] * 6], [2, 1, 0], [5, 4, 0], [0, 1, 0, 1, 0, 1, 0, 0], 4)
    P.fork([0], [2])
    assert P.table[2][:3] == [3, 5, -1] and P.refs == [0, 1, 0, 2, 0, 2, 0, 0] and P.lengths[2] == 5
    copies, refused = P.reserve([0, 1, 4])
    # sequence 1 (full pages) takes page 0; sequence 2 replaces its shared page 5 by 2 and takes 4
    assert P.table[1][:3] == [1, 0, -1] and P.table[2][:4] == [3, 2, 4, -1]
    assert copies == [(5, 2, 1)] and not refused and P.refs == [1, 1, 1, 2, 1, 1, 0, 0]
    P.free([0, 0])
    assert P.refs == [1, 1, 1, 1, 1, 0, 0, 0] and P.held[0] == 0 and P.table[0] == [-1] * 6
    copies, refused = P.reserve([0, 20, 1])  # sequence 1 needs four pages, three are free
    assert refused == [1] and not copies


def test_compaction_by_hand():
    K = np.arange(1 * 2 * 4, dtype=float).reshape(1, 2, 4, 1, 1)
    k, v, n = opg.compact(K, K + 100, [[1, 0]], [2], [[0, 2, 5]], [3])
    # rows 2, 3, 4 receive rows 2, 4, 7
    assert k[0, 1, 2] == K[0, 1, 2] and k[0, 1, 3] == K[0, 0, 0] and k[0, 0, 0] == K[0, 0, 3] and n[0] == 5
    assert v[0, 0, 0] == 100 + K[0, 0, 3]


def test_a_sequence_whose_pages_behind_a_window_were_given_back_is_freed():
    P = opg.Pages([[2, -1, -1, 1], [0, 1, -1, -1]], [4, 2], [60, 20], [1, 2, 1], 16)
    P.free([0])
    assert P.refs == [1, 1, 0] and P.table[0] == [-1] * 4 and P.held == [0, 2] and P.lengths == [0, 20]
