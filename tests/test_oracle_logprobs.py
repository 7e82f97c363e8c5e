"""The log-probability oracle against something other than itself."""
import numpy as np
import pytest
import torch

from oracle import logprobs as olp


@pytest.mark.parametrize("T", [1.0, 0.6, 2.0])
def test_law_is_torch_log_softmax(T):
    rng = np.random.default_rng(0)
    x = rng.normal(size=(4, 300)) * 5
    x[1, 40:] = -np.inf
    ref = torch.log_softmax(torch.from_numpy(x) / T, 1).numpy()
    law = torch.distributions.Categorical(logits=torch.from_numpy(np.where(np.isinf(x), -1e300, x)) / T)
    for i in range(4):
        lp, h, rank, ids, lps = olp.row(x[i], 7, 5, T)
        assert lp == pytest.approx(ref[i, 7], rel=1e-12)
        assert h == pytest.approx(law.entropy()[i].item(), rel=1e-10)
        best = sorted(range(300), key=lambda v: (-x[i, v], v))
        assert ids.tolist() == best[:5] and best[rank] == 7
        np.testing.assert_allclose(lps, ref[i, best[:5]], rtol=1e-12)


def test_by_hand():
    # p = (1/2, 1/4, 1/4)
    lp, h, rank, ids, lps = olp.row(np.log([2.0, 1.0, 1.0]), 2, 3)
    np.testing.assert_allclose([lp, h], [np.log(0.25), 1.5 * np.log(2)])
    assert rank == 2 and ids.tolist() == [0, 1, 2]
    np.testing.assert_allclose(lps, np.log([0.5, 0.25, 0.25]))


def test_equal_logits_and_none():
    lp, h, rank, ids, _ = olp.row(np.zeros(10), 4, 3)
    assert rank == 4 and ids.tolist() == [0, 1, 2] and lp == pytest.approx(-np.log(10)) and h == pytest.approx(np.log(10))
    assert olp.row(np.zeros(10), -1, 0)[0] == 0 and olp.row(np.zeros(10), -1, 0)[2] == -1


def test_rows_without_a_law():
    for x in ([0.0, np.nan, 1.0], [np.inf, 0.0, 1.0], [-np.inf] * 3):
        lp, h, _, ids, lps = olp.row(np.array(x), 0, 3)
        assert np.isnan(lp) and np.isnan(h) and np.isnan(lps).all()
    assert olp.row(np.array([0.0, np.nan, 1.0, -np.inf]), 0, 4)[3].tolist() == [2, 0, 1, 3]


def test_rows_and_blocks():
    x = np.arange(24.0).reshape(6, 4) % 5
    got = olp.tokens(x, [1, 2, -1, 3, 0, 1], rows=[0, 2, -1, 1, 0, -1], block=3, top=1)
    ref = [olp.row(x[0], 1, 1), olp.row(x[2], 2, 1), None, olp.row(x[4], 3, 1), olp.row(x[3], 0, 1), None]
    for i, r in enumerate(ref):
        if r is None:
            assert got["rank"][i] == -1 and got["top_id"][i, 0] == -1 and got["entropy"][i] == 0
        else:
            assert got["logprob"][i] == r[0] and got["rank"][i] == r[2] and got["top_id"][i, 0] == r[3][0]


def test_ranks_beside_nan():
    # NaN ranks with -inf: a token's rank is its place among the alternatives
    for x in ([0.0, np.nan, 1.0, -np.inf], [np.nan] * 4, [-np.inf, np.nan, -np.inf, 2.0], [np.nan, np.inf, -np.inf, np.inf]):
        ids = olp.row(np.array(x), 0, 4)[3].tolist()
        assert [olp.row(np.array(x), v, 0)[2] for v in ids] == [0, 1, 2, 3]
    assert [olp.row(np.array([0.0, np.nan, 1.0, -np.inf]), v, 0)[2] for v in range(4)] == [1, 2, 0, 3]
