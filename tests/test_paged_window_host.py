"""Host-side checks of the windowed attention's entry points (no GPU needed)."""
import ctypes
import math

import pytest

from tests.helpers import gb
from tests.test_paged_host import BAD_CACHES, FAKE, cache


def attend(c, N=4, Hq=32, max_new=1, window=128, first=4, plan=FAKE, plan_bytes=1 << 30, Q=FAKE, stride=4096, mask=None,
           scale=0.1, O=FAKE, tuning=None, ws=FAKE, ws_bytes=1 << 40, K=FAKE, V=FAKE):
    return gb().lib().graft_paged_attention_window(c, K, V, N, Hq, max_new, window, first, plan, plan_bytes, Q, stride, mask,
                                                   scale, O, tuning, ws, ws_bytes, None)


def plan(c, N=4, Hq=32, starts=FAKE, max_new=1, tree=0, window=128, first=4, buf=FAKE, nbytes=1 << 30):
    return gb().lib().graft_paged_plan_window(c, N, Hq, starts, max_new, tree, window, first, buf, nbytes, None)


@pytest.mark.parametrize("kw,rc", BAD_CACHES)
def test_bad_caches_are_refused(kw, rc):
    c, keep = cache(**kw)
    assert attend(c) == rc and plan(c) == rc


def test_arguments():
    c, keep = cache()
    for window, first in ((0, 0), (-1, 0), (-2**31, 0), (5, -1), (5, -2**31)):
        assert attend(c, window=window, first=first) == -1 and plan(c, window=window, first=first) == -1
        assert attend(c, window=window, first=first, N=0) == -1
    assert attend(None) == -1 and plan(None) == -1
    assert attend(c, Hq=12) == -1 and plan(c, Hq=12) == -1
    assert attend(c, mask=FAKE, max_new=65) == -2 and plan(c, tree=1, max_new=65) == -2
    assert attend(c, stride=4095) == -1 and attend(c, Q=FAKE + 2) == -1 and attend(c, O=FAKE + 8) == -1
    assert attend(c, Q=None) == -1 and attend(c, O=None) == -1 and attend(c, K=None) == -1 and plan(c, starts=None) == -1
    assert attend(c, scale=0.0) == -1 and attend(c, scale=math.nan) == -1
    assert attend(c, plan=None) == -3 and attend(c, plan_bytes=64) == -3 and attend(c, ws=None) == -3
    assert plan(c, buf=None) == -3 and plan(c, nbytes=64) == -3 and plan(c, buf=FAKE + 16) == -3
    t = gb().GraftAttnTuning()
    t.tiles = 1
    assert attend(c, tuning=ctypes.addressof(t)) == -1
    assert attend(c, N=0) == 0 and attend(c, N=0, window=2**31 - 1, first=2**31 - 1) == 0


@pytest.mark.parametrize("window,first", [(True, 0), (0, 0), (-1, 0), (2**31, 0), (1.0, 0), (5, -1), (5, 2**31), (5, True),
                                          (None, 1)])
def test_the_handle_refuses(window, first):
    from tree_verification_gb300.paged import _kind
    with pytest.raises(ValueError):
        _kind(window, first)


def test_the_handle_takes():
    from tree_verification_gb300.paged import _kind
    assert _kind(None, 0) is None and _kind(1, 0) == (1, 0) and _kind(2**31 - 1, 2**31 - 1) == (2**31 - 1, 2**31 - 1)
