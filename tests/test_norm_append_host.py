"""Host-side checks of the normed append (no GPU needed)."""
import math

import pytest

from tests.helpers import gb
from tests.test_paged_host import BAD_CACHES, FAKE, cache


def call(c, N=4, Hq=32, starts=FAKE, freq=FAKE, rot=128, qw=FAKE, kw=FAKE, eps=1e-6, Q=FAKE, qs=4096, K=FAKE, ks=1024, V=FAKE,
         vs=1024, out=FAKE, os=4096, pool=FAKE):
    return gb().lib().graft_norm_rope_append(c, pool, FAKE, N, Hq, starts, None, freq, rot, 0, 1.0, qw, kw, eps, Q, qs, K, ks,
                                             V, vs, out, os, None)


@pytest.mark.parametrize("kw,rc", BAD_CACHES)
def test_bad_caches_are_refused(kw, rc):
    c, keep = cache(**kw)
    assert call(c) == rc


def test_arguments():
    c, keep = cache()
    for eps in (0.0, -1e-6, math.nan, math.inf, -math.inf):
        assert call(c, eps=eps) == -1 and call(c, eps=eps, qw=None) == -1 and call(c, eps=eps, kw=None) == -1
        assert call(c, eps=eps, N=0) == -1
    assert call(c, qw=FAKE + 2) == -1 and call(c, kw=FAKE + 1) == -1
    assert call(c, rot=24) == -2 and call(c, freq=None) == -1 and call(c, starts=None) == -1
    assert call(c, N=-1) == -1 and call(c, Hq=-1) == -1
    assert call(c, K=None) == -1 and call(c, V=None) == -1 and call(c, Q=None) == -1 and call(c, out=None) == -1
    assert call(c, ks=1016) == -1 and call(c, qs=100) == -1 and call(c, Q=FAKE + 8) == -1 and call(c, pool=None) == -1
    assert call(None) == -1
    assert call(c, N=0) == 0 and call(c, N=0, qw=None, kw=None, eps=-1.0) == 0
