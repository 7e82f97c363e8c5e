"""Host-side checks of graft_token_logprobs (no GPU needed): refusals and sizes."""
import ctypes
import math

import pytest
import torch

from tests.helpers import gb

FAKE = 0x10000  # never dereferenced: every call below fails a host check first, or launches nothing


def call(N=4, V=100, R=4, dtype=2, logits=FAKE, stride=100, rows=None, block=0, tokens=FAKE, T=1.0, top=2, lp=FAKE, H=FAKE,
         rank=FAKE, ids=FAKE, lps=FAKE, ws=FAKE, ws_bytes=1 << 40):
    return gb().lib().graft_token_logprobs(N, V, R, dtype, logits, stride, rows, block, tokens, T, top, lp, H, rank, ids, lps,
                                           None, ws, ws_bytes, None)


def test_arguments():
    assert call(N=0) == 0
    assert call(N=-1) == -1 and call(V=0, top=0) == -1 and call(top=-1) == -1 and call(V=1, top=2, stride=1) == -1
    assert call(N=65536, R=65536) == -2 and call(top=33) == -2 and call(V=(1 << 24) + 1, stride=1 << 25) == -2
    assert call(dtype=3) == -1 and call(dtype=-1) == -1
    for T in (0.0, -1.0, math.nan, math.inf, 1e-39, -1e-39):
        assert call(T=T) == -1
    assert call(logits=None) == -1 and call(tokens=None) == -1 and call(lp=None) == -1
    assert call(ids=None) == -1 and call(lps=None) == -1
    assert call(R=3) == -1 and call(R=-1) == -1 and call(block=4) == -1 and call(rows=FAKE, block=-1) == -1
    assert call(R=1 << 31) == -2
    assert call(stride=99) == -1 and call(stride=1 << 41) == -1
    assert call(logits=FAKE + 2) == -1 and call(logits=FAKE + 1, dtype=0) == -1
    assert call(ws=None) == -3 and call(ws=FAKE + 16) == -3 and call(ws_bytes=64) == -3


def test_workspace_sizes():
    n, size = ctypes.c_size_t(), gb().graft_token_logprobs_workspace_size
    assert gb().lib().graft_token_logprobs_workspace_size(4, 100, 2, None) == -1
    assert gb().lib().graft_token_logprobs_workspace_size(4, 100, 101, ctypes.byref(n)) == -1
    assert gb().lib().graft_token_logprobs_workspace_size(4, 100, 33, ctypes.byref(n)) == -2
    assert 0 < size(4, 100, 0) < size(4, 100, 20) < size(1000, 100, 20)


def test_the_binding_refuses_what_it_cannot_take():
    f = gb().graft_token_logprobs
    x, t = torch.zeros(4, 10), torch.zeros(4, dtype=torch.int32)
    for bad in (x, x[0], x.double(), None):  # on the host, of one dimension, of another type, nothing
        with pytest.raises((ValueError, TypeError)):
            f(bad, t)
