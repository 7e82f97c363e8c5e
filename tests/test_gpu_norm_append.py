"""Norms of queries and keys in the pass that rotates and appends, against the oracle on the GPU."""
import numpy as np
import pytest
import torch

from oracle import paged as opg
from tests.helpers import gb
from tests.test_gpu_paged import HALF, Setup, np64

pytestmark = pytest.mark.gpu
DEV = "cuda"


def run(s, G, rot, interleaved, norms="both", factor=1.0, pos=None, pad=0, eps=1e-6, size=1.0, stride=0):
    N, H = int(s.starts[-1]) + pad, s.Hkv
    Hq = H * G
    w = 10000.0 ** (-np.arange(rot // 2) * 2 / max(rot, 1))
    x = torch.zeros(N, Hq + 2 * H + stride, 128, dtype=s.dtype)
    # heads of unlike size
    x[:, :Hq + 2 * H] = (s.randn(N, Hq + 2 * H, 128).float() * size * torch.exp(torch.randn(Hq + 2 * H, 1, generator=s.g))).to(s.dtype)
    x = x.to(DEV)
    Q, K, V = x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:Hq + 2 * H]
    qw, kw = (1 + 0.5 * torch.randn(128, generator=s.g) for _ in range(2))
    qw, kw = (qw if norms != "k" else None), (kw if norms != "q" else None)
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    out = torch.full((N, Hq, 128), 7.0, dtype=s.dtype, device=DEV)
    got = s.cache.append(0, Q, K, V, s.q_start, inv_freq=torch.from_numpy(w).to(DEV) if rot else None,
                         interleaved=interleaved, positions=None if pos is None else s.i32(pos), factor=factor, out=out,
                         q_norm=dev(qw), k_norm=dev(kw), eps=eps)
    assert got is out and s.status() == 0
    live = int(s.starts[-1])
    row = np.concatenate([np.arange(n) + L for n, L in zip(s.new, s.lens)])
    at = row if pos is None else np.asarray(pos)[:live]
    want_k, want_v, tol_k = np64(s.K0[0]), np64(s.V0[0]), np.zeros(s.K0[0].shape)
    b = np.repeat(np.arange(len(s.new)), s.new)
    for x, weight, y in ((Q, qw, out), (K, kw, None)):
        x = opg.head_norm(np64(x)[:live], None if weight is None else weight.numpy(), eps)
        ref = opg.rope(x, at, w, interleaved, factor)
        # half a step of the result; 32-bit cosines and products of the pair (2^-20 of the largest); and the norm: a
        # sum of 128 squares in at most 20 roundings a term, halved by the root, its inverse to 2 ulp, two products:
        # 10 * 2^-24 + 2^-22 + 2^-23 < 2^-20
        tol = HALF[s.dtype] * np.abs(ref) + 2.0 ** -19 * factor * np.abs(x).max(-1, keepdims=True)
        if weight is None:
            tol = HALF[s.dtype] * np.abs(ref) + 2.0 ** -20 * factor * np.abs(x).max()
            tol[..., rot:] = 0
        if y is not None:
            assert (np.abs(np64(y)[:live] - ref) <= tol).all()
        else:
            for i in range(live):
                p, x_ = s.table[b[i], row[i] // s.page], row[i] % s.page
                want_k[p, x_], tol_k[p, x_], want_v[p, x_] = ref[i], tol[i], np64(V)[i]
    assert bool((out[live:] == 7).all())
    got_k, got_v = np64(s.K[0]), np64(s.V[0])
    assert np.array_equal(np.isnan(got_k), np.isnan(want_k)) and np.array_equal(got_v, want_v, equal_nan=True)
    assert (np.nan_to_num(np.abs(got_k - want_k)) <= tol_k).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [0, 16, 32, 96, 128])
def test_norm_append(dtype, interleaved, rot):
    s = Setup([5, 0, 100, 31, 64], [3, 1, 0, 2, 5], 2, 16, dtype, seed=rot)
    run(s, 3, rot, interleaved, factor=1.1, pad=3)


@pytest.mark.parametrize("norms", ["q", "k"])
@pytest.mark.parametrize("rot,interleaved", [(0, False), (64, False), (128, True)])
def test_one_norm_alone(norms, rot, interleaved):
    run(Setup([5, 0, 100], [3, 1, 7], 2, 32, torch.float16, seed=rot), 4, rot, interleaved, norms=norms)


@pytest.mark.parametrize("Hkv,G,page,new", [(8, 4, 64, [64]), (4, 16, 128, [7, 9]), (1, 1, 256, [1, 1, 1]), (5, 3, 32, [33]),
                                            (8, 16, 16, [3])])
def test_norm_append_heads(Hkv, G, page, new):
    run(Setup([77] * len(new), new, Hkv, page, seed=G), G, 128, False, stride=1)


@pytest.mark.parametrize("eps,size", [(1e-6, 1e-3), (1e-5, 1e-6), (1e-12, 30.0), (0.5, 1.0)])
def test_sizes_of_eps_and_elements(eps, size):
    run(Setup([9], [6], 2, 16, seed=3), 2, 128, False, eps=eps, size=size)


def test_norm_append_of_rows_that_fill_waves():
    wave = 5 * torch.cuda.get_device_properties(0).multi_processor_count
    for N in (wave, wave + 1, 3 * wave, 3 * wave + 1):
        new = [N // 3 + 1, 0, 5, N - N // 3 - 6]
        run(Setup([7, 3, 40, 0], new, 1, 64, seed=N % 97), 1, 32, False, pad=2)


def test_positions_of_a_tree_and_in_place():
    s = Setup([40, 9], [4, 3], 2, 16, seed=3)
    run(s, 2, 128, False, pos=[40, 41, 41, 42, 9, 10, 10])
    Q, K = s.randn(7, 4, 128).to(DEV), s.randn(7, 2, 128).to(DEV)
    w = torch.from_numpy(10000.0 ** (-np.arange(64) / 64)).to(DEV)
    qw = torch.randn(128, device=DEV)
    out = s.cache.append(0, Q.clone(), K, K, s.q_start, inv_freq=w, q_norm=qw, k_norm=qw)
    q2 = Q.clone()
    assert s.cache.append(0, q2, K, K, s.q_start, inv_freq=w, out=q2, q_norm=qw, k_norm=qw) is q2
    assert s.status() == 0 and torch.equal(out, q2)


def test_heads_of_zeros_infinities_and_nan():
    s = Setup([9], [3], 2, 16, seed=5)
    Q, K = s.randn(3, 4, 128), s.randn(3, 2, 128)
    Q[0, 1] = 0
    Q[1, 2, 7] = float("nan")
    K[2, 0, 3] = float("inf")
    one = torch.ones(128, device=DEV)
    out = s.cache.append(0, Q.to(DEV), K.to(DEV), K.to(DEV), s.q_start, q_norm=one, k_norm=one)
    got = np64(out)
    with np.errstate(invalid="ignore"):
        ref = opg.head_norm(np64(Q), np.ones(128), 1e-6)
    assert (got[0, 1] == 0).all() and np.isnan(got[1, 2]).all() and np.isfinite(got).sum() == got.size - 128
    fine = np.isfinite(ref)
    assert (np.abs(got - ref)[fine] <= 2.0 ** -8 * np.abs(ref)[fine] + 2.0 ** -18).all()
    k = np64(s.K[0])[s.table[0, 0], 11]
    assert np.isnan(k[0, 3]) and (np.delete(k[0], 3) == 0).all() and np.isfinite(k[1]).all()


def test_append_without_weights_is_append():
    a, b = (Setup([30, 4], [5, 2], 2, 16, seed=8) for _ in range(2))
    Q, K, V = (a.randn(7, h, 128).to(DEV) for h in (4, 2, 2))
    w = torch.from_numpy(10000.0 ** (-np.arange(64) / 64)).to(DEV)
    x = a.cache.append(0, Q, K, V, a.q_start, inv_freq=w)
    y = b.cache.append(0, Q, K, V, b.q_start, inv_freq=w, q_norm=None, k_norm=None, eps=-1.0)
    assert torch.equal(x, y) and torch.equal(a.K.view(torch.int16), b.K.view(torch.int16))


def test_idle_sequences_and_keys_alone():
    s = Setup([30, 20], [2, 3], 2, 16, seed=9)
    K, V, kw = s.randn(5, 2, 128), s.randn(5, 2, 128), torch.rand(128, generator=s.g)
    on = torch.tensor([False, True], device=DEV)
    assert s.cache.append(0, None, K.to(DEV), V.to(DEV), s.q_start, k_norm=kw.to(DEV), active=on) is None
    assert s.status() == 0
    ref = opg.head_norm(np64(K), kw.numpy(), 1e-6)
    got, want = np64(s.K[0]), np64(s.K0[0])
    for i, r in enumerate((20, 21, 22)):
        p = s.table[1, r // 16], r % 16
        assert (np.abs(got[p] - ref[2 + i]) <= 2.0 ** -8 * np.abs(ref[2 + i]) + 2.0 ** -18).all()
        want[p] = got[p]
    assert np.array_equal(got, want, equal_nan=True)


def test_a_captured_norm_append_and_another_stream():
    s = Setup([30, 20], [2, 3], 2, 16, seed=10)
    Q, K, V = (s.randn(5, h, 128).to(DEV) for h in (4, 2, 2))
    qw = torch.rand(128, device=DEV)
    out, again = torch.zeros_like(Q), torch.zeros_like(Q)
    call = lambda o: s.cache.append(0, Q, K, V, s.q_start, out=o, q_norm=qw, k_norm=qw)  # noqa: E731
    call(out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(again)
    Q.mul_(2)  # (a norm takes the size out again, all but eps)
    g.replay()
    torch.cuda.synchronize()
    assert s.status() == 0 and not torch.equal(again, torch.zeros_like(again))
    np.testing.assert_allclose(np64(again), np64(out), rtol=2.0 ** -7, atol=1e-6)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        other = s.cache.append(0, Q, K, V, s.q_start, q_norm=qw, k_norm=qw)
    st.synchronize()
    assert torch.equal(other, again)


def test_refusals():
    s = Setup([30], [2], 2, 16, seed=11)
    Q, K, qw = s.randn(2, 4, 128).to(DEV), s.randn(2, 2, 128).to(DEV), torch.ones(128, device=DEV)
    before = s.K.clone()
    call = lambda **kw: s.cache.append(0, Q, K, K, s.q_start, **kw)  # noqa: E731
    for bad in (qw.bfloat16(), qw[:64], qw.cpu(), qw[None], torch.ones(256, device=DEV)[::2]):
        with pytest.raises((ValueError, TypeError)):
            call(q_norm=bad)
        with pytest.raises((ValueError, TypeError)):
            call(k_norm=bad)
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(gb().GraftError):
            call(q_norm=qw, eps=eps)
    torch.cuda.synchronize()
    assert torch.equal(torch.nan_to_num(s.K.float()), torch.nan_to_num(before.float()))
