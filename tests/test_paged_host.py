"""Host-side checks of the paged-cache entry points (no GPU needed): refusals, sizes, frequency tables."""
import ctypes
import math

import pytest

from tests.helpers import gb

FAKE = 0x10000  # never dereferenced: every call below fails a host check first, or launches nothing


def cache(**kw):
    c = gb().GraftPagedCache(0, 8, 128, 16, 100, 4, 10, 2, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE)
    for k, v in kw.items():
        setattr(c, k, v)
    return ctypes.addressof(c), c


def attend(c, N=4, Hq=32, max_new=1, plan=FAKE, plan_bytes=1 << 30, Q=FAKE, stride=4096, mask=None, scale=0.1, O=FAKE,
           ws=FAKE, ws_bytes=1 << 40, K=FAKE, V=FAKE):
    return gb().lib().graft_paged_attention(c, K, V, N, Hq, max_new, plan, plan_bytes, Q, stride, mask, scale, O, ws,
                                            ws_bytes, None)


def append(c, N=4, Hq=32, starts=FAKE, freq=FAKE, rot=128, Q=FAKE, qs=4096, K=FAKE, ks=1024, V=FAKE, vs=1024, out=FAKE,
           os=4096, pool=FAKE):
    return gb().lib().graft_rope_append(c, pool, FAKE, N, Hq, starts, None, freq, rot, 0, 1.0, Q, qs, K, ks, V, vs, out, os,
                                        None)


BAD_CACHES = [(dict(dtype=2), -1), (dict(Hkv=0), -1), (dict(head_dim=64), -2), (dict(page_rows=8), -2),
              (dict(page_rows=48), -2), (dict(page_rows=512), -2), (dict(num_pages=0), -1), (dict(n_seqs=0), -1),
              (dict(n_seqs=4097), -2), (dict(max_pages=0), -1), (dict(num_pages=1 << 27), -2),
              (dict(max_pages=1 << 27), -2), (dict(block_table=None), -1), (dict(lengths=None), -1),
              (dict(n_layers=-1), -1), (dict(n_seqs=4096, max_pages=1 << 20, page_rows=16), -2),
              (dict(n_seqs=1, max_pages=(1 << 26) + 1, page_rows=16), -2)]


@pytest.mark.parametrize("kw,rc", BAD_CACHES)
def test_bad_caches_are_refused_by_every_entry(kw, rc):
    lib, n = gb().lib(), ctypes.c_size_t()
    c, keep = cache(**kw)
    assert lib.graft_paged_plan_size(c, 4, 32, 1, ctypes.byref(n)) == rc
    assert lib.graft_paged_attention_workspace_size(c, 4, 32, 1, ctypes.byref(n)) == rc
    assert lib.graft_paged_plan(c, 4, 32, FAKE, 1, 0, FAKE, 1 << 30, None) == rc
    assert attend(c) == rc
    assert append(c) == rc
    assert lib.graft_pages_compact(c, 8, FAKE, FAKE, FAKE, None) == rc
    assert lib.graft_pages_reserve_workspace_size(c, ctypes.byref(n)) == rc
    assert lib.graft_pages_reserve(c, FAKE, FAKE, 1 << 30, None) == rc
    assert lib.graft_pages_fork(c, 1, FAKE, FAKE, None) == rc
    assert lib.graft_pages_free(c, 1, FAKE, None) == rc


def test_the_longest_sequence_is_taken():
    """2^30 rows, so that a row's number plus a call's new rows stays below 2^31."""
    n = ctypes.c_size_t()
    c, keep = cache(n_seqs=1, max_pages=1 << 26, page_rows=16)
    assert gb().lib().graft_paged_plan_size(c, 4, 32, 1, ctypes.byref(n)) == 0 and n.value > 0


def test_null_caches_are_refused():
    lib, n = gb().lib(), ctypes.c_size_t()
    assert lib.graft_paged_plan_size(None, 4, 32, 1, ctypes.byref(n)) == -1
    assert attend(None) == -1 and append(None) == -1
    assert lib.graft_pages_free(None, 1, FAKE, None) == -1


def test_attention_arguments():
    lib = gb().lib()
    c, keep = cache()
    assert attend(c, Hq=12) == -1             # no multiple of Hkv
    assert attend(c, Hq=8 * 65, stride=8 * 65 * 128) == -2
    assert attend(c, N=-1) == -1
    assert attend(c, max_new=-1) == -1
    assert attend(c, mask=FAKE, max_new=65) == -2
    assert attend(c, stride=4095) == -1 and attend(c, stride=4097) == -1 and attend(c, stride=2048) == -1
    assert attend(c, Q=FAKE + 2) == -1 and attend(c, O=FAKE + 8) == -1 and attend(c, K=FAKE + 4) == -1
    assert attend(c, Q=None) == -1 and attend(c, O=None) == -1 and attend(c, V=None) == -1
    assert attend(c, scale=0.0) == -1 and attend(c, scale=math.nan) == -1 and attend(c, scale=-1.0) == -1
    assert attend(c, plan=None) == -3 and attend(c, plan_bytes=64) == -3 and attend(c, plan=FAKE + 16) == -3
    assert attend(c, ws=None) == -3 and attend(c, ws_bytes=64) == -3 and attend(c, ws=FAKE + 128) == -3
    assert attend(c, N=0) == 0                # nothing to do, nothing launched
    assert lib.graft_paged_plan(c, 4, 32, None, 1, 0, FAKE, 1 << 30, None) == -1
    assert lib.graft_paged_plan(c, 4, 32, FAKE, 65, 1, FAKE, 1 << 30, None) == -2
    assert lib.graft_paged_plan(c, 4, 32, FAKE, 1, 0, FAKE, 64, None) == -3


@pytest.mark.parametrize("bad", [dict(tiles=1), dict(min_chunk=256), dict(persist_ctas=-1), dict(split=1), dict(wait_ns=-1),
                                 dict(reserved=(ctypes.c_int32 * 3)(0, 0, 1))])
def test_attention_tuning(bad):
    c, keep = cache()
    t = gb().GraftAttnTuning()
    ex = lambda N, t: gb().lib().graft_paged_attention_ex(  # noqa: E731
        c, FAKE, FAKE, N, 32, 1, FAKE, 1 << 30, FAKE, 4096, None, 0.1, FAKE, t, FAKE, 1 << 40, None)
    assert ex(0, None) == 0 and ex(0, ctypes.addressof(t)) == 0
    for k, v in bad.items():
        setattr(t, k, v)
    assert ex(4, ctypes.addressof(t)) == -1 and ex(0, ctypes.addressof(t)) == -1


def test_append_arguments():
    c, keep = cache()
    assert append(c, rot=24) == -2 and append(c, rot=144) == -2 and append(c, rot=-16) == -2
    assert append(c, freq=None) == -1 and append(c, starts=None) == -1
    assert append(c, N=-1) == -1 and append(c, Hq=-1) == -1
    assert append(c, K=None) == -1 and append(c, V=None) == -1 and append(c, Q=None) == -1 and append(c, out=None) == -1
    assert append(c, ks=1016) == -1 and append(c, vs=1028) == -1 and append(c, qs=100) == -1 and append(c, os=4100) == -1
    assert append(c, Q=FAKE + 8) == -1 and append(c, pool=FAKE + 8) == -1 and append(c, pool=None) == -1
    assert append(c, N=0) == 0


def test_page_calls_arguments():
    lib, n = gb().lib(), ctypes.c_size_t()
    c, keep = cache()
    assert lib.graft_pages_compact(c, 0, FAKE, FAKE, FAKE, None) == -1
    assert lib.graft_pages_compact(c, 65, FAKE, FAKE, FAKE, None) == -2
    assert lib.graft_pages_compact(c, 8, None, FAKE, FAKE, None) == -1
    assert lib.graft_pages_compact(c, 8, FAKE, FAKE, None, None) == -1
    assert lib.graft_pages_reserve_workspace_size(c, ctypes.byref(n)) == 0 and n.value >= 100 * 8
    assert lib.graft_pages_reserve(c, None, FAKE, 1 << 30, None) == -1
    assert lib.graft_pages_reserve(c, FAKE, FAKE, n.value - 1, None) == -3
    for fn, args in ((lib.graft_pages_fork, (FAKE, FAKE)), (lib.graft_pages_free, (FAKE,))):
        assert fn(c, -1, *args, None) == -1
        assert fn(c, 4097, *args, None) == -2
        assert fn(c, 0, *args, None) == 0
    assert lib.graft_pages_fork(c, 1, None, FAKE, None) == -1 and lib.graft_pages_free(c, 1, None, None) == -1
    c, keep = cache(held=None)
    assert lib.graft_pages_free(c, 1, FAKE, None) == -1 and lib.graft_pages_reserve(c, FAKE, FAKE, 1 << 30, None) == -1
    c, keep = cache(K_layers=None)
    assert lib.graft_pages_compact(c, 8, FAKE, FAKE, FAKE, None) == -1


def test_frequencies():
    b = gb()
    w, f = b.graft_rope_inv_freq(128, 10000.0)
    assert f == 1.0 and w.shape == (64,)
    for i in (0, 1, 31, 63):
        assert w[i].item() == pytest.approx(10000.0 ** (-i / 64), rel=1e-14)
    w2, _ = b.graft_rope_inv_freq(128, 10000.0, "linear", 4.0)
    assert (w2 * 4).tolist() == w.tolist()
    # by wavelength: short waves as they were, long ones divided, a blend between that falls
    w3, f = b.graft_rope_inv_freq(128, 500000.0, "wavelength", 8.0, 1.0, 4.0, 8192.0)
    w0, _ = b.graft_rope_inv_freq(128, 500000.0)
    r = (w0 / w3).tolist()
    wave = (2 * math.pi / w0).tolist()
    assert f == 1.0
    for x, v in zip(wave, r):
        if x < 8192 / 4:
            assert v == 1.0
        elif x > 8192:
            assert v == pytest.approx(8.0, rel=1e-14)
        else:
            assert 1.0 <= v <= 8.0
    assert r == sorted(r)
    w4, f = b.graft_rope_inv_freq(64, 10000.0, "yarn", 16.0, 1.0, 32.0, 8192.0)
    w0, _ = b.graft_rope_inv_freq(64, 10000.0)
    r = (w0 / w4).tolist()
    assert f == pytest.approx(0.1 * math.log(16.0) + 1.0, rel=1e-6)
    turns = (8192.0 * w0 / (2 * math.pi)).tolist()
    assert all(v == pytest.approx(1.0) for t, v in zip(turns, r) if t > 64)
    assert all(v == pytest.approx(16.0) for t, v in zip(turns, r) if t < 0.5)
    assert r == sorted(r)


@pytest.mark.parametrize("kw", [dict(rot_dim=7), dict(rot_dim=0), dict(rot_dim=130), dict(base=0.0), dict(base=math.inf),
                                dict(scaling="linear", stretch=0.0), dict(scaling="wavelength", low=4.0, high=1.0),
                                dict(scaling="yarn", original=0.0), dict(scaling="yarn", base=1.0)])
def test_bad_frequencies_are_refused(kw):
    args = dict(rot_dim=64, base=10000.0, stretch=2.0)
    args.update(kw)
    with pytest.raises(gb().GraftError):
        gb().graft_rope_inv_freq(**args)


def test_unknown_scaling_is_refused():
    with pytest.raises(ValueError):
        gb().graft_rope_inv_freq(64, 10000.0, "other")
