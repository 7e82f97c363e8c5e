"""Attention over pages with a sliding window and first tokens that stay visible, against the oracle on the GPU."""
import numpy as np
import pytest
import torch

from oracle import paged as opg
from tests.helpers import gb
from tests.test_gpu_paged import HALF, Setup, np64, tree_masks

pytestmark = pytest.mark.gpu
DEV = "cuda"


def evict(s, window, first, poison=True):
    """Gives back every page that no row sees: its entry becomes nonsense; rows that no row sees become NaN."""
    for b, L in enumerate(s.lens):
        lo = L - window + 1
        for j in range(s.counts[b]):
            if j * s.page >= first and (j + 1) * s.page <= lo:
                s.table[b, j] = s.rng.choice([-1, 10**6, -2**31])
            elif poison:
                for x in range(s.page):
                    if first <= j * s.page + x < lo:
                        s.K0[:, s.table[b, j], x] = s.V0[:, s.table[b, j], x] = float("nan")
    s.K.copy_(s.K0)
    s.V.copy_(s.V0)
    s.t.copy_(s.i32(s.table))


def check(s, O, Q, scale, window, first, mask=None, layer=0):
    """Tolerance as in test_gpu_paged: the result's rounding, the weights' in the product and in their sum (half a step
    each, the sum's cancelling at most), 2^-12 for 32-bit sums, exponentials and scores."""
    ref, size = opg.attention(np64(Q), np64(s.K0[layer]), np64(s.V0[layer]), s.table, s.lens, s.starts, scale, mask,
                              absolute=True, window=window, first=first)
    got, live, u = np64(O), s.starts[-1], HALF[s.dtype]
    tol = u * (2 * np.abs(ref) + size) + 2.0 ** -12 * size + 1e-6
    fine = np.isfinite(ref[:live])
    assert np.array_equal(np.isfinite(got[:live]), fine)
    with np.errstate(invalid="ignore"):
        bad = (np.abs(got[:live] - ref[:live]) > tol[:live])[fine]
    assert not bad.any(), f"{bad.sum()} of {bad.size} off"
    odd = ~fine & ~np.isnan(ref[:live])
    assert np.array_equal(got[:live][odd], ref[:live][odd])


def run(s, G, window, first, mask=None, pad=0, scale=0.09, q_scale=1.0, layer=0, out_of=True):
    if out_of:
        evict(s, window, first)
    N, Hq = int(s.starts[-1]) + pad, s.Hkv * G
    Q = (s.randn(N, Hq, 128).float() * q_scale).to(s.dtype)
    O = torch.full((N, Hq, 128), 7.0, dtype=s.dtype, device=DEV)
    md = None
    if mask is not None:
        md = torch.from_numpy(np.concatenate([mask, np.zeros(pad, np.uint64)]).view(np.int64)).to(DEV)
    s.cache.plan(s.q_start, N, Hq, max(s.new), tree=mask is not None, window=window, first=first)
    s.cache.attend(layer, Q.to(DEV), scale, mask=md, out=O, window=window, first=first)
    assert s.status() == 0
    assert bool((O[int(s.starts[-1]):] == 7).all())  # rows behind the last sequence stay as they were
    check(s, O, Q, scale, window, first, mask, layer)
    return Q, O


WINDOWS = [(1, 0), (1, 1), (2, 5), (15, 0), (16, 16), (17, 4), (100, 0), (128, 128), (129, 1), (300, 33), (1 << 30, 0),
           (2**31 - 1, 2**31 - 1), (1, 2**31 - 1)]


def mixed(windows, shapes):
    """Every window with two of the shapes, once in either type."""
    n = len(shapes)
    return [(dtype, *w, *shapes[(i + k * (1 + i // n)) % n]) for i, w in enumerate(windows)
            for k, dtype in enumerate((torch.bfloat16, torch.float16))]


# single tokens: lengths from none, around units, pages and windows
@pytest.mark.parametrize("dtype,window,first,Hkv,G,page", mixed(WINDOWS, [(2, 4, 16), (1, 1, 32), (1, 16, 128), (3, 5, 256)]))
def test_single_tokens(dtype, window, first, Hkv, G, page):
    lens = [0, 1, 15, 16, 17, 127, 128, 129, 400, 33]
    run(Setup(lens, [1] * 10, Hkv, page, dtype, seed=G + window % 97), G, window, first)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("window,first", WINDOWS)
@pytest.mark.parametrize("tree", [False, True])
def test_a_few_tokens(dtype, window, first, tree):
    new = [3, 0, 6, 4, 1, 6]
    s = Setup([100, 30, 0, 259, 16, 900], new, 2, 16, dtype, seed=window % 91)
    run(s, 4, window, first, mask=tree_masks(s.rng, new) if tree else None, pad=3)


@pytest.mark.parametrize("dtype,window,first,Hkv,G,page,new,lens", mixed(WINDOWS, [
    (2, 4, 16, [37, 64, 1, 0, 5], [0, 100, 300, 77, 511]),
    (1, 16, 32, [64, 64], [700, 1]),
    (1, 3, 64, [43, 200], [85, 0]),
    (2, 1, 128, [130, 300, 3], [127, 0, 400]),
    (1, 8, 256, [300], [500]),
]))
def test_chunks(dtype, window, first, Hkv, G, page, new, lens):
    run(Setup(lens, new, Hkv, page, dtype, seed=G + page + window % 89, wide=2), G, window, first, pad=5)


# (3, 0): shorter than the trees are deep; (5, 202): first tokens past the prefix
@pytest.mark.parametrize("dtype,window,first,Hkv,G,page,new,lens", mixed(WINDOWS + [(3, 0), (5, 202), (4, 0)], [
    (2, 4, 16, [64, 64, 64], [0, 100, 317]),
    (1, 16, 64, [64, 30], [200, 1000]),
    (1, 5, 32, [50, 1, 64], [130, 20, 64]),
]))
def test_trees(dtype, window, first, Hkv, G, page, new, lens):
    s = Setup(lens, new, Hkv, page, dtype, seed=G + window % 83)
    run(s, G, window, first, mask=tree_masks(s.rng, new))


@pytest.mark.parametrize("new", [[5], [64]])
def test_chains_see_what_causal_rows_see(new):
    s = Setup([200], new, 2, 16, seed=4)
    chain = np.array([2**(i + 1) - 1 for i in range(new[0])], np.uint64)
    Q = s.randn(new[0], 8, 128).to(DEV)
    m = torch.from_numpy(chain.view(np.int64)).to(DEV)
    for window, first in ((3, 0), (20, 2), (90, 203), (1, 0)):
        s.cache.plan(s.q_start, new[0], 8, new[0], window=window, first=first)
        a = s.cache.attend(0, Q, 0.1, window=window, first=first)
        s.cache.plan(s.q_start, new[0], 8, new[0], tree=True, window=window, first=first)
        b = s.cache.attend(0, Q, 0.1, mask=m, window=window, first=first)
        assert s.status() == 0
        np.testing.assert_allclose(np64(a), np64(b), rtol=2.0 ** -7, atol=2.0 ** -7)


@pytest.mark.parametrize("new,G", [([6, 3], 4), ([64, 20], 8)])
def test_masks_of_any_bits_and_of_none(new, G):
    s = Setup([40, 7], new, 2, 16, seed=5)
    mask = s.rng.integers(0, 2**63, sum(new)).astype(np.uint64) << np.uint64(1) | s.rng.integers(0, 2, sum(new)).astype(np.uint64)
    mask[::3] = 0  # a row without a bit sees the window's rows before the new ones
    for window, first in ((1, 0), (4, 0), (9, 42), (30, 2)):
        run(s, G, window, first, mask=mask, out_of=False)
    Q, O = run(s, G, 1, 0, mask=mask, out_of=False)
    assert bool((O[::3] == 0).all())  # whose window is its own position alone sees nothing


@pytest.mark.parametrize("new", [[1, 1], [300, 9]])
@pytest.mark.parametrize("q_scale,scale", [(8.0, 0.5), (30.0, 1.0), (0.0, 1.0)])
def test_sharp_and_flat_scores(q_scale, scale, new):
    run(Setup([300, 41], new, 2, 16, seed=6), 4, 50, 3, scale=scale, q_scale=q_scale)


@pytest.mark.parametrize("low", [-200.0, -20.0])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_windows_that_start_in_a_later_block_meet_low_scores(low, dtype):
    # all keys alike to a row, with scores far below zero: a maximum left at zero would lose every weight
    s = Setup([500], [300], 1, 16, dtype, seed=7)
    s.K0[:] = torch.where(torch.isnan(s.K0), s.K0, torch.full_like(s.K0, 1.0))
    s.K.copy_(s.K0)
    N = 300
    Q = torch.full((N, 1, 128), low / 128, dtype=dtype)
    for window, first in ((40, 0), (10, 1)):
        s.cache.plan(s.q_start, N, 1, N, window=window, first=first)
        O = s.cache.attend(0, Q.to(DEV), 1.0, window=window, first=first)
        assert s.status() == 0
        check(s, O, Q, 1.0, window, first)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("new,G", [([5, 4], 4), ([40, 64], 8), ([64, 64], 1)])
def test_infinite_values_that_some_rows_see(dtype, tree, new, G):
    s = Setup([300, 150], new, 2, 16, dtype, seed=8)
    mask = tree_masks(s.rng, new) if tree else None
    window, first = 30, 4
    for b, n in enumerate(new):
        for r, kind in ((1, "inf"), (s.lens[b] - 28, "nan"), (s.lens[b] - 20, "-inf"), (s.lens[b] - 3, "inf"),
                        (s.lens[b] + n // 2, "nan"), (s.lens[b] + n - 1, "inf")):
            p = s.table[b, r // 16], r % 16
            s.V0[0, p[0], p[1], b % 2, int(s.rng.integers(128))] = float(kind)
    run(s, G, window, first, mask=mask)


@pytest.mark.parametrize("Hkv,G,page,new,lens", [
    (2, 8, 16, [200, 1, 1, 1], [5, 900, 300, 0]),            # both kinds of rows
    (8, 16, 16, [64] * 5, [700, 650, 600, 64, 0]),           # items shared out by keys
    (8, 16, 32, [64] * 6, [1500, 1400, 700, 600, 64, 0]),    # what is left over past a round is split
    (2, 16, 64, [200, 2, 64], [700, 1500, 10]),
    (1, 4, 16, [1] * 40, list(range(0, 1200, 30))),          # one item a sequence
    (8, 4, 16, [2] * 45, list(range(0, 675, 15))),           # more items than CTAs: even runs over them
    (8, 4, 32, [20, 40, 20, 64, 9, 30], [700, 650, 130, 600, 64, 0]),  # single tiles and pairs
])
@pytest.mark.parametrize("window,first", [(250, 20)])
def test_every_schedule_and_the_same_bits_every_time(Hkv, G, page, new, lens, window, first):
    s = Setup(lens, new, Hkv, page, seed=len(new))
    Q, O = run(s, G, window, first)
    Qd = Q.to(DEV)
    for _ in range(4):
        again = torch.full_like(O, 7.0)
        s.cache.plan(s.q_start, O.shape[0], O.shape[1], max(new), window=window, first=first)
        s.cache.attend(0, Qd, 0.09, out=again, window=window, first=first)
        assert torch.equal(again, O)
    assert s.status() == 0


def test_a_window_past_everything_is_none():
    s = Setup([300, 20, 900], [64, 1, 30], 2, 16, seed=9)
    Q = s.randn(95, 8, 128).to(DEV)
    s.cache.plan(s.q_start, 95, 8, 64)
    s.cache.plan(s.q_start, 95, 8, 64, window=5000)
    a, b = s.cache.attend(0, Q, 0.1), s.cache.attend(0, Q, 0.1, window=5000)
    assert s.status() == 0 and torch.equal(a, b)


def test_layers_of_several_kinds_side_by_side():
    s = Setup([600, 20], [40, 3], 2, 16, layers=3, seed=10)
    N, kinds = 43, [dict(), dict(window=64), dict(window=64, first=5)]
    Q = s.randn(N, 8, 128)
    for k in kinds:
        s.cache.plan(s.q_start, N, 8, 40, **k)
    outs = [s.cache.attend(l, Q.to(DEV), 0.1, **k) for l, k in enumerate(kinds)]
    assert s.status() == 0
    for l, (o, k) in enumerate(zip(outs, kinds)):
        check(s, o, Q, 0.1, k.get("window", 10**6), k.get("first", 0), layer=l)


def test_a_cache_far_past_the_window_reads_the_window_alone():
    # 2^20 rows of which 40 pages are held; the rest of the block table is nonsense
    from tree_verification_gb300.paged import PagedCache
    page, L, window, first = 32, 1 << 20, 300, 10
    K, V = (torch.randn(40, page, 2, 128, device=DEV).bfloat16() for _ in range(2))
    table = torch.full((1, L // page + 2), 10**6, dtype=torch.int32, device=DEV)
    table[0, 0] = 7
    held = range((L - window + 1) // page, L // page + 2)
    table[0, held[0]:held[-1] + 1] = torch.arange(8, 8 + len(held), dtype=torch.int32, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    for n, G in ((1, 4), (40, 8)):
        c = PagedCache([K], [V], table, torch.tensor([L], **i32))
        Q = torch.randn(n, 2 * G, 128, device=DEV).bfloat16()
        c.plan(torch.tensor([0, n], **i32), n, 2 * G, n, window=window, first=first)
        O = c.attend(0, Q, 0.1, window=window, first=first)
        assert int(c.status.item()) == 0
        at = list(range(first)) + list(range(L - window + 1, L + n))
        pick = lambda x: torch.stack([x[table[0, r // page], r % page] for r in at]).double()  # noqa: E731
        k, v = pick(K), pick(V)
        for i in range(n):
            seen = torch.tensor([r < first or L + i - window < r <= L + i for r in at], device=DEV)
            s_ = torch.einsum("hd,khd->hk", Q[i].double(), k.repeat_interleave(G, 1)) * 0.1
            w = torch.softmax(s_.masked_fill(~seen, -float("inf")), 1)
            ref = torch.einsum("hk,khd->hd", w, v.repeat_interleave(G, 1))
            size = torch.einsum("hk,khd->hd", w, v.repeat_interleave(G, 1).abs())
            tol = 2.0 ** -8 * (2 * ref.abs() + size) + 2.0 ** -12 * size + 1e-6
            assert bool(((O[i].double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("new", [[2], [64]])
def test_missing_pages_in_the_window_are_flagged(new):
    s = Setup([400], new, 2, 16, seed=11)
    s.t[0, 24] = -1  # rows 384 .. 399
    Q = s.randn(new[0], 8, 128).to(DEV)
    s.cache.plan(s.q_start, new[0], 8, new[0], window=50)
    s.cache.attend(0, Q, 0.1, window=50)
    assert s.status() == gb().STATUS_PAGE
    s.t[0, 24] = int(s.table[0, 24])
    s.t[0, :20] = -1  # rows 0 .. 319
    s.cache.attend(0, Q, 0.1, window=50)
    assert s.status() == 0
    s.cache.plan(s.q_start, new[0], 8, new[0], window=50, first=1)
    s.cache.attend(0, Q, 0.1, window=50, first=1)
    assert s.status() == gb().STATUS_PAGE


@pytest.mark.parametrize("new", [[2], [64]])
def test_plans_of_other_windows_compute_nothing(new):
    s = Setup([400], new, 2, 16, seed=12)
    Q, N = s.randn(new[0], 8, 128).to(DEV), new[0]
    c = s.cache
    c.plan(s.q_start, N, 8, N)
    for k in ((50, 0), (50, 2), (51, 0)):
        c.plan(s.q_start, N, 8, N, window=k[0], first=k[1])
    plans = {k: c._buffers[k].clone() for k in ("plan", (50, 0), (50, 2), (51, 0))}
    for mine in plans:
        for other in plans:
            O = torch.full((N, 8, 128), 7.0, dtype=s.dtype, device=DEV)
            c._buffers[mine] = plans[other]  # another plan in its place: the kernels' own check
            kw = {} if mine == "plan" else dict(window=mine[0], first=mine[1])
            c.attend(0, Q, 0.1, out=O, **kw)
            want = 0 if mine == other else gb().STATUS_PLAN
            assert s.status() == want and bool((O == 7).all()) == (mine != other)
        c._buffers[mine] = plans[mine]


def test_captured_steps_follow_the_lengths():
    s = Setup([300, 40], [60, 2], 2, 16, seed=13, wide=8)
    Q = s.randn(62, 8, 128).to(DEV)
    O = torch.zeros_like(Q)

    def step():
        s.cache.plan(s.q_start, 62, 8, 60, window=70, first=3)
        s.cache.attend(0, Q, 0.1, out=O, window=70, first=3)
    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for lens in ([300, 40], [17, 0], [250, 39], [0, 5], [300, 40]):
        s.lens = lens
        s.lengths.copy_(s.i32(lens))
        for _ in range(2):
            g.replay()
        assert s.status() == 0
        check(s, O, Q, 0.1, 70, 3)


def test_windows_share_a_workspace_with_full_layers():
    s = Setup([2000, 10, 700], [64, 1, 3], 2, 16, seed=14)
    for _ in range(3):
        for kw in (dict(), dict(window=128, first=4), dict(window=1000)):
            Q = s.randn(68, 16, 128)
            s.cache.plan(s.q_start, 68, 16, 64, **kw)
            O = s.cache.attend(0, Q.to(DEV), 0.1, **kw)
            assert s.status() == 0
            check(s, O, Q, 0.1, kw.get("window", 10**6), kw.get("first", 0))


def test_idle_sequences_and_bad_lengths():
    s = Setup([100, 33, 50, 70], [3, 64, 2, 40], 2, 16, seed=15)
    on = torch.tensor([True, False, True, True], device=DEV)
    s.lengths[2] = -4
    Q = s.randn(109, 8, 128)
    O = torch.full((109, 8, 128), 7.0, dtype=s.dtype, device=DEV)
    s.cache.plan(s.q_start, 109, 8, 64, active=on, window=20, first=2)
    s.cache.attend(0, Q.to(DEV), 0.1, out=O, window=20, first=2)
    assert s.status() == gb().STATUS_LENGTH
    assert bool((O[3:69] == 7).all())
    ref, size = opg.attention(np64(Q), np64(s.K0[0]), np64(s.V0[0]), s.table, s.lens, s.starts, 0.1, absolute=True, window=20,
                              first=2)
    for lo, hi in ((0, 3), (69, 109)):
        tol = 2.0 ** -8 * (2 * np.abs(ref[lo:hi]) + size[lo:hi]) + 2.0 ** -12 * size[lo:hi] + 1e-6
        assert (np.abs(np64(O[lo:hi]) - ref[lo:hi]) <= tol).all()


@pytest.mark.parametrize("tree,Hkv,G,page,new,lens", [
    (True, 8, 4, 16, [64], [1000]), (False, 2, 16, 64, [64] * 3, [700, 300, 129]),
    (False, 2, 8, 128, [200, 1, 1, 1], [5, 900, 300, 0])])
def test_a_bounded_wait_runs_out_and_the_device_stays_usable(tree, Hkv, G, page, new, lens):
    # (a wait bound of 2 ns on valid inputs: every load stays in bounds and completes)
    s = Setup(lens, new, Hkv, page, seed=len(new) + G)
    mask = tree_masks(s.rng, new) if tree else None
    md = torch.from_numpy(mask.view(np.int64)).to(DEV) if tree else None
    N = int(s.starts[-1])
    Q = s.randn(N, Hkv * G, 128).to(DEV)
    for _ in range(2):
        s.cache.plan(s.q_start, N, Hkv * G, max(new), tree=tree, window=300, first=4)
        s.cache.attend(0, Q, 0.09, mask=md, tuning=dict(wait_ns=2), window=300, first=4)
        torch.cuda.synchronize()
        assert s.status() == gb().STATUS_TIMEOUT
        s.cache._buffers["attention"].zero_()
        run(s, G, 300, 4, mask=mask, out_of=False)


def test_another_stream_and_strided_queries():
    s = Setup([900, 30], [5, 64], 2, 32, seed=16)
    base = s.randn(69, 12, 128)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        q = base.to(DEV)[:, 2:10]
        s.cache.plan(s.q_start, 69, 8, 64, window=77, first=1)
        O = s.cache.attend(0, q, 0.1, window=77, first=1)
    st.synchronize()
    assert s.status() == 0
    check(s, O, base[:, 2:10], 0.1, 77, 1)


def test_refusals():
    s = Setup([70, 10], [2, 2], 2, 16, seed=17)
    c, Q = s.cache, s.randn(4, 8, 128).to(DEV)
    c.plan(s.q_start, 4, 8, 2)
    for bad in (dict(window=0), dict(window=-1), dict(window=2**31), dict(window=5, first=-1), dict(window=5, first=2**31),
                dict(first=1), dict(window=5.0), dict(window=None, first=2)):
        with pytest.raises(ValueError):
            c.plan(s.q_start, 4, 8, 2, **bad)
        with pytest.raises(ValueError):
            c.attend(0, Q, 0.1, **bad)
    with pytest.raises(ValueError):
        c.attend(0, Q, 0.1, window=5)  # planned without a window
    c.plan(s.q_start, 4, 8, 2, window=5)
    with pytest.raises(ValueError):
        c.attend(0, Q, 0.1, window=6)
    with pytest.raises(ValueError):
        c.attend(0, Q, 0.1, window=5, first=1)
    with pytest.raises(ValueError):
        c.attend(0, Q, 0.1, window=5, mask=torch.zeros(4, dtype=torch.int64, device=DEV))
    with pytest.raises(gb().GraftError):
        c.plan(s.q_start, 4, 7, 2, window=5)  # refused: it leaves none
    with pytest.raises(ValueError):
        c.attend(0, Q, 0.1, window=5)
    assert c.attend(0, Q, 0.1).shape == Q.shape  # the other plan still stands


@pytest.mark.parametrize("window,first", [(300, 1), (8192, 1), (8193, 1), (300, 9000)])
@pytest.mark.parametrize("new,lens", [([1, 2], [500, 310]), ([64] * 20, [500] * 20)])
def test_small_weights_beside_a_large_one(new, lens, window, first):
    """fp16: a first token that takes all but some thousandths of the weight and holds nothing, and many keys of equal
    weights of 2^-20.5 of its: what the rows read is those keys' values, so their weights' rounding (half a step, 2^-11)
    is all that may show, as it is without a window."""
    s = Setup(lens, new, 8, 16, torch.float16, seed=18)
    s.K0[:] = torch.where(torch.isnan(s.K0), s.K0, torch.zeros_like(s.K0))
    for b in range(len(lens)):
        for r in range(lens[b] + new[b]):
            s.K0[:, s.table[b, r // 16], r % 16, :, 0] = 0.0 if r == 0 else -20.5 * np.log(2.0)
            if r == 0:
                s.V0[:, s.table[b, 0], 0] = 0.0
    s.V0[:] = s.V0.abs() * 100 + 100 * (s.V0 != 0)
    s.K.copy_(s.K0)
    s.V.copy_(s.V0)
    N = sum(new)
    Q = torch.zeros(N, 8, 128, dtype=torch.float16)
    Q[..., 0] = 1.0
    for kw in (dict(window=window, first=first), dict()):
        s.cache.plan(s.q_start, N, 8, max(new), **kw)
        O = s.cache.attend(0, Q.to(DEV), 1.0, **kw)
        assert s.status() == 0
        check(s, O, Q, 1.0, kw.get("window", 10**6), kw.get("first", 0))


@pytest.mark.parametrize("rise", [0.01, 0.05, 0.06, 0.07, 0.08, 0.125, 0.3, 2.0])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_scores_that_rise_from_key_to_key(dtype, rise):
    # every block's largest score lies 128 `rise` (of log2) above the one before: around what fp16 weights by an old
    # maximum can hold (2^9), and far past it
    s = Setup([600] * 4, [200] * 4, 2, 16, dtype, seed=21)
    s.K0[:] = torch.where(torch.isnan(s.K0), s.K0, torch.zeros_like(s.K0))
    for b in range(4):
        for r in range(800):
            x = rise * np.log(2.0) * (r if b % 2 == 0 else 800 - r)
            high = float(torch.tensor(x).to(dtype))
            s.K0[:, s.table[b, r // 16], r % 16, :, 0], s.K0[:, s.table[b, r // 16], r % 16, :, 1] = high, x - high
    s.K.copy_(s.K0)
    Q = torch.zeros(800, 4, 128, dtype=dtype)
    Q[..., :2] = 1.0
    for window, first in ((500, 0), (500, 4), (129, 130)):
        s.cache.plan(s.q_start, 800, 4, 200, window=window, first=first)
        O = s.cache.attend(0, Q.to(DEV), 1.0, window=window, first=first)
        assert s.status() == 0
        check(s, O, Q, 1.0, window, first)


def test_a_plan_of_the_next_step_leaves_none_of_the_last():
    # a kind that is planned again begins a step: plans that the last one attended are not attended in it
    s = Setup([70, 10], [2, 2], 2, 16, seed=19)
    c, Q = s.cache, s.randn(4, 8, 128).to(DEV)
    kinds = [dict(), dict(window=5), dict(window=5, first=2)]
    plan, attend = (lambda k: c.plan(s.q_start, 4, 8, 2, **k)), (lambda k: c.attend(0, Q, 0.1, **k))
    for again in kinds:
        for order in (kinds, kinds[::-1], kinds[1:] + kinds[:1]):  # steps that plan every kind first, in any order
            for k in order:
                plan(k)
            for k in kinds + kinds:
                attend(k)
        for k in kinds:  # one that plans them as they come
            plan(k)
            attend(k)
        attend(kinds[0])
        plan(again)
        for k in kinds:
            if k is again:
                attend(k)
            else:
                with pytest.raises(ValueError):
                    attend(k)
    assert s.status() == 0


def test_pages_given_back_behind_the_window():
    """A sequence whose pages behind the window were given back reserves, attends and is freed like any other; a fork of it
    is refused, and a number that is no page is still flagged."""
    window, first, b = 50, 4, gb()
    s = Setup([200, 40, 0], [8, 8, 0], 2, 16, seed=20, wide=4, tables=True)
    c, refs = s.cache, s.refs.copy()
    for j in range(s.counts[0]):
        if j * s.page >= first and (j + 1) * s.page - 1 <= s.lens[0] - window:
            refs[s.table[0, j]] = 0
            s.table[0, j] = -1
    given_back = int((s.table[0, :s.counts[0]] == -1).sum())
    assert given_back == 8  # pages 1 to 8: rows 16 .. 143, before row 151 - 1
    s.t.copy_(s.i32(s.table))
    c.page_refs.copy_(s.i32(refs))
    c.reserve(s.i32([30, 0, 0]))
    assert s.status() == 0
    held = c.held.tolist()
    assert held == [15, 3, 0] and (np.array(c.page_refs.tolist()) > 0).sum() == 15 - given_back + 3
    assert s.t[0, 1:9].tolist() == [-1] * 8
    run(s, 4, window, first, out_of=False)
    before = [t.tolist() for t in (c.page_refs, c.held, c.lengths, s.t)]
    c.fork(s.i32([0]), s.i32([2]))
    assert s.status() == b.STATUS_PAGE
    assert before == [t.tolist() for t in (c.page_refs, c.held, c.lengths, s.t)]
    kept = c.page_refs.clone()
    for p in s.t[0, :15].tolist():
        if p >= 0:
            kept[p] = 0
    c.free(s.i32([0]))
    assert s.status() == 0
    assert torch.equal(c.page_refs, kept) and c.held.tolist() == [0, 3, 0] and c.lengths.tolist() == [0, 40, 0]
    assert bool((s.t[0] == -1).all())
    for nonsense in (-2, 10**6, -2**31):  # no page, and none given back
        s.t[1, 0] = nonsense
        c.held[1] = 1
        c.free(s.i32([1]))
        assert s.status() == b.STATUS_PAGE
