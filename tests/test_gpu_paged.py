"""The paged-cache kernels against the oracle on the GPU."""
import numpy as np
import pytest
import torch

from oracle import paged as opg
from tests.helpers import gb

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # a rounding: half a step, relative


class Setup:
    """A cache of B sequences in shuffled pages (a few spare), with NaN wherever no row lies."""

    def __init__(self, lens, new, Hkv, page, dtype=torch.bfloat16, layers=1, seed=0, wide=0, tables=False):
        from tree_verification_gb300.paged import PagedCache
        self.rng = rng = np.random.default_rng(seed)
        self.lens, self.new, self.page = list(lens), list(new), page
        B = len(lens)
        counts = [-(-(a + b) // page) for a, b in zip(lens, new)]
        P = sum(counts) + 3
        ids = rng.permutation(P)
        self.table = np.full((B, max(max(counts), 1) + wide), -1, np.int32)
        self.table[:] = rng.choice([-1, 10**6], self.table.shape)  # past the rows: nothing to go by
        K = torch.full((layers, P, page, Hkv, 128), float("nan"), dtype=dtype)
        V = K.clone()
        at = 0
        g = torch.Generator().manual_seed(seed + 1)
        for b in range(B):
            self.table[b, :counts[b]] = ids[at:at + counts[b]]
            at += counts[b]
            for r in range(lens[b] + new[b]):
                p, s = int(self.table[b, r // page]), r % page
                K[:, p, s] = torch.randn(layers, Hkv, 128, generator=g).to(dtype)
                V[:, p, s] = torch.randn(layers, Hkv, 128, generator=g).to(dtype)
        self.K0, self.V0 = K, V
        self.dtype, self.Hkv, self.layers, self.g = dtype, Hkv, layers, g
        self.K, self.V = K.to(DEV), V.to(DEV)
        self.starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        i32 = lambda x: torch.from_numpy(np.asarray(x, np.int32)).to(DEV)  # noqa: E731
        self.i32 = i32
        self.q_start, self.lengths, self.t = i32(self.starts), i32(self.lens), i32(self.table)
        self.counts, self.P = counts, P
        refs = np.zeros(P, np.int32)
        refs[ids[:at]] = 1
        self.refs = refs
        self.cache = PagedCache(list(self.K), list(self.V), self.t, self.lengths,
                                page_refs=i32(refs) if tables else None, held=i32(counts) if tables else None)

    def randn(self, *shape):
        return torch.randn(shape, generator=self.g).to(self.dtype)

    def status(self):
        torch.cuda.synchronize()
        s = int(self.cache.status.item())
        self.cache.status.zero_()
        return s


def np64(t):
    return t.detach().double().cpu().numpy()


def check_attention(s, O, Q, scale, mask=None, layer=0, K=None, V=None):
    """O within: its own rounding, the weights' rounding in the product and in their sum (half a step each, the sum's
    cancelling at most), and 2^-12 for 32-bit sums, exponentials and scores."""
    ref, size = opg.attention(np64(Q), np64(s.K0[layer]) if K is None else K, np64(s.V0[layer]) if V is None else V,
                              s.table, s.lens, s.starts, scale, mask, absolute=True)
    got = np64(O)
    live = s.starts[-1]
    u = HALF[s.dtype]
    tol = u * (2 * np.abs(ref) + size) + 2.0 ** -12 * size + 1e-6
    fine = np.isfinite(ref[:live])
    assert np.array_equal(np.isfinite(got[:live]), fine)
    bad = np.abs(got[:live] - ref[:live])[fine] > tol[:live][fine]
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(got[:live] - ref[:live]) / tol[:live])}"


def tree_masks(rng, new):
    m = []
    for n in new:
        row = []
        for i in range(n):
            row.append((row[int(rng.integers(max(0, i - 9), i))] if i else 0) | 1 << i)
        m += row
    return np.array(m, np.uint64)


def run_attention(s, G, pad=0, mask=None, max_new=None, scale=0.09, q_scale=1.0, layer=0):
    N, Hq = int(s.starts[-1]) + pad, s.Hkv * G
    Q = (s.randn(N, Hq, 128).float() * q_scale).to(s.dtype)
    O = torch.full((N, Hq, 128), 7.0, dtype=s.dtype, device=DEV)
    md = None
    if mask is not None:
        md = torch.from_numpy(np.concatenate([mask, np.zeros(pad, np.uint64)]).view(np.int64)).to(DEV)
    s.cache.plan(s.q_start, N, Hq, max(s.new) if max_new is None else max_new, tree=mask is not None)
    s.cache.attend(layer, Q.to(DEV), scale, mask=md, out=O)
    assert s.status() == 0
    assert bool((O[int(s.starts[-1]):] == 7).all())  # rows behind the last sequence stay as they were
    return Q, O


# single tokens and a few: lengths from none, around pages and blocks
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("Hkv,G,page", [(2, 4, 16), (1, 1, 32), (3, 5, 64), (2, 16, 128), (1, 8, 256)])
def test_single_tokens(dtype, Hkv, G, page):
    s = Setup([0, 1, 15, 16, 17, 127, 128, 129, 700, 33], [1] * 10, Hkv, page, dtype, seed=G)
    Q, O = run_attention(s, G)
    check_attention(s, O, Q, 0.09)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("new", [[3, 0, 2, 4, 1], [0, 0, 0, 5, 0], [2, 2, 2, 2, 2]])
def test_a_few_tokens_ragged(dtype, new):
    s = Setup([100, 30, 0, 259, 16], new, 2, 16, dtype, seed=sum(new))
    Q, O = run_attention(s, 4, pad=3, max_new=6)
    check_attention(s, O, Q, 0.09)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("Hkv,G,page,new,lens", [
    (2, 4, 16, [37, 64, 1, 0, 5], [0, 100, 300, 77, 511]),
    (1, 16, 32, [64, 64], [130, 1]),
    (2, 3, 64, [43, 20], [85, 0]),
    (1, 64, 16, [9], [50]),
    (4, 1, 128, [130, 257, 3], [127, 0, 600]),
    (1, 7, 256, [300], [211]),
    (2, 8, 16, [200, 1, 1, 1], [5, 900, 300, 0]),
])
def test_chunks(dtype, Hkv, G, page, new, lens):
    s = Setup(lens, new, Hkv, page, dtype, seed=G + page, wide=2)
    Q, O = run_attention(s, G, pad=5)
    check_attention(s, O, Q, 0.09)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("Hkv,G,page,new,lens", [
    (2, 4, 16, [64, 64, 64], [0, 100, 517]),
    (1, 16, 32, [64, 33, 1, 0], [128, 120, 0, 9]),
    (2, 5, 64, [7, 64], [1000, 64]),
    (2, 1, 16, [64], [300]),
    (8, 4, 16, [32], [512]),
])
def test_trees(dtype, Hkv, G, page, new, lens):
    s = Setup(lens, new, Hkv, page, dtype, seed=7 * G + page)
    mask = tree_masks(s.rng, new)
    Q, O = run_attention(s, G, pad=2, mask=mask)
    check_attention(s, O, Q, 0.09, mask)


@pytest.mark.parametrize("q_scale,scale", [(8.0, 0.5), (30.0, 1.0), (1.0, 1e-6), (0.0, 1.0)])
@pytest.mark.parametrize("new", [[1, 1], [70, 9]])
def test_sharp_and_flat_scores(q_scale, scale, new):
    s = Setup([600, 40], new, 2, 16, seed=5)
    Q, O = run_attention(s, 4, scale=scale, q_scale=q_scale)
    check_attention(s, O, Q, scale)


@pytest.mark.parametrize("new", [[1], [60]])
def test_scores_that_rise_along_the_keys(new):
    # every block's maximum passes the running one by far: the sums are rescaled all along
    s = Setup([900], new, 1, 16, seed=11)
    for r in range(900 + new[0]):
        p, x = int(s.table[0, r // 16]), r % 16
        s.K0[0, p, x] = (r - 450) / 100.0
    s.K.copy_(s.K0)
    N = new[0]
    Q = torch.ones(N, 4, 128, dtype=s.dtype) * 0.5
    O = torch.zeros(N, 4, 128, dtype=s.dtype, device=DEV)
    s.cache.plan(s.q_start, N, 4, N)
    s.cache.attend(0, Q.to(DEV), 0.3, out=O)
    assert s.status() == 0
    check_attention(s, O, Q, 0.3)


@pytest.mark.parametrize("new,G", [([6, 3], 4), ([64, 20], 8)])
def test_rows_that_see_nothing_are_zero(new, G):
    s = Setup([0, 0], new, 2, 16, seed=3)
    mask = tree_masks(s.rng, new)
    mask[[0, 2, new[0] + 1]] = 0
    Q, O = run_attention(s, G, mask=mask)
    check_attention(s, O, Q, 0.09, mask)
    assert bool((O[[0, 2, new[0] + 1]] == 0).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("new,G", [([5, 4], 4), ([40, 64], 8), ([64, 64], 1)])
def test_what_a_row_does_not_see_has_no_effect(dtype, tree, new, G):
    s = Setup([50, 121], new, 2, 16, dtype, seed=4)
    mask = tree_masks(s.rng, new) if tree else None
    for b, j, kind in ((0, 3, float("nan")), (1, 2, float("inf")), (1, 1, float("-inf"))):
        r = s.lens[b] + j
        p, x = int(s.table[b, r // 16]), r % 16
        s.V0[0, p, x, 1, 5:9] = kind
        if kind != kind:
            s.K0[0, p, x, 0] = kind
    s.K.copy_(s.K0)
    s.V.copy_(s.V0)
    Q, O = run_attention(s, G, mask=mask)
    check_attention(s, O, Q, 0.09, mask)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("j", [0, 127, 300, 899])
def test_one_infinity_in_a_long_chunk(dtype, j):
    s = Setup([70, 5], [900, 40], 1, 64, dtype, seed=17)
    r = 70 + j
    s.V0[0, int(s.table[0, r // 64]), r % 64, 0, 3:9] = float("inf")
    s.V0[0, int(s.table[0, 969 // 64]), 969 % 64, 0, 8] = float("-inf")
    s.V.copy_(s.V0)
    Q, O = run_attention(s, 4)
    check_attention(s, O, Q, 0.09)


def test_one_infinity_in_a_long_chunk_takes_no_longer():
    """The elements taken out of the products are looked for in the blocks that were cleaned, not in the whole chunk."""
    from tree_verification_gb300.paged import PagedCache
    n, page = 12000, 64
    pages = -(-n // page)
    K, V = (torch.randn(pages, page, 1, 128, device=DEV).bfloat16() for _ in range(2))
    table = torch.randperm(pages, device=DEV).int().view(1, -1)
    c = PagedCache([K], [V], table, torch.zeros(1, dtype=torch.int32, device=DEV))
    starts = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    Q = torch.randn(n, 4, 128, device=DEV).bfloat16()
    c.plan(starts, n, 4, n)

    def best():
        got = 1e9
        for _ in range(5):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            O = c.attend(0, Q, 0.09)
            b.record()
            torch.cuda.synchronize()
            got = min(got, a.elapsed_time(b))
        return got, O

    plain, O = best()
    V[int(table[0, (n - 2) // page]), (n - 2) % page, 0, 5] = float("inf")
    odd, O2 = best()
    assert int(c.status.item()) == 0
    assert torch.equal(O2[:n - 2], O[:n - 2]) and bool(torch.isinf(O2[n - 2:, :, 5]).all())
    assert odd < 2 * plain + 0.5


def test_strided_queries_and_layers():
    s = Setup([70, 0, 130], [4, 1, 2], 2, 32, layers=3, seed=9)
    N, Hq = 7, 8
    wide = s.randn(N, Hq + 5, 128).to(DEV)
    s.cache.plan(s.q_start, N, Hq, 4)
    for layer in range(3):
        O = s.cache.attend(layer, wide[:, 2:2 + Hq], 0.1)
        assert s.status() == 0
        check_attention(s, O, wide[:, 2:2 + Hq], 0.1, layer=layer)


def test_lengths_change_between_replays_of_one_graph():
    s = Setup([900, 500], [2, 2], 2, 16, seed=10)
    Q = s.randn(4, 8, 128)
    O = torch.zeros(4, 8, 128, dtype=s.dtype, device=DEV)
    Qd = Q.to(DEV)

    def step():
        s.cache.plan(s.q_start, 4, 8, 2)
        s.cache.attend(0, Qd, 0.1, out=O)

    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for lens, starts in (([10, 0], [0, 2, 4]), ([898, 499], [0, 1, 3]), ([0, 77], [0, 0, 2])):
        s.lens, s.starts = lens, np.array(starts, np.int32)
        s.lengths.copy_(s.i32(lens))
        s.q_start.copy_(s.i32(starts))
        g.replay()
        assert s.status() == 0
        check_attention(s, O, Q, 0.1)


@pytest.mark.parametrize("B,L,Hkv", [(1, 3000, 2), (40, 300, 4)])
def test_lengths_that_rise_by_one_a_pass(B, L, Hkv):
    """Decoding: the plan that the attention reads ahead is another one in every pass."""
    s = Setup([L - 3 * b for b in range(B)], [40] * B, Hkv, 16, seed=16)
    s.new, s.starts = [1] * B, np.arange(B + 1, dtype=np.int32)
    s.q_start = s.i32(s.starts)
    Q = s.randn(B, 4 * Hkv, 128)
    O = torch.zeros(B, 4 * Hkv, 128, dtype=s.dtype, device=DEV)
    Qd = Q.to(DEV)

    def step():
        s.lengths.add_(1)
        s.cache.plan(s.q_start, B, 4 * Hkv, 1)
        s.cache.attend(0, Qd, 0.1, out=O)

    step()
    s.lens = [x + 1 for x in s.lens]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(20):
        g.replay()
        s.lens = [x + 1 for x in s.lens]
        got = O.clone()
        s.cache.plan(s.q_start, B, 4 * Hkv, 1)
        torch.cuda.synchronize()
        s.cache.attend(0, Qd, 0.1, out=O)
        assert s.status() == 0 and torch.equal(O, got)
    check_attention(s, O, Q, 0.1)


def test_wide_plans_change_between_replays_of_one_graph():
    """What is split by keys, into how many ranges and where its partial rows lie is another plan's each time; short
    sequences run beside."""
    s = Setup([4000, 700, 900], [64, 40, 2], 2, 32, seed=18)
    N = 106
    Q = s.randn(N, 8, 128)
    O = torch.zeros(N, 8, 128, dtype=s.dtype, device=DEV)
    Qd = Q.to(DEV)

    def step():
        s.cache.plan(s.q_start, N, 8, 64)
        for _ in range(2):  # (two layers: the second call's kernels follow the first's directly)
            s.cache.attend(0, Qd, 0.1, out=O)

    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    cases = [([4000, 700, 900], [0, 64, 104, 106]), ([130, 700, 900], [0, 64, 104, 106]), ([3000, 0, 902], [0, 2, 42, 42]),
             ([4064, 740, 800], [0, 0, 0, 64]), ([0, 0, 0], [0, 33, 64, 106]), ([2222, 600, 840], [0, 3, 40, 102])]
    for lens, starts in cases + cases[::-1]:
        s.lens, s.starts = lens, np.array(starts, np.int32)
        s.lengths.copy_(s.i32(lens))
        s.q_start.copy_(s.i32(starts))
        g.replay()
        assert s.status() == 0
        check_attention(s, O, Q, 0.1)


def test_a_plan_of_fewer_sequences_right_before_its_attention():
    """One sequence after another leaves (its pages given back, its row of Q turned into padding) and the captured
    plan and attention run back to back: what the last plan said of it must not count against the call."""
    B = 40
    s = Setup([100 + 5 * b for b in range(B)], [1] * B, 2, 16, seed=15, tables=True)
    Q = s.randn(B, 8, 128)
    O = torch.zeros(B, 8, 128, dtype=s.dtype, device=DEV)
    Qd = Q.to(DEV)

    def step():
        s.cache.plan(s.q_start, B, 8, 1)
        s.cache.attend(0, Qd, 0.1, out=O)

    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    g.replay()
    assert s.status() == 0
    for b in range(B - 1):
        s.cache.free(s.i32([b]))
        s.lens[b], s.new[b] = 0, 0
        s.starts = np.concatenate([[0], np.cumsum(s.new)]).astype(np.int32)
        s.q_start.copy_(s.i32(s.starts))
        g.replay()
        assert s.status() == 0
    check_attention(s, O, Q, 0.1)


def test_other_streams():
    s = Setup([300], [3], 2, 16, seed=12)
    Q = s.randn(3, 8, 128)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        Qd = Q.to(DEV)
        s.cache.plan(s.q_start, 3, 8, 3)
        O = s.cache.attend(0, Qd, 0.1)
    st.synchronize()
    assert s.status() == 0
    check_attention(s, O, Q, 0.1)


def test_calls_of_many_shapes_share_the_buffers():
    from tree_verification_gb300.paged import PagedCache
    a = Setup([600, 20], [1, 1], 2, 16, seed=13)
    for k, (new, G) in enumerate((([1, 1], 4), ([64, 30], 8), ([1, 0], 1), ([2, 2], 16), ([1, 1], 4))):
        s = Setup([600 - new[0], 20], new, 2, 16, seed=13 + k)
        s.cache._buffers, s.cache._kept = a.cache._buffers, a.cache._kept
        assert isinstance(s.cache, PagedCache)
        Q, O = run_attention(s, G)
        check_attention(s, O, Q, 0.09)


def test_caches_of_other_sizes_share_a_workspace():
    few = Setup([1500], [1], 2, 16, seed=40)
    many = Setup([300 + 17 * x for x in range(90)], [1] * 90, 4, 16, seed=41)
    mixed = Setup([700, 20, 900], [64, 1, 2], 2, 16, seed=42)
    sizes = [(few, 1, 4), (many, 1, 8), (mixed, 64, 2)]
    for s, max_new, G in sizes:
        s.cache.plan(s.q_start, int(s.starts[-1]), s.Hkv * G, max_new)
    ws = torch.zeros(max(s.cache._buffers["attention"].numel() for s, _, _ in sizes), dtype=torch.uint8, device=DEV)
    for s, _, _ in sizes:
        s.cache._buffers["attention"] = ws
    for _ in range(2):
        for s, max_new, G in sizes:
            Q, O = run_attention(s, G)
            assert s.cache._buffers["attention"] is ws
            check_attention(s, O, Q, 0.09)


def test_a_pool_past_32_bit_offsets():
    """Rows whose element offset in the pool passes 2^32."""
    from tree_verification_gb300.paged import PagedCache
    Hkv, page, n = 8, 64, 200
    P = (1 << 32) // (page * Hkv * 128) + 40
    pools = [torch.empty(P, page, Hkv, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    ids = [P - 1 - 7 * i for i in range(4)]
    table = torch.tensor([ids], dtype=torch.int32, device=DEV)
    for pool in pools:
        for p in ids:
            pool[p].normal_()
    lengths = torch.tensor([n], dtype=torch.int32, device=DEV)
    c = PagedCache([pools[0]], [pools[1]], table, lengths)
    starts = torch.tensor([0, 2], dtype=torch.int32, device=DEV)
    q, k, v = (torch.randn(2, h, 128, device=DEV).bfloat16() for h in (32, Hkv, Hkv))
    c.append(0, None, k, v, starts)
    c.plan(starts, 2, 32, 2)
    O = c.attend(0, q, 0.09)
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0
    small = [np64(pool[ids]) for pool in pools]
    assert np.array_equal(small[0][3, n - 192:n - 190], np64(k)) and np.array_equal(small[1][3, n - 192:n - 190], np64(v))
    ref, size = opg.attention(np64(q), *small, [[0, 1, 2, 3]], [n], [0, 2], 0.09, absolute=True)
    assert (np.abs(np64(O) - ref) <= 2.0 ** -8 * (2 * np.abs(ref) + size) + 2.0 ** -12 * size).all()


# ------------------------------------------------------------------ refusals on the device
def test_bad_lengths_leave_their_rows_alone():
    s = Setup([30, 20, 10], [2, 2, 2], 2, 16, seed=20)
    s.lengths[1] = -1
    s.lengths[2] = 10**6
    Q = s.randn(6, 8, 128).to(DEV)
    O = torch.full((6, 8, 128), 7.0, dtype=s.dtype, device=DEV)
    s.cache.plan(s.q_start, 6, 8, 2)
    s.cache.attend(0, Q, 0.1, out=O)
    assert s.status() == gb().STATUS_LENGTH
    assert bool((O[2:] == 7).all()) and bool((O[:2] != 7).any())


@pytest.mark.parametrize("starts,max_new", [([0, 3, 2, 6], 6), ([-1, 2, 4, 6], 6), ([0, 2, 4, 7], 6), ([0, 2, 4, 6], 1)])
def test_bad_starts_are_flagged(starts, max_new):
    s = Setup([30, 20, 10], [2, 2, 2], 2, 16, seed=21)
    Q = s.randn(6, 8, 128).to(DEV)
    s.cache.plan(s.i32(starts), 6, 8, max_new)
    s.cache.attend(0, Q, 0.1)
    assert s.status() & gb().STATUS_LENGTH


@pytest.mark.parametrize("new", [[2], [64]])
@pytest.mark.parametrize("page_id", [-1, 10**6, -2**31, 2**31 - 1])
def test_bad_pages_read_as_zeros(page_id, new):
    s = Setup([70], new, 2, 16, seed=22)
    old = int(s.table[0, 2])
    s.t[0, 2] = page_id
    s.K0[0, old] = 0
    s.V0[0, old] = 0
    Q = s.randn(new[0], 8, 128)
    s.cache.plan(s.q_start, new[0], 8, new[0])
    O = s.cache.attend(0, Q.to(DEV), 0.1)
    assert s.status() == gb().STATUS_PAGE
    check_attention(s, O, Q, 0.1)


def test_a_plan_of_other_arguments_computes_nothing():
    s = Setup([70, 10], [2, 2], 2, 16, seed=23)
    Q = s.randn(4, 8, 128).to(DEV)
    O = torch.full((4, 8, 128), 7.0, dtype=s.dtype, device=DEV)
    s.cache.plan(s.q_start, 4, 16, 2)
    s.cache._plan_of = (4, 8, 2, False)  # the host's note of the plan is set wrong on purpose: the kernel's check
    s.cache.attend(0, Q, 0.1, out=O)
    assert s.status() == gb().STATUS_PLAN
    assert bool((O == 7).all())


def test_host_refusals_of_the_handle():
    s = Setup([70, 10], [2, 2], 2, 16, seed=24, tables=True)
    c, Q = s.cache, s.randn(4, 8, 128).to(DEV)
    with pytest.raises(ValueError):
        c.attend(0, Q, 0.1)  # no plan yet
    c.plan(s.q_start, 4, 8, 2)
    with pytest.raises(ValueError):
        c.attend(1, Q, 0.1)
    with pytest.raises(ValueError):
        c.attend(0, Q.half(), 0.1)
    with pytest.raises(ValueError):
        c.attend(0, Q[:3], 0.1)
    with pytest.raises(ValueError):
        c.attend(0, Q.transpose(0, 1).contiguous().transpose(0, 1), 0.1)
    with pytest.raises(ValueError):
        c.attend(0, Q, 0.1, mask=torch.zeros(4, dtype=torch.int64, device=DEV))
    with pytest.raises(ValueError):
        c.attend(0, Q.cpu(), 0.1)
    with pytest.raises(ValueError):
        c.plan(s.q_start.long(), 4, 8, 2)
    with pytest.raises(gb().GraftError):
        c.plan(s.q_start, 4, 7, 2)
    with pytest.raises(ValueError):
        c.compact(torch.zeros(3, 8, dtype=torch.int32, device=DEV), s.lengths)
    with pytest.raises(ValueError):
        c.reserve(s.lengths[:1])
    with pytest.raises(ValueError):
        c.append(0, Q, Q[:, :2], Q[:3, :2], s.q_start)
    c.held = None
    with pytest.raises(ValueError):
        c.free(s.lengths)
    # a buffer that would have to grow while a graph is being captured (two sequences of at most two rows never
    # need one, whatever N: the premise is checked first)
    import ctypes
    n = ctypes.c_size_t()
    assert gb().lib().graft_paged_plan_size(c._c, 100000, 8, 100000, ctypes.byref(n)) == 0
    assert n.value > c._buffers["plan"].numel()
    g = torch.cuda.CUDAGraph()
    with pytest.raises(ValueError):
        with torch.cuda.graph(g):
            c.plan(s.q_start, 100000, 8, 100000)
    torch.cuda.synchronize()


@pytest.mark.parametrize("which", ["K", "V"])
@pytest.mark.parametrize("offset", [1, 4])
def test_pools_that_are_not_aligned_are_refused(which, offset):
    """Layers carved out of one buffer at an odd place (nothing is launched on them)."""
    from tree_verification_gb300.paged import PagedCache
    shape, n = (4, 16, 2, 128), 4 * 16 * 2 * 128
    flat = torch.zeros(2 * n + 16, dtype=torch.bfloat16, device=DEV)
    even = [flat[:n].view(shape), flat[n:2 * n].view(shape)]
    odd = [even[0], flat[n + offset:2 * n + offset].view(shape)]
    table, lengths = torch.zeros(1, 4, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    PagedCache(even, even, table, lengths)
    with pytest.raises(ValueError, match=which):
        PagedCache(odd if which == "K" else even, odd if which == "V" else even, table, lengths)


def test_a_refused_plan_leaves_none():
    s = Setup([70, 10], [2, 2], 2, 16, seed=25)
    Q = s.randn(4, 8, 128).to(DEV)
    s.cache.plan(s.q_start, 4, 8, 2)
    with pytest.raises(ValueError):
        s.cache.plan(s.q_start.long(), 4, 8, 3)
    with pytest.raises(ValueError):
        s.cache.attend(0, Q, 0.1)
    s.cache.plan(s.q_start, 4, 8, 2)
    with pytest.raises(gb().GraftError):
        s.cache.plan(s.q_start, 4, 7, 2)
    with pytest.raises(ValueError):
        s.cache.attend(0, Q, 0.1)


# ------------------------------------------------------------------ rotary and append
def run_append(s, G, rot, interleaved, factor=1.0, pos=None, pad=0, far=1.0, strided=True):
    N, Hq, H = int(s.starts[-1]) + pad, s.Hkv * G, s.Hkv
    w = 10000.0 ** (-np.arange(rot // 2) * 2 / max(rot, 1)) * far
    base = s.randn(N, Hq + 2 * H, 128).to(DEV)
    Q, K, V = base[:, :Hq], base[:, Hq:Hq + H], base[:, Hq + H:]
    if not strided:
        Q, K, V = Q.contiguous(), K.contiguous(), V.contiguous()
    out = torch.full((N, Hq, 128), 7.0, dtype=s.dtype, device=DEV)
    s.cache.append(0, Q, K, V, s.q_start, inv_freq=torch.from_numpy(w).to(DEV) if rot else None,
                   interleaved=interleaved, positions=None if pos is None else s.i32(pos), factor=factor, out=out)
    assert s.status() == 0
    live = int(s.starts[-1])
    row = np.concatenate([np.arange(n) + L for n, L in zip(s.new, s.lens)]) if live else np.zeros(0, int)
    at = row if pos is None else np.asarray(pos)[:live]
    u = HALF[s.dtype]
    want_k, want_v = np64(s.K0[0]), np64(s.V0[0])
    tol_k = np.zeros_like(want_k)
    b = np.repeat(np.arange(len(s.new)), s.new)
    for name, x, y in (("Q", Q, out), ("K", K, None)):
        x = np64(x)[:live]
        ref = opg.rope(x, at, w, interleaved, factor)
        # half a step of the result, and 32-bit cosines and products of the pair
        tol = u * np.abs(ref) + 2.0 ** -20 * factor * np.abs(x).max()
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
def test_append(dtype, interleaved, rot):
    s = Setup([5, 0, 100, 31, 64], [3, 1, 0, 2, 5], 2, 16, dtype, seed=rot)
    run_append(s, 3, rot, interleaved, factor=1.1, pad=3, strided=rot != 32)


@pytest.mark.parametrize("Hkv,G,page,new", [(8, 4, 64, [64]), (4, 16, 128, [7, 9]), (1, 1, 256, [1, 1, 1]), (5, 3, 32, [33])])
def test_append_heads(Hkv, G, page, new):
    s = Setup([77] * len(new), new, Hkv, page, seed=G)
    run_append(s, G, 128, False)


def test_append_of_rows_that_fill_one_wave_three_at_a_time():
    wave = 5 * torch.cuda.get_device_properties(0).multi_processor_count
    for N in (2 * wave + 1, 2 * wave + 2, 3 * wave, 3 * wave + 1):
        new = [N // 3 + 1, 0, 5, N - N // 3 - 6]
        run_append(Setup([7, 3, 40, 0], new, 1, 64, seed=N % 97), 1, 32, False, pad=2)


def test_append_at_far_positions():
    # 64-bit angles: a position past 2^30 times frequencies up to one radian
    s = Setup([40], [6], 1, 16, torch.float16, seed=2)
    run_append(s, 2, 64, True, pos=[2**30 + 12345, 2**31 - 1, 0, 1, 131071, 10**9 + 7])


def test_append_positions_of_a_tree_and_in_place():
    s = Setup([40, 9], [4, 3], 2, 16, seed=3)
    run_append(s, 2, 128, False, pos=[40, 41, 41, 42, 9, 10, 10])
    Q = s.randn(7, 4, 128).to(DEV)
    K = s.randn(7, 2, 128).to(DEV)
    w = torch.from_numpy(10000.0 ** (-np.arange(64) / 64)).to(DEV)
    out = s.cache.append(0, Q.clone(), K, K, s.q_start, inv_freq=w)
    q2 = Q.clone()
    assert s.cache.append(0, q2, K, K, s.q_start, inv_freq=w, out=q2) is q2
    assert s.status() == 0 and torch.equal(out, q2)


def test_append_refuses_bad_rows_and_pages():
    s = Setup([30, 20, 10], [2, 2, 2], 2, 16, seed=30)
    before = s.K.clone()
    K = s.randn(6, 2, 128).to(DEV)
    s.t[0, 1] = -5          # rows 30, 31 lie in page 1
    s.lengths[1] = 10**6
    s.lengths[2] = -3
    s.cache.append(0, None, K, K, s.q_start)
    assert s.status() == gb().STATUS_PAGE | gb().STATUS_LENGTH
    assert torch.equal(torch.nan_to_num(s.K.float()), torch.nan_to_num(before.float()))


@pytest.mark.parametrize("first", [-1, -2**31, -2**31 + 1, -2**31 + 5])
def test_append_refuses_starts_before_the_rows(first):
    s = Setup([3, 9], [4, 2], 2, 16, seed=9)
    s.q_start[0] = first
    K0, V0 = s.K.clone(), s.V.clone()
    K, V = s.randn(6, 2, 128).to(DEV), s.randn(6, 2, 128).to(DEV)
    s.cache.append(0, None, K, V, s.q_start)
    assert s.status() == gb().STATUS_LENGTH
    bits = lambda x: x.view(torch.int16)  # noqa: E731
    rows = [int(s.table[1, r // 16]) * 16 + r % 16 for r in (9, 10)]
    for pool, was, new in ((s.K[0], K0[0], K), (s.V[0], V0[0], V)):
        flat, old = bits(pool).view(-1, 2, 128), bits(was).view(-1, 2, 128).clone()
        old[rows] = bits(new)[4:]  # the other sequence's rows alone
        assert torch.equal(flat, old)


# ------------------------------------------------------------------ compaction
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("Hkv,page", [(2, 16), (8, 32), (5, 64)])
def test_compaction(dtype, in_place, Hkv, page):
    lens, Kmax = [0, 15, 100, 37, 64, 3], 64
    s = Setup(lens, [Kmax] * 6, Hkv, page, dtype, layers=3, seed=page)
    path = np.full((6, Kmax), -1, np.int32)
    acc = [1, 9, 0, 64, 20, 2]
    for b, a in enumerate(acc):
        # adjacent nodes, gaps, and a move onto rows that later moves read
        path[b, :a] = np.arange(a) if a == 64 else np.sort(s.rng.choice(Kmax, a, replace=False))
    path[1, :9] = [0, 2, 3, 4, 5, 6, 7, 8, 63]
    k, v, want = opg.compact(s.K0.float().numpy(), s.V0.float().numpy(), s.table, lens, path, acc)
    out = s.lengths if in_place else torch.zeros(6, dtype=torch.int32, device=DEV)
    got = s.cache.compact(s.i32(path), s.i32(acc), lengths_out=None if in_place else out)
    assert s.status() == 0 and got.tolist() == list(want)
    assert in_place or s.lengths.tolist() == lens
    assert np.array_equal(s.K.float().cpu().numpy(), k, equal_nan=True)
    assert np.array_equal(s.V.float().cpu().numpy(), v, equal_nan=True)


@pytest.mark.parametrize("in_place", [False, True])
def test_compaction_refuses_bad_paths(in_place):
    s = Setup([10] * 6, [20] * 6, 2, 16, layers=2, seed=31)
    path = np.tile(np.arange(20, dtype=np.int32), (6, 1))
    acc = [3, 3, 3, 21, 3, 3]
    path[0, :3] = [0, 2, 2]
    path[1, :3] = [0, 5, 20]
    path[2, :3] = [-1, 1, 2]
    path[5, :3] = [0, 4, 9]
    s.t[4, 0] = 9999
    before = s.K.clone()
    got = s.cache.compact(s.i32(path), s.i32(acc), lengths_out=None if in_place else torch.zeros_like(s.lengths))
    assert s.status() == gb().STATUS_TREE | gb().STATUS_PAGE
    assert got.tolist() == [10, 10, 10, 10, 10, 13]
    changed = (torch.nan_to_num(s.K.float()) != torch.nan_to_num(before.float())).any(-1).any(-1).any(0).nonzero()
    want = sorted((int(s.table[5, r // 16]), r % 16) for r in (11, 12))
    assert sorted(map(tuple, changed.tolist())) == want


# ------------------------------------------------------------------ reserve, fork, free
def pages_setup(lens, new, page=16, spare=40, wide=6, layers=2, seed=0):
    s = Setup(lens, new, 2, page, layers=layers, seed=seed, wide=wide, tables=True)
    # more spare pages: pools of P + spare pages
    return s


def mirror(s):
    table = np.where(np.arange(s.table.shape[1])[None] < np.array(s.counts)[:, None], s.table, -1)
    return opg.Pages(table, s.counts, s.lens, s.refs, s.page)


def same_state(s, P):
    held = s.cache.held.tolist()
    assert held == P.held and s.lengths.tolist() == P.lengths and s.cache.page_refs.tolist() == P.refs
    for b, h in enumerate(held):
        assert s.t[b, :h].tolist() == P.table[b][:h]


def bigger(lens, new, extra, page=16, layers=2, seed=0, wide=4):
    """A Setup with `extra` more free pages: one more sequence holds them, then is freed."""
    s = Setup(list(lens) + [0], list(new) + [extra * page], 2, page, layers=layers, seed=seed, wide=wide, tables=True)
    P = mirror(s)
    last = len(lens)
    s.cache.free(s.i32([last]))
    P.free([last])
    assert s.status() == 0
    s.lens[last] = 0
    same_state(s, P)
    return s, P


@pytest.mark.parametrize("page", [16, 64])
def test_fork_reserve_free(page):
    lens = [37, 16, 5, 0, 0, 0, 0]
    s, P = bigger(lens, [0] * 7, 40, page, seed=page)
    P.lengths = list(lens) + [0]
    s.lengths.copy_(s.i32(P.lengths))
    src, dst = [0, 0, 1, 2], [3, 4, 5, 6]
    s.cache.fork(s.i32(src), s.i32(dst))
    P.fork(src, dst)
    assert s.status() == 0
    same_state(s, P)
    K, V = s.K.clone(), s.V.clone()
    for new in ([0, 0, 0, 3, 40, 1, 100, 0], [20, 1, 1, 0, 0, 0, 0, 0], [0] * 8):
        copies, refused = P.reserve(new)
        s.cache.reserve(s.i32(new))
        assert s.status() == 0 and not refused
        same_state(s, P)
        for a, b, r in copies:
            K[:, b, :r] = K[:, a, :r]
            V[:, b, :r] = V[:, a, :r]
        assert torch.equal(torch.nan_to_num(s.K.float()), torch.nan_to_num(K.float()))
        assert torch.equal(torch.nan_to_num(s.V.float()), torch.nan_to_num(V.float()))
    for seqs in ([0, 4], [1, 2, 3, 5, 6]):
        s.cache.free(s.i32(seqs))
        P.free(seqs)
        assert s.status() == 0
        same_state(s, P)
    assert not any(P.refs)


def test_reserve_replaces_a_page_that_several_share_for_each_of_them():
    s, P = bigger([20, 0, 0], [0] * 3, 10, seed=1)
    for i in (1, 2):
        s.cache.fork(s.i32([0]), s.i32([i]))
        P.fork([0], [i])
    copies, _ = P.reserve([1, 1, 1, 0])
    s.cache.reserve(s.i32([1, 1, 1, 0]))
    assert s.status() == 0 and len(copies) == 3
    same_state(s, P)
    assert P.refs.count(3) == 1 and max(P.refs) == 3  # the full page stays shared, the old last page is free


def test_reserve_when_pages_run_out():
    s, P = bigger([16, 16, 16, 16], [0] * 4, 3, seed=2)  # 3 + 3 spare pages are free
    new = [30, 0, 33, 1, 0]                              # 2 pages, none, 3, 1: six, all there are
    copies, refused = P.reserve(new)
    s.cache.reserve(s.i32(new))
    assert s.status() == 0 and not refused
    same_state(s, P)
    s, P = bigger([16, 16, 16, 16], [0] * 4, 3, seed=2)
    new = [30, 2, 60, 1, 0]                              # 2, 1, 4: too many, and what follows too
    copies, refused = P.reserve(new)
    s.cache.reserve(s.i32(new))
    assert s.status() == gb().STATUS_CACHE_OVERFLOW and refused == [2, 3]
    same_state(s, P)


def test_reserve_over_many_sequences_and_pages():
    # more sequences than the planning block has threads, more pages than one of its tiles
    from tree_verification_gb300.paged import PagedCache
    B, page, Pn = 1500, 16, 9000
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 40, B)
    counts = -(-lens // page)
    ids = rng.permutation(Pn)[:counts.sum()]
    table = np.full((B, 9), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :counts[b]] = ids[at:at + counts[b]]
        at += counts[b]
    refs = np.zeros(Pn, np.int32)
    refs[ids] = 1
    P = opg.Pages(table, counts, lens, refs, page)
    i32 = lambda x: torch.from_numpy(np.asarray(x, np.int32)).to(DEV)  # noqa: E731
    K = torch.zeros(Pn, page, 1, 128, dtype=torch.bfloat16, device=DEV)
    c = PagedCache([K], [K.clone()], i32(table), i32(lens), page_refs=i32(refs), held=i32(counts))
    for k in range(3):
        new = rng.integers(0, 50, B) * (rng.random(B) < 0.5)
        copies, refused = P.reserve(new)
        c.reserve(i32(new))
        torch.cuda.synchronize()
        assert bool(refused) == bool(int(c.status.item()) & gb().STATUS_CACHE_OVERFLOW)
        c.status.zero_()
        assert c.held.tolist() == P.held and c.page_refs.tolist() == P.refs
        got = c.block_table.tolist()
        assert all(got[b][:P.held[b]] == P.table[b][:P.held[b]] for b in range(B))
        gone = np.nonzero(rng.random(B) < 0.3)[0]
        c.free(i32(gone))
        P.free(gone)
        assert c.page_refs.tolist() == P.refs


def test_bad_page_calls_are_flagged_and_skipped():
    s, P = bigger([20, 20, 0, 0], [0] * 4, 10, seed=3)
    b = gb()
    for src, dst in (([0], [9]), ([-1], [2]), ([0], [1]), ([0], [0])):
        s.cache.fork(s.i32(src), s.i32(dst))
        assert s.status() == b.STATUS_SEQUENCE
        same_state(s, P)
    s.cache.fork(s.i32([0, 1, 2]), s.i32([2, 2, 3]))  # 2 twice, and 3 from 2: the first alone
    P.fork([0], [2])
    assert s.status() == b.STATUS_SEQUENCE
    same_state(s, P)
    s.cache.free(s.i32([2, 2, 77]))
    P.free([2])
    assert s.status() == b.STATUS_SEQUENCE
    same_state(s, P)
    s.cache.reserve(s.i32([-1, 10**6, 0, 0, 0]))
    assert s.status() == b.STATUS_LENGTH
    same_state(s, P)
    s.cache.page_refs[int(s.t[0, 1])] = 0  # a held page that nobody counts
    s.cache.reserve(s.i32([1, 0, 0, 0, 0]))
    assert s.status() == b.STATUS_PAGE
    s.cache.free(s.i32([0]))
    assert s.status() == b.STATUS_PAGE
    assert min(s.cache.page_refs.tolist()) == 0


def rows_changed(now, before):
    """(page, row) of a layer's pool whose bits changed."""
    return sorted(map(tuple, (now.view(torch.int16) != before.view(torch.int16)).any(-1).any(-1).nonzero().tolist()))


def test_rows_go_only_to_pages_that_a_sequence_holds_alone():
    """One page short: of two sequences that share their last page the first gets a copy, the second has the old one to
    itself; a third shares and a fourth lacks pages (its table names others' behind those it holds)."""
    new = [8] * 5
    s, P = bigger([20, 0, 20, 0, 32], new, 2, seed=60)
    c, b = s.cache, gb()
    c.free(s.i32([1, 3]))
    c.fork(s.i32([0, 2]), s.i32([1, 3]))
    s.t[4, 2] = int(s.t[0, 0])
    c.held[4] = 2
    c.page_refs[c.page_refs == 0] = 1
    shared01 = int(s.t[0, 1])
    # one free page for the first sequence's copy
    spare = [p for p in range(s.P) if not (s.t == p).any()][0]
    c.page_refs[spare] = 0
    c.reserve(s.i32([8, 8, 8, 8, 8, 0]))
    assert s.status() == b.STATUS_CACHE_OVERFLOW
    assert int(s.t[0, 1]) == spare and int(c.page_refs[shared01]) == 1
    starts = s.i32([0, 8, 16, 24, 32, 40, 40])
    K, V = s.randn(40, 2, 128).to(DEV), s.randn(40, 2, 128).to(DEV)
    K0 = s.K.clone()
    c.append(0, None, K, V, starts)
    assert s.status() == b.STATUS_PAGE
    want = sorted([(spare, 4 + i) for i in range(8)] + [(shared01, 4 + i) for i in range(8)])
    assert rows_changed(s.K[0], K0[0]) == want
    for q, page in ((0, spare), (1, shared01)):
        assert torch.equal(s.K[0, page, 4:12], K[8 * q:8 * q + 8]) and torch.equal(s.V[0, page, 4:12], V[8 * q:8 * q + 8])
    K0 = s.K.clone()
    path = s.i32(np.tile([0, 3, 5, -1, -1, -1], (6, 1)))
    c.compact(path, s.i32([3, 3, 3, 3, 3, 0]))
    assert s.status() == b.STATUS_PAGE
    assert c.lengths.tolist() == [23, 23, 20, 20, 32, 0]
    assert rows_changed(s.K[0], K0[0]) == sorted([(p, r) for p in (spare, shared01) for r in (5, 6)])


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("new,G", [([3, 2, 4, 1], 4), ([40, 64, 30, 64], 8), ([64, 64, 2, 1], 4)])
def test_sequences_that_take_no_part(tree, new, G):
    lens = [100, 33, 0, 70]
    s, P = bigger(lens, new, 4, seed=61)
    c = s.cache
    s.lengths.copy_(s.i32(lens + [0]))
    on = torch.tensor([True, False, True, False, True], device=DEV)
    s.lengths[3] = -5  # (what a call would flag)
    state = [t.clone() for t in (s.t, c.held, c.page_refs)]
    c.reserve(s.i32([0, 500, 0, 10**6, 0]), active=on)
    assert s.status() == 0
    for t, x in zip((s.t, c.held, c.page_refs), state):
        assert torch.equal(t, x)
    N, H = sum(new), s.Hkv
    starts = s.i32(np.concatenate([[0], np.cumsum(new), [N]]))
    Q, K, V = s.randn(N, H * G, 128).to(DEV), s.randn(N, H, 128).to(DEV), s.randn(N, H, 128).to(DEV)
    mask = tree_masks(s.rng, new) if tree else None
    md = torch.from_numpy(mask.view(np.int64)).to(DEV) if tree else None
    out, O = torch.full_like(Q, 7.0), torch.full_like(Q, 7.0)
    K0, V0 = s.K.clone(), s.V.clone()
    c.append(0, Q, K, V, starts, out=out, active=on)
    c.plan(starts, N, H * G, max(new), tree=tree, active=on)
    c.attend(0, out, 0.09, mask=md, out=O)
    assert s.status() == 0
    at = np.concatenate([[0], np.cumsum(new)])
    s.K0, s.V0 = s.K.cpu(), s.V.cpu()
    s.lens, s.starts = lens, at.astype(np.int32)
    s.table = s.t.cpu().numpy()
    want = []
    for b in range(4):
        rows = slice(at[b], at[b + 1])
        if b in (1, 3):
            assert bool((out[rows] == 7).all()) and bool((O[rows] == 7).all())
        else:
            assert torch.equal(out[rows], Q[rows])
            want += [(int(s.t[b, r // 16]), r % 16) for r in range(lens[b], lens[b] + new[b])]
    assert rows_changed(s.K[0], K0[0]) == rows_changed(s.V[0], V0[0]) == sorted(want)
    ref, size = opg.attention(np64(Q), np64(s.K0[0]), np64(s.V0[0]), s.table, lens, at, 0.09, mask, absolute=True)
    for b in (0, 2):
        rows = slice(at[b], at[b + 1])
        tol = 2.0 ** -8 * (2 * np.abs(ref[rows]) + size[rows]) + 2.0 ** -12 * size[rows] + 1e-6
        assert (np.abs(np64(O[rows]) - ref[rows]) <= tol).all()
    for in_place in (False, True):
        K0 = s.K.clone()
        got = c.compact(s.i32(np.tile([0, 2, -1], (5, 1))), s.i32([2, 2, 2, 99, 0]), active=on,
                        lengths_out=None if in_place else torch.zeros_like(s.lengths))
        assert s.status() == 0 and got.tolist() == [102, 33, 2, -5, 0]
        assert set(rows_changed(s.K[0], K0[0])) <= {(int(s.t[b, (lens[b] + 1) // 16]), (lens[b] + 1) % 16) for b in (0, 2)}
    # calls of two masks and of none in turn: each goes by its own
    masks = [on, torch.tensor([False, True, True, False, True], device=DEV), None]
    s.lengths.copy_(s.i32(lens + [0]))
    for m in masks * 2:
        out.fill_(7.0)
        c.append(0, Q, K, V, starts, out=out, active=m)
        for b in range(4):
            assert bool((out[at[b]:at[b + 1]] == 7).all()) == (m is not None and not bool(m[b]))
    s.status()
    with pytest.raises(ValueError):
        c.plan(starts, N, H * G, max(new), tree=tree, active=on[:4])
    with pytest.raises(ValueError):
        c.reserve(s.i32([0] * 5), active=on.int())


# ------------------------------------------------------------------ schedules
@pytest.mark.parametrize("Hkv,G,page,new,lens", [
    (2, 8, 16, [200, 1, 1, 1], [5, 900, 300, 0]),            # both kinds: the few rows run beside the wide ones
    (8, 16, 16, [64] * 5, [700, 650, 600, 64, 0]),           # two thirds of a wave of items: shared out by keys
    (8, 16, 32, [64] * 6, [1500, 1400, 700, 600, 64, 0]),    # past one round: what is left over is split
    (4, 16, 64, [300, 2, 64], [1000, 3000, 10]),
    (1, 4, 16, [1] * 40, list(range(0, 4000, 100))),         # one item a sequence
    (8, 4, 16, [2] * 45, list(range(0, 900, 20))),           # more items than CTAs: even runs over them
])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_every_schedule_and_the_same_bits_every_time(dtype, Hkv, G, page, new, lens):
    s = Setup(lens, new, Hkv, page, dtype, seed=len(new))
    Q, O = run_attention(s, G)
    check_attention(s, O, Q, 0.09)
    Qd = Q.to(DEV)
    for _ in range(5):
        again = torch.full_like(O, 7.0)
        s.cache.plan(s.q_start, O.shape[0], O.shape[1], max(new))
        s.cache.attend(0, Qd, 0.09, out=again)
        assert torch.equal(again, O)
    assert s.status() == 0


# few items, single tiles among them, and several items a CTA
ONE_TILE = [(32, 2, 64, [64], [n]) for n in (0, 64, 65, 128, 300, 4100)] + [
    (8, 4, 16, [20] * 12, list(range(0, 1200, 100))),
    (8, 4, 16, [9] * 45, [37 * x % 1100 for x in range(45)]),  # several a CTA, of one block and of more
    (8, 4, 32, [20, 40, 20, 64, 9, 30], [700, 650, 130, 600, 64, 0]),  # single tiles and pairs
    (2, 16, 128, [3, 8, 5], [2000, 100, 5000]),
    (1, 5, 256, [25], [1500])]


@pytest.mark.parametrize("Hkv,G,page,new,lens", ONE_TILE)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tree,odd", [(False, False), (True, False), (False, True), (True, True)])
def test_single_tiles(dtype, tree, odd, Hkv, G, page, new, lens):
    s = Setup(lens, new, Hkv, page, dtype, seed=len(new) + lens[0])
    mask = tree_masks(s.rng, new) if tree else None
    if odd:
        for b, n in enumerate(new):
            for j, kind in ((0, float("inf")), (n // 2, float("nan")), (n - 1, float("-inf"))):
                r = lens[b] + j
                s.V0[0, int(s.table[b, r // page]), r % page, b % Hkv, 60 + 3 * j % 64:68 + 3 * j % 64] = kind
        s.V.copy_(s.V0)
    Q, O = run_attention(s, G, mask=mask, q_scale=4.0)
    check_attention(s, O, Q, 0.09, mask)
    again = torch.full_like(O, 7.0)
    md = torch.from_numpy(mask.view(np.int64)).to(DEV) if tree else None
    s.cache.attend(0, Q.to(DEV), 0.09, mask=md, out=again)
    assert torch.equal(again.view(torch.int16), O.view(torch.int16)) and s.status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_a_cta_takes_pairs_and_single_tiles_in_turn(dtype):
    """Rounds of two-tile and of one-tile items, the one-tile ones ever shorter: the second tile's warps sit them out."""
    Hkv = 8
    each = torch.cuda.get_device_properties(0).multi_processor_count // Hkv
    new = [40 if k % 2 == 0 else 9 for k in range(8) for _ in range(each)]
    lens = [max(0, 128 * (5 - k)) + (3 * i) % 80 for k in range(8) for i in range(each)]
    s = Setup(lens, new, Hkv, 64, dtype, seed=50)
    Q, O = run_attention(s, 4)
    check_attention(s, O, Q, 0.09)
    again = torch.full_like(O, 7.0)
    for _ in range(20):
        s.cache.attend(0, Q.to(DEV), 0.09, out=again)
        assert torch.equal(again, O)
    assert s.status() == 0


@pytest.mark.parametrize("extra", [1, 3])
def test_a_few_short_items_past_a_whole_round(extra):
    """Every CTA is as busy as the next, and the blocks left over are fewer than the CTAs."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    s = Setup([2440] * (sms + extra), [17] * (sms + extra), 1, 128, seed=extra)
    Q, O = run_attention(s, 8)
    check_attention(s, O, Q, 0.09)
    again = torch.full_like(O, 7.0)
    s.cache.attend(0, Q.to(DEV), 0.09, out=again)
    assert torch.equal(again, O) and s.status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("Hkv,G,new,lens", [
    (1, 64, [4200, 30, 0, 9], [500, 40, 7, 0]),   # more row blocks than the plan ranks: placed by buckets, nothing split
    (8, 16, [2500, 1, 60, 2], [77, 900, 0, 128]),  # eight whole rounds and more: no partial rows, no join
])
def test_long_chunks_of_many_rounds(dtype, Hkv, G, new, lens):
    s = Setup(lens, new, Hkv, 64, dtype, seed=70)
    N, Hq = int(s.starts[-1]), Hkv * G
    blocks = -(-new[0] // (2 * (128 // G)))
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert blocks > 1024 or blocks * Hkv >= 8 * sms
    Q = torch.randn(N, Hq, 128, generator=torch.Generator(DEV).manual_seed(1), device=DEV).to(dtype)
    O = torch.full((N + 3, Hq, 128), 7.0, dtype=dtype, device=DEV)
    s.cache.plan(s.q_start, N, Hq, max(new))
    s.cache.attend(0, Q, 0.09, out=O[:N])
    assert s.status() == 0 and bool((O[N:] == 7).all())
    # sampled rows, each as a sequence of its own of one new row
    at = [(b, i) for b, n in enumerate(new) for i in {0, n // 2, n - 1, *s.rng.integers(0, max(n, 1), 12).tolist()} if 0 <= i < n]
    rows = [int(s.starts[b]) + i for b, i in at]
    ref, size = opg.attention(np64(Q[rows]), np64(s.K0[0]), np64(s.V0[0]), [s.table[b] for b, _ in at],
                              [lens[b] + i for b, i in at], np.arange(len(at) + 1), 0.09, absolute=True)
    tol = HALF[dtype] * (2 * np.abs(ref) + size) + 2.0 ** -12 * size + 1e-6
    assert (np.abs(np64(O[rows]) - ref) <= tol).all()
    again = torch.full_like(O, 7.0)
    s.cache.attend(0, Q, 0.09, out=again[:N])
    assert torch.equal(again, O) and s.status() == 0


def test_more_sequences_than_a_block_has_threads():
    rng = np.random.default_rng(8)
    n = 1100
    new = [int(x) for x in rng.integers(0, 3, n)]
    new[700] = 20
    s = Setup([int(x) for x in rng.integers(0, 30, n)], new, 1, 16, seed=8)
    Q, O = run_attention(s, 2, pad=1)
    check_attention(s, O, Q, 0.09)


def test_two_graphs_of_one_handle_one_after_another():
    s = Setup([300, 90], [64, 1], 2, 16, seed=14)
    Q = s.randn(65, 8, 128)
    Qd, outs, graphs = Q.to(DEV), [], []
    for _ in range(2):
        O = torch.zeros(65, 8, 128, dtype=s.dtype, device=DEV)

        def step():
            s.cache.plan(s.q_start, 65, 8, 64)
            s.cache.attend(0, Qd, 0.1, out=O)

        step()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        outs.append(O)
        graphs.append(g)
    # a larger plan in between replaces the handle's buffers; the graphs keep theirs
    s.cache.plan(s.q_start, 5000, 8, 4000)
    for g, O in zip(graphs, outs):
        O.zero_()
        g.replay()
        assert s.status() == 0
        check_attention(s, O, Q, 0.1)
