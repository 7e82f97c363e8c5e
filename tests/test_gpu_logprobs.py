"""Log probabilities, entropy, rank and alternatives against the oracle on the GPU."""
import numpy as np
import pytest
import torch

from oracle import logprobs as olp
from tests.helpers import gb

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, np.int32))).to(DEV)


def check(x, toks, got, rows=None, block=0, top=0, T=1.0):
    """Ids and ranks equal.  Numbers: an exponent z log2 e is off by its three roundings (2^-23 |z|, twice over) where the
    weight counts, a weight by 2^-21 besides, sums of a thread by a rounding a term at most (a chunk's 32 terms of unlike
    size: 2^-19 in all), so ln s by 2^-18 at most (|z| < 8 carries the weight, the rest is smaller than its error); log p
    takes |z| / T 2^-24 more, entropy twice that of ln s times the largest |z| that carries weight, and both a rounding."""
    ref = olp.tokens(x.double().numpy(), toks, rows, block, top, T)
    for name in ("rank", "top_id"):
        assert np.array_equal(got[name].cpu().numpy(), ref[name]), name
    for name in ("logprob", "entropy", "top_logprob"):
        a, b = got[name].double().cpu().numpy(), ref[name]
        assert np.array_equal(np.isnan(a), np.isnan(b)) and np.array_equal(np.isinf(a), np.isinf(b)), name
        fine = np.isfinite(b)
        assert (a[np.isinf(b)] == b[np.isinf(b)]).all()
        tol = 2.0 ** -18 * (8 if name == "entropy" else 1) + 2.0 ** -22 * np.abs(b[fine])
        err = np.abs(a[fine] - b[fine])
        assert (err <= tol).all(), f"{name}: {err.max()}, {(err / tol).max()} of the tolerance"


def run(x, toks, rows=None, block=0, top=0, T=1.0, pad=0, offset=0, **kw):
    R, V = x.shape
    store = torch.full((R * (V + pad) + offset,), float("nan"), dtype=x.dtype)  # what lies around the rows is no logit
    view = store[offset:].view(R, V + pad)[:, :V]
    view.copy_(x)
    dev = store.to(DEV)[offset:].view(R, V + pad)[:, :V]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = gb().graft_token_logprobs(dev, i32(toks), rows=None if rows is None else i32(rows), block=block, top=top,
                                    temperature=T, status=status, **kw)
    torch.cuda.synchronize()
    return got, int(status.item())


def logits(R, V, dtype, seed, scale=3.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(R, V, generator=g) * scale).to(dtype)


TYPES = [torch.float32, torch.bfloat16, torch.float16]


# vocabularies around vectors, threads, chunks; rows that start off 16 bytes
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V,pad,offset", [(1, 0, 0), (2, 0, 1), (3, 1, 0), (7, 0, 0), (8, 0, 0), (31, 0, 3), (255, 0, 0), (513, 0, 0),
                                          (700, 2, 0), (1000, 0, 0), (4095, 0, 0), (4096, 0, 0), (4097, 0, 2), (8192, 0, 0),
                                          (8193, 0, 0), (12289, 5, 1), (32003, 0, 0), (50257, 0, 7)])
def test_sizes(dtype, V, pad, offset):
    R = 5
    x = logits(R, V, dtype, V)
    rng = np.random.default_rng(V)
    toks = rng.integers(0, V, R)
    for top in {0, 1, min(5, V), min(20, V), min(32, V)}:
        got, status = run(x, toks, top=top, pad=pad, offset=offset)
        assert status == 0
        check(x, toks, got, top=top)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,V", [(1, 128256), (3, 151936), (100, 2000), (700, 601), (2000, 40), (60, 50257)])
def test_rows_over_many_ctas(dtype, N, V):
    x = logits(N, V, dtype, N)
    toks = np.random.default_rng(N).integers(0, V, N)
    got, status = run(x, toks, top=8, T=0.7)
    assert status == 0
    check(x, toks, got, top=8, T=0.7)


@pytest.mark.parametrize("T", [0.05, 0.5, 3.0, 100.0])
def test_temperatures(T):
    x = logits(6, 5000, torch.float32, 1)
    toks = x.argmax(1).numpy()
    got, _ = run(x, toks, top=4, T=T)
    check(x, toks, got, top=4, T=T)


@pytest.mark.parametrize("block", [0, 8])
def test_named_rows(block):
    V, K = 3001, 8
    x = logits(4 * K, V, torch.float32, 2)
    rng = np.random.default_rng(2)
    rows = np.full((4, K), -1)
    for b, n in enumerate((3, 8, 1, 5)):
        rows[b, :n] = np.sort(rng.choice(K, n, replace=False)) + (0 if block else b * K)
    rows = rows.reshape(-1)
    toks = np.where(rows >= 0, rng.integers(0, V, 4 * K), -1)
    toks[0] = -1  # a row without a token: its entropy and alternatives all the same
    got, status = run(x, toks, rows=rows, block=block, top=6)
    assert status == 0
    check(x, toks, got, rows=rows, block=block, top=6)
    # the same row for several entries, none for all
    for rows in (np.full(32, 3), np.full(32, -1)):
        got, status = run(x, toks, rows=rows, top=6)
        assert status == 0
        check(x, toks, got, rows=rows, top=6)


def test_many_entries_few_rows():
    N, V = 65535, 501
    x = logits(20, V, torch.bfloat16, 3)
    rows = np.full(N, -1)
    rows[[0, 77, 78, 4096, 40000, 65534]] = [3, 19, 0, 7, 7, 11]
    toks = np.where(rows >= 0, 17, -1)
    got, status = run(x, toks, rows=rows, top=3)
    assert status == 0
    check(x, toks, got, rows=rows, top=3)


@pytest.mark.parametrize("top", [0, 4])
@pytest.mark.parametrize("V", [300, 4099])
def test_the_most_entries(V, top):
    # the longest lists of rows a CTA keeps: 65535 entries that name 61 rows; each as in a call of those rows alone
    x = logits(61, V, torch.bfloat16, V)
    toks = np.arange(61) * 4 % V
    at = np.arange(65535) % 61
    small, _ = run(x, toks, top=top)
    check(x, toks, small, top=top)
    got, status = run(x, toks[at], rows=at, top=top)
    assert status == 0
    pick = torch.from_numpy(at).to(DEV)
    for k in small:
        if small[k].dtype == torch.int32:
            assert torch.equal(got[k], small[k][pick])
        else:  # (a row that a CTA's run cuts is added up in another order: twice a check's tolerance)
            ref = small[k][pick]
            assert bool(((got[k] - ref).abs() <= 2 * (2.0 ** -18 * (8 if k == "entropy" else 1) + 2.0 ** -22 * ref.abs())).all())


def test_rows_and_tokens_out_of_range():
    b = gb()
    x = logits(4, 300, torch.float32, 4)
    got, status = run(x, [5, 300, -1, -7], top=2)
    assert status == b.STATUS_TOKEN_RANGE
    check(x, [5, -1, -1, -1], got, top=2)
    for rows, block, ok in (([0, 4, 2, -2], 0, [0, -1, 2, -1]), ([1, 2, 0, 1], 2, [1, -1, 0, 1])):
        got, status = run(x, [1, 2, 3, 4], rows=rows, block=block, top=2)
        assert status == b.STATUS_ROW
        check(x, [1, -1 if ok[1] < 0 else 2, 3, -1 if ok[3] < 0 else 4], got, rows=ok, block=block, top=2)


# ties, orders and values that a threshold can go wrong on
def _shape(kind, V, rng):
    x = rng.normal(size=V) * 2
    if kind == "equal":
        x[:] = 1.5
    elif kind == "zeros of both signs":
        x[:] = 0.0
        x[::3] = -0.0
    elif kind == "rising":
        x = np.arange(V) / 64.0
    elif kind == "falling":
        x = -np.arange(V) / 64.0
    elif kind == "two values":
        x = rng.integers(0, 2, V).astype(float)
    elif kind == "few values":
        x = rng.integers(-3, 3, V).astype(float)
    elif kind == "one above -inf":
        x[:] = -np.inf
        x[V // 3] = 0.25
    elif kind == "nine above -inf":
        x[:] = -np.inf
        x[rng.choice(V, 9, replace=False)] = rng.normal(size=9)
    elif kind == "lowest ids banned":
        x[:40] = -np.inf
    elif kind == "nine tenths banned":
        x[rng.random(V) < 0.9] = -np.inf
    elif kind == "first chunks banned":
        x[:V - 40] = -np.inf
    elif kind == "late best":
        x[-1] = 100.0
    elif kind == "lowest of the type":
        x[rng.random(V) < 0.5] = -3e38
        x[5] = 0.0
    elif kind == "equal tail":
        x[V // 2:] = x.max() + 1
    elif kind == "all -inf":
        x[:] = -np.inf
    elif kind == "one nan":
        x[V // 2] = np.nan
    elif kind == "one inf":
        x[V // 2] = np.inf
    elif kind == "all nan":
        x[:] = np.nan
    return x


KINDS = ["equal", "zeros of both signs", "rising", "falling", "two values", "few values", "one above -inf", "nine above -inf",
         "lowest ids banned", "nine tenths banned", "first chunks banned", "late best", "equal tail", "all -inf", "one nan",
         "one inf", "all nan"]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [200, 9001, 33000])
@pytest.mark.parametrize("kind", KINDS)
def test_ties_bans_and_orders(kind, V, dtype):
    rng = np.random.default_rng(V)
    N = 3 if V > 20000 else 500  # (a row over several CTAs; several rows a CTA)
    x = torch.from_numpy(np.stack([_shape(kind, V, rng) for _ in range(min(N, 6))])).to(dtype)
    x = x[torch.arange(N) % len(x)]
    toks = rng.integers(0, V, N)
    toks[0], toks[1], toks[-1] = 0, V - 1, V // 3
    got, status = run(x, toks, top=20)
    assert status == 0
    few = np.unique(np.concatenate([np.arange(0, N, max(1, N // 12)), [0, 1, N - 1]]))
    pick = {k: v[torch.from_numpy(few).to(DEV)] for k, v in got.items()}
    check(x[torch.from_numpy(few)], toks[few], pick, top=20)
    # rows alike give results alike, wherever they lie
    for k in range(min(N, 6)):
        same = np.arange(k, N, 6)
        assert (got["top_id"][same.tolist()] == got["top_id"][k]).all()


def test_the_lowest_number_as_a_mask():
    x = logits(4, 6000, torch.float32, 6)
    x[:, ::2] = torch.finfo(torch.float32).min
    got, _ = run(x, [0, 1, 2, 3], top=5)
    ref = olp.tokens(x.double().numpy(), [0, 1, 2, 3], top=5)
    assert np.array_equal(got["top_id"].cpu().numpy(), ref["top_id"]) and np.array_equal(got["rank"].cpu().numpy(), ref["rank"])
    np.testing.assert_allclose(got["entropy"].cpu().numpy(), ref["entropy"], rtol=1e-5)
    np.testing.assert_allclose(got["logprob"].cpu().numpy(), ref["logprob"], rtol=1e-6)  # (-3.4e38 for even tokens)


@pytest.mark.parametrize("big", [1e4, 3e38])
def test_huge_logits(big):
    x = logits(2, 3000, torch.float32, 7)
    x[:, 100] = big
    x[:, 200] = -big
    got, _ = run(x, [100, 5], top=3)
    ref = olp.tokens(x.double().numpy(), [100, 5], top=3)
    assert got["logprob"][0] == 0 and got["entropy"].abs().max() < 1e-6
    np.testing.assert_allclose(got["logprob"].cpu().numpy(), ref["logprob"], rtol=1e-6, atol=1e-6)
    assert np.array_equal(got["top_id"].cpu().numpy(), ref["top_id"])


def test_a_pool_of_logits_past_32_bit_offsets():
    V, R = 151936, 15000  # 2.3e9 logits
    x = torch.zeros(R, V, dtype=torch.bfloat16, device=DEV)
    x[R - 1, V - 7] = 9.0
    x[R - 1, 3] = 8.0
    got = gb().graft_token_logprobs(x, i32([V - 7, 3]), rows=i32([R - 1, R - 1]), top=3)
    s = np.exp(9.0) + np.exp(8.0) + V - 2
    np.testing.assert_allclose(got["logprob"].cpu().numpy(), [9 - np.log(s), 8 - np.log(s)], rtol=1e-5)
    assert got["top_id"].tolist() == [[V - 7, 3, 0]] * 2 and got["rank"].tolist() == [0, 1]


def test_temperatures_at_their_ends():
    x = logits(3, 300, torch.float32, 10)
    x[1, 7] = x[1].max()  # (two tokens share the largest: half each however cold it is)
    best = x.argmax(1).numpy()
    got, _ = run(x, best, top=2, T=1.2e-38)
    ref = [0.0 if (x[i] == x[i].max()).sum() == 1 else -np.log((x[i] == x[i].max()).sum().item()) for i in range(3)]
    np.testing.assert_allclose(got["logprob"].cpu().numpy(), ref, atol=1e-6)
    got, _ = run(x, best, top=2, T=3e38)
    np.testing.assert_allclose(got["logprob"].cpu().numpy(), -np.log(300), rtol=1e-6)
    np.testing.assert_allclose(got["entropy"].cpu().numpy(), np.log(300), rtol=1e-6)


def test_numbers_below_the_normal_ones():
    for dtype, step in ((torch.float32, 2.0 ** -149), (torch.bfloat16, 2.0 ** -133), (torch.float16, 2.0 ** -24)):
        x = (torch.arange(-200, 201) * step).to(dtype).flip(0)[None].repeat(2, 1)
        toks = [200, 30]  # zero, and one of the larger ones
        got, _ = run(x, toks, top=5)
        check(x, toks, got, top=5)


def test_captured_and_on_another_stream():
    x = logits(3, 40000, torch.float32, 8).to(DEV)
    toks = i32([1, 2, 3])
    size = gb().graft_token_logprobs_workspace_size(3, 40000, 5)
    ws = torch.empty(size, dtype=torch.uint8, device=DEV).fill_(255)  # (a workspace need not be zeroed)
    eager = gb().graft_token_logprobs(x, toks, top=5, ws=ws)
    out = {k: torch.zeros_like(v) for k, v in eager.items()}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gb().graft_token_logprobs(x, toks, top=5, ws=ws, out=out)
    for _ in range(3):
        x += 0.5  # (shifts leave the law as it is, up to the logits' rounding)
        x.copy_(x.roll(1, 0))
        g.replay()
        torch.cuda.synchronize()
        check(x.cpu(), [1, 2, 3], out, top=5)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        other = gb().graft_token_logprobs(x, toks, top=5)
    st.synchronize()
    for k in out:
        assert torch.equal(out[k], other[k])


@pytest.mark.parametrize("top", [0, 3])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V,offset", [(4001, 0), (4001, 5), (20011, 3), (20016, 0)])
def test_tokens_anywhere_in_a_piece_among_equals(V, offset, dtype, top):
    # three values and -inf: ranks go by the ids of equal logits, from any place in 16 bytes and beside a chunk's ends
    rng = np.random.default_rng(V + offset)
    at = [e + d for e in (0, 64, 1024, 2048, 8192, 16384, V) for d in range(-17, 18) if 0 <= e + d < V]
    toks = np.array(at)
    x = torch.from_numpy(rng.choice([-2.0, 0.0, 1.5, -np.inf], (len(toks), V))).to(dtype)
    got, status = run(x, toks, top=top, offset=offset)
    check(x, toks, got, top=top)
    assert status == 0


def test_buffers_belong_to_the_given_stream(monkeypatch):
    # (scratch of the current stream could be handed to its next kernels before the call on the other one has run)
    x, st, made = logits(3, 40000, torch.float32, 12).to(DEV), torch.cuda.Stream(), []
    toks, empty = i32([4, 5, 6]), torch.empty
    st.wait_stream(torch.cuda.current_stream())

    def spy(*args, **kw):
        made.append(torch.cuda.current_stream())
        return empty(*args, **kw)

    monkeypatch.setattr(torch, "empty", spy)
    got = gb().graft_token_logprobs(x, toks, top=5, stream=st)
    monkeypatch.undo()
    assert made and all(s == st for s in made)
    st.synchronize()
    check(x.cpu(), [4, 5, 6], got, top=5)


def test_calls_of_other_shapes_share_a_workspace():
    ws = torch.empty(gb().graft_token_logprobs_workspace_size(300, 5000, 32), dtype=torch.uint8, device=DEV)
    for N, V, top in ((300, 5000, 32), (1, 90000, 2), (20, 70, 0), (2, 8191, 5)):
        x = logits(N, V, torch.bfloat16, N)
        toks = np.arange(N) % V
        got, _ = run(x, toks, top=top, ws=ws)
        check(x, toks, got, top=top)


def test_refusals_of_the_binding():
    x, f = logits(4, 50, torch.float32, 9).to(DEV), gb().graft_token_logprobs
    t = i32([0, 1, 2, 3])
    for bad in (dict(tokens=t.long()), dict(tokens=t.cpu()), dict(rows=i32([0, 1])), dict(rows=t.long()),
                dict(out=dict(logprob=t)), dict(ws=torch.empty(16, dtype=torch.uint8, device=DEV))):
        with pytest.raises((ValueError, TypeError, KeyError)):
            f(x, **{"tokens": t, **bad})
    for bad in (x.t(), x[None], x.expand(4, 50)[:1].expand(4, 50), x.double(), x.cpu()):
        with pytest.raises(ValueError):
            f(bad, t)
    for bad in (dict(top=33), dict(top=51), dict(temperature=0.0), dict(block=2), dict(top=-1)):
        with pytest.raises((gb().GraftError, RuntimeError)):
            f(x, t, **bad)
    with pytest.raises(gb().GraftError):
        f(x[:3], t)  # more entries than rows
    assert f(x[:0], t[:0])["logprob"].numel() == 0


def places(x, toks):
    """Place of every row's token by (logit descending, id ascending), NaN as low as -inf."""
    x = np.where(np.isnan(x), -np.inf, x)
    at = np.arange(x.shape[1])[None]
    own = np.take_along_axis(x, toks[:, None], 1)
    return ((x > own) | ((x == own) & (at < toks[:, None]))).sum(1)


@pytest.mark.parametrize("top", [0, 6])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V,offset,N", [(37, 0, 40), (4001, 5, 60), (9001, 0, 700), (33000, 3, 4), (151936, 0, 2)])
def test_ranks_where_logits_are_nan(V, offset, N, dtype, top):
    # tokens that are NaN themselves, and tokens of -inf, of +inf and of numbers with NaN at lower and at higher ids
    rng = np.random.default_rng(V)
    R = min(N, 8)
    x = np.round(rng.normal(size=(R, V)) * 4) / 4
    odd = rng.random((R, V))
    x[odd < 0.3] = np.nan
    x[(odd >= 0.3) & (odd < 0.6)] = -np.inf
    x[R // 2:][(odd[R // 2:] >= 0.6) & (odd[R // 2:] < 0.61)] = np.inf
    x[R - 1] = np.nan
    rows = np.arange(N) % R
    toks = rng.integers(0, V, N)
    for i in range(N):  # a token of every kind, early, late and at the row's ends
        r = x[rows[i]]
        pick = np.flatnonzero([np.isnan, np.isneginf, np.isfinite, np.isposinf][(i // R + i) % 4](r))
        if len(pick):
            toks[i] = pick[[0, -1, len(pick) // 2][i % 3]]
    x = torch.from_numpy(x).to(dtype)
    got, status = run(x, toks, rows=rows, top=top, offset=offset)
    assert status == 0
    assert np.array_equal(got["rank"].cpu().numpy(), places(x.double().numpy()[rows], toks))
    assert bool(torch.isnan(got["logprob"]).all()) and bool(torch.isnan(got["entropy"]).all())
    for k in range(min(top, V)):  # the alternatives' own ranks are their places
        again, _ = run(x, got["top_id"][:, k].cpu().numpy(), rows=rows, offset=offset)
        assert bool((again["rank"] == k).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V,N", [(151936, 2500), (1 << 20, 2500), ((1 << 24) - 24, 1300)])
def test_sums_of_long_rows_of_equal_logits(V, N, dtype):
    """Rows whose first 16384 logits are 0 and whose others are all the same number below: a thread adds the same weight
    again and again, so its roundings go one way.  So many entries name a row that CTAs take it whole.

    ln s is off by: a chunk's 32 equal terms a lane of a pair, whose partial sums round by k / 32 of 2^-24 each (2^-20);
    the chunks', which keep what they round off (2^-23); 16 sums of lanes, warps and pieces (2^-20); a weight by 2^-22
    and by its exponent's two roundings (ln 2 x 4 x 2^-23 < 2^-21); log and differences 2^-23: 2^-18 in all.  log p takes
    a rounding of the result more (2^-24 of it).  The entropy is ln s - ln 2 t / s with |t / s| < 4, t off as s is: 2^-18
    (1 + 2 x 2.8) < 2^-15."""
    C, low = 16384, [-0.21484375, -0.65625, -1.375, -1.484375, -2.21875, -2.4375, -2.6875, -2.71875]
    low = low[:len(low) if V < 1 << 22 else 2]
    x = torch.zeros(len(low), V, dtype=dtype, device=DEV)
    for r, v in zip(x, low):
        r[C:] = v
    rows, toks = np.arange(N) * len(low) // N, np.where(np.arange(N) % 2, 5, V - 5)
    got = gb().graft_token_logprobs(x, i32(toks), rows=i32(rows), top=1)
    z = np.array(low)[rows]
    s = C + (V - C) * np.exp(z)
    for name, ref, tol in (("logprob", np.where(np.arange(N) % 2, 0, z) - np.log(s), 2.0 ** -18),
                           ("entropy", np.log(s) - (V - C) * np.exp(z) * z / s, 2.0 ** -15),
                           ("top_logprob", -np.log(s), 2.0 ** -18)):
        err = np.abs(got[name].double().cpu().numpy().reshape(-1) - ref)
        tol = tol + 2.0 ** -24 * np.abs(ref)
        assert (err <= tol).all(), f"{name}: {err.max()}, {(err / tol).max()} of the tolerance"
    assert got["rank"].tolist() == np.where(np.arange(N) % 2, 5, V - 5).tolist() and bool((got["top_id"] == 0).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [3000, 40000])
def test_all_but_certain_tokens(dtype, V):
    """Two tokens a row, the less likely one first in the same thread's logits, others -inf.  s = 1 + w with w <= e^-8 is
    one rounding off (2^-24), a weight by 2^-22 and its exponent's roundings (16 x 2^-23): less than 2^-18 w < 2^-29, and
    13 times that in the entropy (|z| <= 11.5); the last operations round numbers below 0.005: 2^-23 in all.  (Relative
    to the first token's maximum ln s and t / s would be as large as 11 and cancel.)"""
    gaps = np.linspace(8.0, 11.5, 15)
    x = torch.full((15, V), -float("inf"))
    step = {3000: 1024 if dtype == torch.float32 else 2048, 40000: 8192 if dtype == torch.float32 else 16384}[V]
    x[:, 700] = torch.from_numpy(1.0 - gaps).float()
    x[:, 700 + step] = 1.0
    x = x.to(dtype)
    N = 900
    rows, toks = np.arange(N) * 15 // N, np.where(np.arange(N) % 2, 700, 700 + step)
    got, status = run(x, toks, rows=rows, top=2)
    assert status == 0
    w = np.exp(x[:, 700].double().numpy() - 1.0)[rows]
    likely = toks != 700
    ref = dict(logprob=np.where(likely, 0.0, np.log(w)) - np.log1p(w), entropy=np.log1p(w) - w * np.log(w) / (1 + w),
               top_logprob=np.stack([-np.log1p(w), np.log(w) - np.log1p(w)], 1))
    for name, want in ref.items():
        err = np.abs(got[name].double().cpu().numpy() - want)
        tol = 2.0 ** -23 + 2.0 ** -24 * np.abs(want)
        assert (err <= tol).all(), f"{name}: {err.max()}, {(err / tol).max()} of the tolerance"


@pytest.mark.parametrize("T", [1.0, 0.7, 3.3])
@pytest.mark.parametrize("high", [1e3, 1e4, 1e5])
def test_log_probabilities_far_below_the_largest(high, T):
    """Logits around zero beside one of 1e3 to 1e5: log p = (x - m) / T - ln s is as large as m / T and rounded once, half a
    step of it (2^-24); what is left of the difference, of the quotient and of 1 / T comes along in a second number (each
    within 2^-24 of 2^-24 of the whole: 2^-40).  ln s is 0 here."""
    x = logits(4, 3000, torch.float32, 13)
    x[:, 9] = torch.tensor([high, high * 1.1, high * 1.37, high * 1.83])
    toks = [40 + i for i in range(2900)]
    rows = np.arange(4).repeat(2900)
    toks = np.array(toks * 4)
    got, status = run(x, toks, rows=rows, top=9, T=T)
    assert status == 0
    T = float(np.float32(T))
    ref = (x.double().numpy()[rows, toks] - x[:, 9].double().numpy()[rows]) / T
    err = np.abs(got["logprob"].double().cpu().numpy() - ref)
    assert (err <= (2.0 ** -24 + 2.0 ** -40) * np.abs(ref)).all(), (err / np.abs(ref)).max() * 2 ** 24
