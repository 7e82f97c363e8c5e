"""The verify step of a model with normed heads and windowed layers, answering log probabilities: every operator together,
against the oracle, over steps in a row, captured, and with slots that sit steps out."""
import numpy as np
import pytest
import torch

from oracle import logprobs as olp
from oracle import paged as opg
from tests.helpers import gb
from tests.test_gpu_paged_step import B, HKV, HQ, KMAX, LAYERS, PAGE, V, World, i32, np64

pytestmark = pytest.mark.gpu
DEV = "cuda"


def serving(world, windows, **kw):
    g = torch.Generator().manual_seed(world)
    weight = lambda: 1 + 0.3 * torch.randn(128, generator=g)  # noqa: E731
    host = [(weight(), weight()), (None, weight())][:LAYERS]
    norms = [tuple(None if t is None else t.to(DEV) for t in p) for p in host]
    return World(world, norms=norms, eps=1e-5, windows=windows, top_logprobs=kw.pop("top", 3), **kw), host


def check_logprobs(st, target_logits, T=1.0, on=None):
    """The emitted tokens' numbers: 2^-18 for ln s and twice the largest weight-carrying |z| for the entropy (fewer than 32
    terms a thread here), 2^-22 relative."""
    for b in range(B):
        n = int(st.acc["acc_len"][b]) if on is None or on[b] else 0
        path, toks = st.acc["path"][b].tolist(), st.acc["out_tok"][b].tolist()
        for t in range(KMAX):
            got = {k: v[b, t].cpu().numpy() for k, v in st.logprobs.items()}
            if t >= n:
                assert got["rank"] == -1 and got["logprob"] == 0 and (got["top_id"] == -1).all()
                continue
            top = got["top_id"].shape[0]
            lp, h, rank, ids, lps = olp.row(target_logits[b, path[t]].cpu().numpy(), toks[t], top, T)
            assert got["rank"] == rank and np.array_equal(got["top_id"], ids)
            assert abs(got["logprob"] - lp) <= 2.0 ** -18 + 2.0 ** -22 * abs(lp)
            assert abs(got["entropy"] - h) <= 2.0 ** -15 + 2.0 ** -22 * abs(h)
            assert (np.abs(got["top_logprob"] - lps) <= 2.0 ** -18 + 2.0 ** -22 * np.abs(lps)).all()


@pytest.mark.parametrize("windows", [[(20, 4), None], [7, (40, 0)], [(3, 50), (3, 50)]])
def test_steps_in_a_row_match_the_oracle(windows):
    w, host = serving(21, windows)
    c, st, P, most = w.cache, w.step, w.pages, 0
    for k in range(3):
        lens, inp, seen = list(P.lengths), w.inputs(), []
        assert c.lengths.tolist() == lens
        st.run(M_succ=w.M[0], M_cnt=w.M[1], attended=lambda l, O: seen.append((st.Qr.clone(), O.clone(), w.K[l].clone(),
                                                                                w.V[l].clone())), **inp)
        torch.cuda.synchronize()
        assert int(st.status.item()) == 0
        P.reserve([KMAX] * B)
        table, starts = np.array(P.table), np.arange(B + 1) * KMAX
        pos = st.tree["pos"].cpu().numpy().reshape(-1)
        mask = st.tree["mask"].cpu().numpy().view(np.uint64).reshape(-1)
        place = [(table[b, (lens[b] + i) // PAGE], (lens[b] + i) % PAGE) for b in range(B) for i in range(KMAX)]
        for l, (q, o, kl, vl) in enumerate(seen):
            for x, weight, got in ((inp["Q"][l], host[l][0], np64(q).reshape(B * KMAX, HQ, 128)),
                                   (inp["K"][l], host[l][1], np.stack([np64(kl)[p] for p in place]))):
                x = opg.head_norm(np64(x), None if weight is None else weight.numpy(), 1e-5)
                ref = opg.rope(x, pos, w.w.cpu().numpy(), False, w.factor)
                assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -19 * w.factor * np.abs(x).max()).all()
            win = windows[l]
            win = (10**6, 0) if win is None else win if isinstance(win, tuple) else (win, 0)
            ref, size = opg.attention(np64(q).reshape(-1, HQ, 128), np64(kl), np64(vl), table, lens, starts, st.scale, mask,
                                      absolute=True, window=win[0], first=win[1])
            err = np.abs(np64(o).reshape(ref.shape) - ref)
            assert (err <= 2.0 ** -8 * (2 * np.abs(ref) + size) + 2.0 ** -12 * size + 1e-6).all()
        check_logprobs(st, inp["target_logits"])
        P.lengths = [a + int(n) for a, n in zip(lens, st.acc["acc_len"])]
        assert c.lengths.tolist() == P.lengths
        most = max(most, *st.acc["acc_len"].tolist())
    assert most > 1  # (else no path was longer than its root)


@pytest.mark.parametrize("top", [0, 5])
def test_a_captured_step_is_the_step(top):
    (a, _), (b, _) = (serving(22, [(9, 2), None], top=top) for _ in range(2))
    first, later = a.inputs(), a.inputs()
    b.inputs(), b.inputs()
    names = [n for n in first if n not in ("Q", "K", "V")]
    held = {n: first[n].clone() for n in names}
    rows = {n: [x.clone() for x in first[n]] for n in "QKV"}
    for inp in (first, first, later):
        a.step.run(M_succ=a.M[0], M_cnt=a.M[1], **inp)
    b.step.capture(M_succ=b.M[0], M_cnt=b.M[1], **held, **rows)
    b.step.graph.replay()
    for n in names:
        held[n].copy_(later[n])
    for n in "QKV":
        for x, y in zip(rows[n], later[n]):
            x.copy_(y)
    b.step.graph.replay()
    torch.cuda.synchronize()
    assert int(a.step.status.item()) == int(b.step.status.item()) == 0
    assert torch.equal(a.cache.lengths, b.cache.lengths) and torch.equal(a.step.O, b.step.O) and torch.equal(a.K, b.K)
    for k in a.step.logprobs:
        assert torch.equal(a.step.logprobs[k], b.step.logprobs[k])
    check_logprobs(b.step, later["target_logits"])


def test_sampled_tokens_and_idle_slots():
    w, _ = serving(23, [5, None], temperature=0.7, seed=3)
    w.cache.free(i32([1]))
    w.step.active[1] = False
    inp = w.inputs()
    w.step.run(M_succ=w.M[0], M_cnt=w.M[1], **inp)
    torch.cuda.synchronize()
    assert int(w.step.status.item()) == 0
    check_logprobs(w.step, inp["target_logits"], T=0.7, on=[True, False, True])


def test_the_dense_step_answers_too():
    from tree_verification_gb300 import synth
    from tree_verification_gb300.step import VerifyStep
    g = torch.Generator(device=DEV).manual_seed(4)
    cfg = gb().graft_config_init(KMAX, 4, 3, V, 4, [0, 1], 0.3)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    Kc, Vc = n(B, 64, HKV, 128).bfloat16(), n(B, 64, HKV, 128).bfloat16()
    Kt, Vt = n(B, KMAX, HKV, 128).bfloat16(), n(B, KMAX, HKV, 128).bfloat16()
    M = [torch.from_numpy(x).to(DEV) for x in synth.empty_M(V, 4)]
    L = i32([20, 30, 1])
    for T, top in ((0.0, 4), (0.5, 0)):
        step = VerifyStep(cfg, B, HQ, HKV, 1, 64, DEV, [Kc], [Vc], [Kt], [Vt], temperature=T, seed=5, top_logprobs=top)
        plain = VerifyStep(cfg, B, HQ, HKV, 1, 64, DEV, [Kc], [Vc], [Kt], [Vt])
        tl = n(B, KMAX, V) * 2
        step.run(n(B, 4, 3, V), i32([1, 2, 3]), M[0], M[1], L.clone(), [n(B, KMAX, HQ, 128).bfloat16()], tl)
        torch.cuda.synchronize()
        assert int(step.status.item()) == 0 and plain.logprobs is None
        check_logprobs(step, tl, T=T or 1.0)


def test_refusals():
    from tree_verification_gb300.paged_step import PagedVerifyStep
    w = World(24)
    one = torch.ones(128, device=DEV)
    make = lambda **kw: PagedVerifyStep(w.cfg, w.cache, HQ, **kw)  # noqa: E731
    for bad in (dict(norms=[(one, one)]), dict(norms=[(one.half(), one), None]), dict(norms=[(one[:64], None), None]),
                dict(windows=[4]), dict(windows=[0, 4]), dict(windows=[(4, -1), None]), dict(windows=[4.5, None]),
                dict(top_logprobs=-1), dict(top_logprobs=33), dict(top_logprobs=2.0), dict(top_logprobs=True)):
        with pytest.raises((ValueError, TypeError)):
            make(**bad)
    assert make(norms=[None, (None, one)], windows=[None, (4, 2)], top_logprobs=32).logprobs["top_id"].shape == (B, KMAX, 32)
