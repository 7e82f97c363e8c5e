"""The paged verify step, chained: every stage against the oracle, over several steps with forks between them."""
import numpy as np
import pytest
import torch

from oracle import accept as oacc
from oracle import paged as opg
from oracle import update_m as oupd
from tests.helpers import gb
from tree_verification_gb300 import synth

pytestmark = pytest.mark.gpu
DEV = "cuda"
B, KMAX, HQ, HKV, LAYERS, PAGE, V, W = 3, 16, 8, 2, 2, 16, 512, 4


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, np.int32))).to(DEV)


class World:
    """A cache of three sequences (the last one empty), its pools, M, and a step."""

    def __init__(self, world, dtype=torch.bfloat16, **kw):
        from tree_verification_gb300.paged import PagedCache
        from tree_verification_gb300.paged_step import PagedVerifyStep
        self.rng = np.random.default_rng(world)
        self.g = torch.Generator(device=DEV).manual_seed(world)
        lens, P, M = [37, 48, 0], 40, 12
        counts = [-(-n // PAGE) for n in lens]
        ids = self.rng.permutation(P)
        table = np.full((B, M), -1, np.int32)
        refs = np.zeros(P, np.int32)
        at = 0
        for b, c in enumerate(counts):
            table[b, :c] = ids[at:at + c]
            at += c
        refs[ids[:at]] = 1
        self.pages = opg.Pages(table, counts, lens, refs, PAGE)
        self.K = torch.randn(LAYERS, P, PAGE, HKV, 128, generator=self.g, device=DEV).to(dtype)
        self.V = torch.randn(LAYERS, P, PAGE, HKV, 128, generator=self.g, device=DEV).to(dtype)
        self.cache = PagedCache(list(self.K), list(self.V), i32(table), i32(lens), page_refs=i32(refs), held=i32(counts))
        self.cfg = gb().graft_config_init(KMAX, 4, 3, V, W, [0, 1], 0.3)
        self.w, self.factor = gb().graft_rope_inv_freq(128, 10000.0, "yarn", 4.0, 1.0, 32.0, 64.0, device=DEV)
        self.step = PagedVerifyStep(self.cfg, self.cache, HQ, inv_freq=self.w, factor=self.factor, **kw)
        s, c = synth.empty_M(V, W)
        self.M = [torch.from_numpy(s).to(DEV), torch.from_numpy(c).to(DEV)]
        self.dtype = dtype

    def inputs(self):
        n = lambda *s: torch.randn(*s, generator=self.g, device=DEV)  # noqa: E731
        dl, roots = n(B, 4, 3, V), i32(self.rng.integers(0, V, B))
        tree = gb().graft_build_tree(self.cfg, dl, roots, self.M[0], self.cache.lengths)
        tl = n(B, KMAX, V)
        synth.plant_paths(tl, tree["tok"].cpu().numpy(), tree["parent"].cpu().numpy(), tree["depth"].cpu().numpy(),
                          self.rng.integers(1, 5, B))
        qkv = [n(B * KMAX, HQ + 2 * HKV, 128).to(self.dtype) for _ in range(LAYERS)]
        return dict(draft_logits=dl, root_tok=roots, Q=[x[:, :HQ] for x in qkv], K=[x[:, HQ:HQ + HKV] for x in qkv],
                    V=[x[:, HQ + HKV:] for x in qkv], target_logits=tl)


def np64(t):
    return t.detach().double().cpu().numpy()


@pytest.mark.parametrize("m_policy", ["tree", "both"])
def test_chained_steps_match_the_oracle(m_policy):
    w = World(1, m_policy=m_policy)
    c, st, P = w.cache, w.step, w.pages
    for k in range(4):
        if k == 2:  # the empty sequence's rows so far go; it becomes a copy of the first one
            c.free(i32([2]))
            c.fork(i32([0]), i32([2]))
            P.free([2])
            P.fork([0], [2])
        lens = list(P.lengths)
        assert c.lengths.tolist() == lens
        inp = w.inputs()
        Kp, Vp = np64(w.K), np64(w.V)
        seen = []
        s0, c0 = w.M[0].cpu().numpy(), w.M[1].cpu().numpy()
        st.run(M_succ=w.M[0], M_cnt=w.M[1], attended=lambda l, O: seen.append((st.Qr.clone(), O.clone(), w.K[l].clone(),
                                                                                w.V[l].clone())), **inp)
        torch.cuda.synchronize()
        assert int(st.status.item()) == 0
        # pages: reserved, the shared last page copied
        copies, refused = P.reserve([KMAX] * B)
        assert not refused and (k != 2 or len(copies) == 2)
        for a, b, r in copies:
            Kp[:, b, :r], Vp[:, b, :r] = Kp[:, a, :r], Vp[:, a, :r]
        assert c.page_refs.tolist() == P.refs and c.held.tolist() == P.held
        table = np.array(P.table)
        pos = st.tree["pos"].cpu().numpy().reshape(-1)
        mask = st.tree["mask"].cpu().numpy().view(np.uint64).reshape(-1)
        starts = np.arange(B + 1) * KMAX
        for l, (q, o, kl, vl) in enumerate(seen):
            # rotated rows: half a step of bf16 and 32-bit products
            for name, x in (("Q", inp["Q"][l]), ("K", inp["K"][l])):
                ref = opg.rope(np64(x), pos, w.w.cpu().numpy(), False, w.factor)
                tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * w.factor * np.abs(np64(x)).max()
                if name == "Q":
                    got = np64(q).reshape(ref.shape)
                else:
                    got = np.stack([np64(kl)[table[b, (lens[b] + i) // PAGE], (lens[b] + i) % PAGE]
                                    for b in range(B) for i in range(KMAX)])
                assert (np.abs(got - ref) <= tol).all()
            for b in range(B):  # (the mirror takes the rows as the GPU rounded them)
                for i in range(KMAX):
                    p, r = table[b, (lens[b] + i) // PAGE], (lens[b] + i) % PAGE
                    Kp[l, p, r] = np64(kl[p, r])
                    Vp[l, p, r] = np64(vl[p, r])
                    assert np.array_equal(Vp[l, p, r], np64(inp["V"][l][b * KMAX + i]))
            ref, size = opg.attention(np64(q).reshape(-1, HQ, 128), Kp[l], Vp[l], table, lens, starts, st.scale, mask,
                                      absolute=True)
            err = np.abs(np64(o).reshape(ref.shape) - ref)
            assert (err <= 2.0 ** -8 * (2 * np.abs(ref) + size) + 2.0 ** -12 * size + 1e-6).all()
        # acceptance and compaction
        acc, path = [], np.full((B, KMAX), -1)
        for b in range(B):
            t = {n: st.tree[n][b].tolist() for n in ("tok", "parent", "depth")}
            _, n, p, out_tok, bonus = oacc.accept(inp["target_logits"][b].cpu().numpy(), t["tok"], t["parent"], t["depth"])
            assert st.acc["acc_len"][b].item() == n and st.acc["path"][b, :n].tolist() == p
            assert st.acc["out_tok"][b, :n].tolist() == out_tok and st.acc["bonus"][b].item() == bonus
            acc.append(n)
            path[b, :n] = p
        Kp, Vp, new = opg.compact(Kp, Vp, table, lens, path, acc)
        assert c.lengths.tolist() == list(new) and max(acc) > 1
        P.lengths = [int(x) for x in new]
        for b in range(B):
            for r in range(P.lengths[b]):
                p, x = table[b, r // PAGE], r % PAGE
                assert np.array_equal(np64(w.K[:, p, x]), Kp[:, p, x]) and np.array_equal(np64(w.V[:, p, x]), Vp[:, p, x])
        if m_policy == "tree":
            g = st.acc["argmax"].cpu().numpy().reshape(-1)
            s1, c1 = oupd.update_M(s0, c0, st.tree["tok"].cpu().numpy().reshape(-1), g)
            assert np.array_equal(w.M[0].cpu().numpy(), s1) and np.array_equal(w.M[1].cpu().numpy(), c1)


def test_a_captured_step_is_the_step():
    a, b = World(5), World(5)
    first, later = a.inputs(), a.inputs()
    b.inputs(), b.inputs()
    names = [n for n in first if n not in ("Q", "K", "V")]
    held = {n: first[n].clone() for n in names}
    rows = {n: [x.clone() for x in first[n]] for n in "QKV"}
    for inp in (first, first, later):
        a.step.run(M_succ=a.M[0], M_cnt=a.M[1], **inp)
    torch.cuda.synchronize()
    b.step.capture(M_succ=b.M[0], M_cnt=b.M[1], **held, **rows)  # runs the first step, then captures it
    b.step.graph.replay()
    for n in names:
        held[n].copy_(later[n])
    for n in "QKV":
        for x, y in zip(rows[n], later[n]):
            x.copy_(y)
    b.step.graph.replay()
    torch.cuda.synchronize()
    assert int(a.step.status.item()) == int(b.step.status.item()) == 0
    assert torch.equal(a.cache.lengths, b.cache.lengths) and torch.equal(a.step.acc["out_tok"], b.step.acc["out_tok"])
    assert torch.equal(a.step.O, b.step.O) and torch.equal(a.K, b.K) and torch.equal(a.V, b.V)
    assert torch.equal(a.cache.page_refs, b.cache.page_refs) and torch.equal(a.M[1], b.M[1])


def test_sampling_and_fp16():
    w = World(9, dtype=torch.float16, temperature=0.7, seed=3)
    inp = w.inputs()
    w.step.run(M_succ=w.M[0], M_cnt=w.M[1], **inp)
    torch.cuda.synchronize()
    assert int(w.step.status.item()) == 0
    y = gb().graft_sample_tokens(inp["target_logits"], w.step.tree["pos"], 0.7, 3)
    assert torch.equal(y, w.step.acc["argmax"])
    assert w.cache.lengths.tolist() == [a + b for a, b in zip([37, 48, 0], w.step.acc["acc_len"].tolist())]


@pytest.mark.parametrize("m_policy", ["tree", "both"])
@pytest.mark.parametrize("captured", [False, True])
def test_idle_slots(m_policy, captured):
    """A slot is freed and sits two steps out with senseless inputs; then a fork takes it."""
    w = World(11, m_policy=m_policy)
    c, st = w.cache, w.step
    c.free(i32([1]))  # the middle one
    st.active[1] = False
    names = ("draft_logits", "root_tok", "target_logits")
    held = w.inputs()
    rows = slice(KMAX, 2 * KMAX)

    def spoil(inp):
        inp["draft_logits"][1] *= 1e6
        inp["target_logits"][1] = float("nan")
        for n in "QKV":
            for x in inp[n]:
                x[rows] = float("nan")

    def step(inp):
        for n in names:
            held[n].copy_(inp[n])
        for n in "QKV":
            for x, y in zip(held[n], inp[n]):
                x.copy_(y)
        if graph is None:
            st.run(M_succ=w.M[0], M_cnt=w.M[1], **held)
        else:
            graph.replay()
        torch.cuda.synchronize()
        assert int(st.status.item()) == 0

    graph = None
    if captured:
        lens, tables = c.lengths.clone(), [t.clone() for t in (c.block_table, c.held, c.page_refs)]
        M = [t.clone() for t in w.M]
        spoil(held)
        graph = st.capture(M_succ=w.M[0], M_cnt=w.M[1], **held)  # (its step is undone)
        for t, x in zip((c.lengths, c.block_table, c.held, c.page_refs, *w.M), (lens, *tables, *M)):
            t.copy_(x)
    refs = int(c.page_refs.sum())
    for k in range(2):
        inp = w.inputs()
        spoil(inp)
        lens, O = c.lengths.tolist(), st.O.clone()
        s0, c0 = w.M[0].cpu().numpy(), w.M[1].cpu().numpy()
        step(inp)
        acc = st.acc["acc_len"].tolist()
        assert acc[1] == 0 and acc[0] >= 1 and acc[2] >= 1
        assert c.lengths.tolist() == [lens[0] + acc[0], 0, lens[2] + acc[2]]
        assert int(c.held[1]) == 0 and bool((c.block_table[1] == -1).all())
        assert int(c.page_refs.sum()) == int(c.held.sum()) and int(c.page_refs.max()) == 1
        assert torch.equal(st.O[1], O[1]) and not torch.equal(st.O[0], O[0])
        for b in (0, 2):  # the others, as ever
            t = {n: st.tree[n][b].tolist() for n in ("tok", "parent", "depth")}
            _, n, p, out_tok, bonus = oacc.accept(inp["target_logits"][b].cpu().numpy(), t["tok"], t["parent"], t["depth"])
            assert acc[b] == n and st.acc["out_tok"][b, :n].tolist() == out_tok
        if m_policy == "tree":
            on = [0, 2]
            s1, c1 = oupd.update_M(s0, c0, st.tree["tok"].cpu().numpy()[on].reshape(-1),
                                   st.acc["argmax"].cpu().numpy()[on].reshape(-1))
            assert np.array_equal(w.M[0].cpu().numpy(), s1) and np.array_equal(w.M[1].cpu().numpy(), c1)
    c.fork(i32([0]), i32([1]))
    st.active[1] = True
    n = int(c.lengths[0])
    step(w.inputs())
    acc = st.acc["acc_len"].tolist()
    assert min(acc) >= 1 and c.lengths.tolist()[:2] == [n + acc[0], n + acc[1]]
    assert int(c.held[1]) == -(-(n + KMAX) // PAGE)


def test_root_tokens_are_checked():
    w = World(14)
    inp = w.inputs()
    for bad in (inp["root_tok"].long(), inp["root_tok"][:1]):
        with pytest.raises(ValueError):
            w.step.run(M_succ=w.M[0], M_cnt=w.M[1], **dict(inp, root_tok=bad))


def test_all_slots_idle():
    w = World(13)
    c, st = w.cache, w.step
    inp = w.inputs()
    st.active.zero_()
    state = [t.clone() for t in (c.block_table, c.held, c.page_refs, c.lengths, w.K, w.V, *w.M)]
    st.run(M_succ=w.M[0], M_cnt=w.M[1], **inp)
    torch.cuda.synchronize()
    assert int(st.status.item()) == 0 and st.acc["acc_len"].tolist() == [0] * B
    for t, x in zip((c.block_table, c.held, c.page_refs, c.lengths, w.K, w.V, *w.M), state):
        assert torch.equal(t, x)


def test_a_step_runs_on_the_caches_device(monkeypatch):
    """Whatever device is current: the calls that take their stream from the current device are made under the cache's.
    (One GPU here: the test sees to it that the step asks for it.)"""
    w = World(12)
    asked, inside = [], []

    class Device(torch.cuda.device):
        def __init__(self, d):
            asked.append(d)
            super().__init__(d)

    monkeypatch.setattr(torch.cuda, "device", Device)
    w.step.run(M_succ=w.M[0], M_cnt=w.M[1], inputs_ready=lambda x: inside.append(list(asked)), **w.inputs())
    torch.cuda.synchronize()
    assert len(inside) == 2 + LAYERS and all(x and x[0] == w.cache.device for x in inside)


def test_copy_on_write_survives_a_refused_reserve():
    """Two sequences share a partly filled page and no page is free: neither may write into it, and both stay as they
    are; once there are pages, the next step goes on as if that one had not been."""
    b = gb()
    w = World(7)
    c, st = w.cache, w.step
    c.free(i32([2]))
    c.fork(i32([0]), i32([2]))
    taken = c.page_refs == 0
    c.page_refs[taken] = 1  # another owner's
    K0, V0 = w.K.clone(), w.V.clone()
    before = [t.clone() for t in (c.block_table, c.held, c.page_refs, c.lengths)]
    inp = w.inputs()
    st.run(M_succ=w.M[0], M_cnt=w.M[1], **inp)
    torch.cuda.synchronize()
    assert int(st.status.item()) == b.STATUS_CACHE_OVERFLOW | b.STATUS_PAGE
    assert c.lengths.tolist() == [37, 48, 37]
    for t, x in zip((c.block_table, c.held, c.page_refs, c.lengths), before):
        assert torch.equal(t, x)
    assert torch.equal(w.K, K0) and torch.equal(w.V, V0)  # (no sequence had room of its own)
    st.status.zero_()
    c.page_refs[taken] = 0
    st.run(M_succ=w.M[0], M_cnt=w.M[1], **inp)
    torch.cuda.synchronize()
    assert int(st.status.item()) == 0
    acc = st.acc["acc_len"].tolist()
    assert c.lengths.tolist() == [37 + acc[0], 48 + acc[1], 37 + acc[2]] and min(acc) >= 1
    for s, n in enumerate((37, 48, 37)):
        for r in range(n):
            old, new = int(before[0][s, r // PAGE]), int(c.block_table[s, r // PAGE])
            assert torch.equal(w.K[:, new, r % PAGE], K0[:, old, r % PAGE])
            assert torch.equal(w.V[:, new, r % PAGE], V0[:, old, r % PAGE])


def test_refusals():
    from tree_verification_gb300.paged import PagedCache
    from tree_verification_gb300.paged_step import PagedVerifyStep
    w = World(2)
    with pytest.raises(ValueError):
        PagedVerifyStep(w.cfg, w.cache, 7)
    with pytest.raises(ValueError):
        PagedVerifyStep(w.cfg, w.cache, 8, m_policy="none")
    bare = PagedCache(list(w.K), list(w.V), w.cache.block_table, w.cache.lengths)
    with pytest.raises(ValueError):
        PagedVerifyStep(w.cfg, bare, 8)
