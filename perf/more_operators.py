"""Cases and plain forms of the operators around the verify step: norms, windows, log probabilities.

Three operators of models whose trees are verified:

* ``norm``     queries and keys normed head by head, rotated, and the new K and V rows written into their pages
* ``window``   attention over pages where a row sees the last ``window`` positions and the ``first`` tokens alone
               (causal chunks, draft trees, single tokens)
* ``logprob``  log probabilities of given tokens, entropy, rank and top alternatives of rows of logits

``run`` computes a case in its plain form, or, where ``own`` is true, by the framework's calls.
"""
import math
import random

import torch

own = False

HD = 128
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one request's 64-node draft tree, positions by depth (latency)
        dict(name="norm_tree", op="norm", dtype="bf16", B=1, new=64, ragged=False, tree=True, Hq=32, Hkv=8, rot=128,
             inter=False, theta=1000000.0, ctx=4096, ctx_low=4096, page=16, pad=0, norms="both"),
        # a serving batch decoding, one row each
        dict(name="norm_decode", op="norm", dtype="bf16", B=64, new=1, ragged=False, tree=False, Hq=64, Hkv=4, rot=128,
             inter=False, theta=1000000.0, ctx=4096, ctx_low=512, page=64, pad=0, norms="both"),
        # prompt chunks far into a long context: interleaved pairs over half of the head, fp16, padded rows behind them
        dict(name="norm_chunks", op="norm", dtype="fp16", B=3, new=3999, ragged=True, tree=False, Hq=64, Hkv=4, rot=64,
             inter=True, theta=10000.0, ctx=65536, ctx_low=30000, page=32, pad=37, norms="both"),
        # one sequence decoding far into a document: the window and four first tokens (latency)
        dict(name="window_one", op="window", dtype="bf16", B=1, new=1, ragged=False, tree=False, Hq=32, Hkv=8, ctx=65536,
             ctx_low=65536, page=16, layers=4, pad=0, window=1024, first=4, evict=False),
        # a serving batch decoding, lengths from short to long, pages behind the window given back
        dict(name="window_batch", op="window", dtype="bf16", B=64, new=1, ragged=False, tree=False, Hq=32, Hkv=8, ctx=32768,
             ctx_low=100, page=64, layers=2, pad=0, window=4096, first=0, evict=True),
        # one request's 64-node draft tree over a window
        dict(name="window_tree", op="window", dtype="bf16", B=1, new=64, ragged=False, tree=True, Hq=32, Hkv=8, ctx=20000,
             ctx_low=20000, page=16, layers=4, pad=0, window=2048, first=16, evict=False),
        # sixteen requests' draft trees, sixteen query heads a KV head
        dict(name="window_trees", op="window", dtype="bf16", B=16, new=64, ragged=False, tree=True, Hq=64, Hkv=4, ctx=16384,
             ctx_low=9000, page=64, layers=1, pad=0, window=4096, first=4, evict=True),
        # chunked prefill: a ragged batch of prompt chunks, some of them short, padded rows behind them, fp16
        dict(name="window_chunks", op="window", dtype="fp16", B=5, new=2048, ragged=True, tree=False, Hq=32, Hkv=8, ctx=8001,
             ctx_low=0, page=32, layers=1, pad=19, window=1024, first=64, evict=False),
        # after one request's verify step: its emitted tokens, five alternatives each (latency)
        dict(name="logprob_one", op="logprob", dtype="fp32", B=1, Kmax=64, acc=8, step=True, V=128256, top=5, T=1.0, pad=0,
             ban=0.0),
        # after a verify step of 64 requests: the emitted tokens' rows among all nodes' logits
        dict(name="logprob_batch", op="logprob", dtype="fp32", B=64, Kmax=64, acc=8, step=True, V=151936, top=5, T=0.7, pad=0,
             ban=0.0),
        # a prompt's tokens scored, bf16 logits of an odd vocabulary, no alternatives
        dict(name="logprob_prompt", op="logprob", dtype="bf16", B=1, Kmax=1999, acc=0, step=False, V=32003, top=0, T=1.0,
             pad=0, ban=0.0),
        # many rows of a large vocabulary with twenty alternatives, some tokens banned
        dict(name="logprob_large", op="logprob", dtype="fp32", B=16, Kmax=64, acc=0, step=False, V=151936, top=20, T=1.0, pad=0,
             ban=0.02),
    ]


def _span(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "window", "window", "window", "logprob", "logprob"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 3, 4, 8, 16] if Hkv < 8 else [1, 4, 5])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "norm":
        tree = rng.random() < 0.4
        new = rng.randint(2, 64) if tree else _span(rng, 1, 3000)
        B = _span(rng, 1, max(1, min(64, 5000 // new)))
        ctx = _span(rng, 64, 65536 if B < 4 else 4096)
        return dict(op=op, dtype=dtype, B=B, new=new, ragged=rng.random() < 0.5, tree=tree, Hq=Hq, Hkv=Hkv,
                    rot=rng.choice([0, 32, 64, 96, 128, 128]), inter=rng.random() < 0.5,
                    theta=rng.choice([10000.0, 500000.0, 1000000.0]), ctx=ctx, ctx_low=rng.randint(0, ctx), page=page,
                    pad=rng.choice([0, 0, 5, 33]), norms=rng.choice(["both", "both", "both", "q", "k"]))
    if op == "window":
        kind = rng.choice(["decode", "tree", "chunk"])
        if kind == "decode":
            new = rng.randint(1, 4)
            B = _span(rng, 1, 64)
            ctx = _span(rng, 16, min(65536, 524288 // B))
        elif kind == "tree":
            new = rng.randint(2, 64)
            B = _span(rng, 1, 16)
            ctx = _span(rng, 16, 20000)
        else:
            new = _span(rng, 5, 1500)
            B = _span(rng, 1, 4)
            ctx = _span(rng, 16, 8000)
        window, first = _span(rng, 1, 4096), rng.choice([0, 1, 4, 16, 100, 128, 300])
        while B * Hq * new * (window + first + new) > 5e8:  # scores that the plain form holds at once
            window = max(1, window // 2)
            new = max(1, new * 3 // 4)
        while B * (window + first + new) > 200000:
            window = window * 3 // 4
        low = 0 if rng.random() < 0.3 else rng.randint(ctx // 4, ctx)
        return dict(op=op, dtype=dtype, B=B, new=new, ragged=rng.random() < 0.5, tree=kind == "tree", Hq=Hq, Hkv=Hkv,
                    ctx=ctx, ctx_low=low, page=page, layers=rng.randint(1, 2), pad=rng.choice([0, 0, 7]), window=window,
                    first=first, evict=rng.random() < 0.4)
    V = _span(rng, 1000, 160000)
    step = rng.random() < 0.5
    if step:
        B, Kmax, acc = _span(rng, 1, 64), rng.randint(8, 64), rng.randint(1, 8)
        while B * Kmax * V > 6e8:
            B = max(1, B // 2)
    else:
        B, Kmax, acc = 1, _span(rng, 1, max(1, min(4000, 150000000 // V))), 0
    return dict(op=op, dtype=rng.choice(["fp32", "fp32", "bf16", "fp16"]), B=B, Kmax=Kmax, acc=acc, step=step, V=V,
                top=rng.choice([0, 1, 5, 8, 20, 32]), T=rng.choice([1.0, 1.0, 0.6, 1.3]), pad=rng.choice([0, 0, 0, 3, 64]),
                ban=rng.choice([0.0, 0.0, 0.05, 0.9]))


def _sizes(case):
    """(new rows, prefix length) of every sequence: fixed by the case, their order by the seed."""
    r = random.Random("%(op)s %(B)d %(new)d %(ctx)d %(ctx_low)d" % case)
    got = []
    for i in range(case["B"]):
        n = case["new"]
        if case.get("ragged") and i > 0:
            n = _span(r, 1, case["new"])
        got.append((n, case["ctx"] if i == 0 else r.randint(case["ctx_low"], case["ctx"])))
    return got


def _accepted(case):
    """Accepted rows of every request: fixed by the case, their order by the seed."""
    r = random.Random("%(B)d %(acc)d %(Kmax)d" % case)
    return [case["acc"] if b == 0 else r.randint(1, case["acc"]) for b in range(case["B"])]


def _tables(need, width, extra, rng, device):
    """Page numbers in shuffled order over a pool with `extra` spare pages; need[b] lists the entries that are held."""
    total = sum(len(x) for x in need) + extra
    ids = list(range(total))
    rng.shuffle(ids)
    table = torch.full((len(need), width), -1, dtype=torch.int32)
    at = 0
    for b, x in enumerate(need):
        table[b, x] = torch.tensor(ids[at:at + len(x)], dtype=torch.int32)
        at += len(x)
    return table.to(device), total


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    rng = random.Random(seed)
    dt = DTYPES[case["dtype"]]
    i32 = dict(dtype=torch.int32, device=dev)

    if case["op"] == "logprob":
        R, V = case["B"] * case["Kmax"], case["V"]
        store = torch.empty(R, V + case["pad"], dtype=dt, device=dev)  # (rows may lie further apart than they are long)
        store.normal_(generator=g)
        # rows are more or less sure of their token
        store *= (1.0 + 3.0 * torch.rand(R, 1, generator=g, device=dev)).to(dt)
        logits = store[:, :V]
        best = torch.randint(V, (R, 1), generator=g, device=dev)
        lift = torch.rand(R, 1, generator=g, device=dev) * 12
        logits.scatter_add_(1, best, lift.to(dt))
        other = torch.randint(V, (R, 1), generator=g, device=dev)
        token = torch.where(torch.rand(R, 1, generator=g, device=dev) < 0.6, best, other)
        if case["ban"] > 0:
            for lo in range(0, R, 64):
                part = logits[lo:lo + 64]
                ban = torch.rand(part.shape, generator=g, device=dev) < case["ban"]
                part.masked_fill_(ban.scatter_(1, token[lo:lo + 64], False), -math.inf)
        token = token[:, 0].int()
        s = dict(case=case, logits=logits, rows=None, tokens=token)
        if case["step"]:
            acc = _accepted(case)
            rng.shuffle(acc)
            rows = torch.full((case["B"], case["Kmax"]), -1, dtype=torch.int32)
            for b, a in enumerate(acc):
                path = [0] + sorted(rng.sample(range(1, case["Kmax"]), a - 1))
                rows[b, :a] = torch.tensor(path, dtype=torch.int32) + b * case["Kmax"]
            rows = rows.view(-1).to(dev)
            s["rows"] = rows
            s["tokens"] = torch.where(rows >= 0, token[rows.clamp(min=0).long()], -1).int()
        return s

    def pool(layers, pages):
        x = torch.empty(layers, pages, case["page"], case["Hkv"], HD, dtype=dt, device=dev)
        x.normal_(generator=g)
        return x

    sizes = _sizes(case)
    rng.shuffle(sizes)
    n, lens, page = [s[0] for s in sizes], [s[1] for s in sizes], case["page"]
    counts = [-(-(a + b) // page) for a, b in sizes]
    if case.get("evict"):
        need = [[j for j in range(c) if j * page < case["first"] or (j + 1) * page > b - case["window"] + 1]
                for c, b in zip(counts, lens)]
    else:
        need = [list(range(c)) for c in counts]
    table, total = _tables(need, max(1, max(counts)), 3, rng, dev)
    starts = [0]
    for x in n:
        starts.append(starts[-1] + x)
    N = starts[-1] + case.get("pad", 0)
    s = dict(case=case, table=table, lengths=torch.tensor(lens, **i32), starts=torch.tensor(starts, **i32), N=N,
             max_new=max(n))
    Hq, Hkv = case["Hq"], case["Hkv"]
    depth, masks = [], []
    if case["tree"]:
        for c in n:  # a tree of c nodes a request: every node hangs below one of those before it
            d, m = [0], [1]
            for i in range(1, c):
                p = rng.randrange(max(0, i - 12), i)
                d.append(d[p] + 1)
                m.append(m[p] | 1 << i)
            depth += d
            masks += [x - (1 << 64) if x >> 63 else x for x in m]
        masks += [0] * (N - len(masks))
    s["mask"] = torch.tensor(masks, dtype=torch.int64, device=dev) if masks else None
    s["depth"] = torch.tensor(depth + [0] * (N - len(depth)), device=dev) if masks else None
    if case["op"] == "norm":
        rot = case["rot"]
        i = torch.arange(rot // 2, dtype=torch.float64)
        s["freq"] = (case["theta"] ** (-2.0 * i / rot)).to(dev) if rot else None
        # Q, K and V as the projection leaves them: columns of one matrix, heads of unlike size
        heads = Hq + 2 * Hkv
        size = torch.exp(torch.randn(heads, 1, generator=g, device=dev)) * torch.exp(
            0.5 * torch.randn(heads, HD, generator=g, device=dev))
        qkv = (torch.randn(N, heads, HD, generator=g, device=dev) * size).to(dt)
        s["Q"], s["Kn"], s["Vn"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        weight = 1.0 + 0.3 * torch.randn(2, HD, generator=g, device=dev)
        s["qw"] = weight[0].clone() if case["norms"] != "k" else None
        s["kw"] = weight[1].clone() if case["norms"] != "q" else None
        s["eps"] = 1e-6
        s["pos"] = None
        if case["tree"]:
            base = [lens[b] for b in range(len(n)) for _ in range(n[b])]
            s["pos"] = torch.tensor([x + y for x, y in zip(base, depth)] + [0] * (N - len(base)), **i32)
        s["out"] = torch.zeros(N, Hq, HD, dtype=dt, device=dev)
        s["K"], s["V"] = pool(1, total), pool(1, total)
    else:
        # heads attend more or less sharply
        sharp = torch.rand(Hq, 1, generator=g, device=dev) * 2.5 + 0.5
        s["Q"] = [(torch.randn(N, Hq, HD, generator=g, device=dev) * sharp).to(dt) for _ in range(case["layers"])]
        s["out"] = [torch.zeros(N, Hq, HD, dtype=dt, device=dev) for _ in range(case["layers"])]
        s["K"], s["V"] = pool(case["layers"], total), pool(case["layers"], total)
    return s


# ------------------------------------------------------------------ the framework's calls
def _cache(s):
    """The cache's handle, which a user's program makes once for its pools and tables."""
    if "cache" not in s:
        from tree_verification_gb300.paged import PagedCache
        s["cache"] = PagedCache(list(s["K"]), list(s["V"]), s["table"], s["lengths"])
    return s["cache"]


def _run_own(s):
    case = s["case"]
    if case["op"] == "logprob":
        from tree_verification_gb300 import binding as gb
        if "ws" not in s:
            n, R, V = s["tokens"].numel(), s["logits"].shape[0], case["V"]
            ws = torch.empty(max(1, gb.graft_token_logprobs_workspace_size(n, V, case["top"])), dtype=torch.uint8,
                             device=s["logits"].device)
            s["ws"] = ws
        got = gb.graft_token_logprobs(s["logits"], s["tokens"], rows=s["rows"], top=case["top"], temperature=case["T"],
                                      ws=s["ws"])
        return got["logprob"], got["entropy"], got["rank"], got["top_id"], got["top_logprob"]
    c = _cache(s)
    if case["op"] == "norm":
        c.append(0, s["Q"], s["Kn"], s["Vn"], s["starts"], inv_freq=s["freq"], interleaved=case["inter"],
                 positions=s["pos"], out=s["out"], q_norm=s["qw"], k_norm=s["kw"], eps=s["eps"])
        return s["out"], s["K"], s["V"]
    c.plan(s["starts"], s["N"], case["Hq"], s["max_new"], tree=s["mask"] is not None, window=case["window"],
           first=case["first"])
    for layer, (q, o) in enumerate(zip(s["Q"], s["out"])):
        c.attend(layer, q, HD ** -0.5, mask=s["mask"], out=o, window=case["window"], first=case["first"])
    return s["out"]


# ------------------------------------------------------------------ the plain forms
def _rows(s):
    """Sequence and place in its chunk of every new row, and which rows are a sequence's."""
    at = torch.arange(s["N"], device=s["starts"].device)
    b = torch.bucketize(at, s["starts"][1:].long(), right=True)
    live = b < s["lengths"].numel()
    b = b.clamp(max=s["lengths"].numel() - 1)
    return b, at - s["starts"].long()[b], live


def _norm(s):
    case, page, rot = s["case"], s["case"]["page"], s["case"]["rot"]
    b, i, live = _rows(s)
    row = s["lengths"].long()[b] + i
    pos = row if s["pos"] is None else s["pos"].long()
    if rot:
        angle = pos.double()[:, None] * s["freq"]
        cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turned(x, weight):
        x = x.float()
        if weight is not None:
            x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * weight
        if rot:
            part, rest = x[..., :rot], x[..., rot:]
            if case["inter"]:
                x1, x2 = part[..., 0::2], part[..., 1::2]
                part = torch.stack((x1 * cos - x2 * sin, x1 * sin + x2 * cos), -1).flatten(-2)
            else:
                x1, x2 = part[..., :rot // 2], part[..., rot // 2:]
                part = torch.cat((x1 * cos - x2 * sin, x1 * sin + x2 * cos), -1)
            x = torch.cat((part, rest), -1)
        return x.to(s["out"].dtype)

    s["out"][live] = turned(s["Q"], s["qw"])[live]
    where = s["table"].long()[b, torch.where(live, row, 0) // page][live], (row % page)[live]
    s["K"][0][where] = turned(s["Kn"], s["kw"])[live]
    s["V"][0][where] = s["Vn"][live]
    return s["out"], s["K"], s["V"]


def _window(s):
    case, page, W, first = s["case"], s["case"]["page"], s["case"]["window"], s["case"]["first"]
    b, i, live = _rows(s)
    B, Hq, Hkv, M = case["B"], case["Hq"], case["Hkv"], s["max_new"]
    dev = s["starts"].device
    n, L = (s["starts"][1:] - s["starts"][:-1]).long()[:, None], s["lengths"].long()[:, None]
    # padded to [B, M] new rows against the first tokens and the rows from the earliest window on
    low = (L - W + 1).clamp(min=0)
    tail = low + torch.arange(int(min(W + M, s["table"].shape[1] * page)), device=dev)
    head = torch.arange(first, device=dev).expand(B, first)
    key = torch.cat((head, tail), 1)
    held = torch.cat((head < torch.minimum(low, L + n), tail < L + n), 1)
    key = torch.where(held, key, 0)
    place = torch.arange(M, device=dev)[None]
    slot = torch.where(place < n, s["starts"].long()[:-1, None] + place, 0)
    new = key - L  # a key's place among the new rows
    if s["mask"] is None:
        pos, at = L + place, key
        seen = key[:, None, :] <= pos[:, :, None]
    else:
        pos = L + s["depth"][slot]
        among = (s["starts"].long()[:-1, None] + new.clamp(min=0)).clamp(max=s["N"] - 1)
        at = torch.where(new < 0, key, L + s["depth"][among])
        bits = s["mask"][slot]
        seen = (bits[:, :, None] >> new.clamp(0, 63)[:, None, :] & 1).bool() | (new < 0)[:, None, :]
    seen = seen & held[:, None, :] & ((at[:, None, :] > pos[:, :, None] - W) | (at < first)[:, None, :])
    entry = s["table"].long().gather(1, key // page)
    entry = torch.where(held, entry, entry.clamp(min=0))
    line = (entry * page + key % page).flatten()
    outs = []
    for q, k, v, out in zip(s["Q"], s["K"], s["V"], s["out"]):
        kk = k.view(-1, Hkv, HD)[line].view(B, -1, Hkv, HD).float().permute(0, 2, 3, 1)
        vv = (v.view(-1, Hkv, HD)[line].view(B, -1, Hkv, HD) * held[:, :, None, None]).float().permute(0, 2, 1, 3)
        qq = q[slot].float().view(B, M, Hkv, Hq // Hkv, HD).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, HD)
        score = (qq @ kk * HD ** -0.5).view(B, Hkv, Hq // Hkv, M, -1)
        score = score.masked_fill(~seen[:, None, None], -math.inf)
        top = score.amax(-1, keepdim=True)
        w = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
        total = w.sum(-1, keepdim=True)
        w = (w / torch.where(total == 0, 1.0, total)).view(B, Hkv, (Hq // Hkv) * M, -1)
        o = (w @ vv).view(B, Hkv, Hq // Hkv, M, HD).permute(0, 3, 1, 2, 4).reshape(B, M, Hq, HD)
        out[live] = o[b[live], i[live]].to(out.dtype)
        outs.append(out)
    return outs


def _ordered(x):
    """Whole numbers in the order of 32-bit numbers (both zeros alike)."""
    bits = (x + 0.0).view(torch.int32).long()
    return torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)


def _logprob(s):
    case, V, top = s["case"], s["case"]["V"], s["case"]["top"]
    rows, tokens = s["rows"], s["tokens"].long()
    n, dev = tokens.numel(), tokens.device
    there = torch.ones(n, dtype=torch.bool, device=dev) if rows is None else rows >= 0
    logprob, entropy = torch.zeros(n, device=dev), torch.zeros(n, device=dev)
    rank = torch.full((n,), -1, dtype=torch.int32, device=dev)
    top_id = torch.full((n, top), -1, dtype=torch.int32, device=dev)
    top_lp = torch.zeros(n, top, device=dev)
    x = (s["logits"] if rows is None else s["logits"][rows[there].long()]).float()
    tok = tokens[there][:, None]
    given = x.gather(1, tok)
    ids = torch.arange(V, device=dev)
    rank[there] = ((x > given) | (x == given) & (ids < tok)).sum(1).int()
    z = x / case["T"]
    m = z.amax(1, keepdim=True)
    z = z - m
    e = torch.exp(z)
    total = e.sum(1, keepdim=True)
    entropy[there] = (total.log() - torch.where(e > 0, z * e, 0.0).sum(1, keepdim=True) / total)[:, 0]
    logprob[there] = (z.gather(1, tok) - total.log())[:, 0]
    if top:
        best = torch.topk(_ordered(x) * (1 << 20) + (V - 1 - ids), top, dim=1).indices
        top_id[there] = best.int()
        top_lp[there] = z.gather(1, best) - total.log()
    return logprob, entropy, rank, top_id, top_lp


def run(state):
    if own:
        return _run_own(state)
    return {"norm": _norm, "window": _window, "logprob": _logprob}[state["case"]["op"]](state)


def work(case):
    if case["op"] == "logprob":
        rows = sum(_accepted(case)) if case["step"] else case["B"] * case["Kmax"]
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": rows * (case["V"] * size + 4) + case["B"] * case["Kmax"] * (12 + 8 * case["top"]),
                "flops": 6 * rows * case["V"]}
    row = case["Hkv"] * HD * 2
    sizes = _sizes(case)
    N = sum(a for a, _ in sizes)
    if case["op"] == "norm":
        return {"bytes": 2 * N * (case["Hq"] * HD * 2 + 2 * row), "flops": N * (case["Hq"] + case["Hkv"]) * (4 * HD + 3 * case["rot"])}
    W, first = case["window"], case["first"]
    pairs, rows = 0, 0
    for n, L in sizes:
        low = max(0, L - W + 1)
        rows += min(first, low) + L + n - low
        for i in range(n):
            # (a tree's node is about as deep as the logarithm of its place)
            p = L + (int(math.log2(i + 1)) if case["tree"] else i)
            pairs += min(p + 1, W + min(first, max(0, p - W + 1)))
    one = 2 * N * case["Hq"] * HD * 2 + rows * row * 2
    return {"bytes": case["layers"] * one, "flops": case["layers"] * 4 * HD * case["Hq"] * pairs}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "logprob":
        n, top = s["tokens"].numel(), case["top"]
        dev = s["tokens"].device
        out = [torch.zeros(n, dtype=torch.float64, device=dev), torch.zeros(n, dtype=torch.float64, device=dev),
               torch.full((n,), -1, dtype=torch.int32, device=dev), torch.full((n, top), -1, dtype=torch.int32, device=dev),
               torch.zeros(n, top, dtype=torch.float64, device=dev)]
        which = torch.arange(n, device=dev) if s["rows"] is None else torch.nonzero(s["rows"] >= 0)[:, 0]
        for at in which.split(128):
            x = s["logits"][at if s["rows"] is None else s["rows"][at].long()].double()
            logp = x / case["T"] - torch.logsumexp(x / case["T"], 1, keepdim=True)
            p = torch.exp(logp)
            out[0][at] = logp[torch.arange(at.numel()), s["tokens"][at].long()]
            out[1][at] = -torch.where(p == 0, 0.0, p * logp).sum(1)
            order = torch.sort(x, dim=1, descending=True, stable=True).indices
            out[2][at] = torch.nonzero(order == s["tokens"][at].long()[:, None])[:, 1].int()
            out[3][at] = order[:, :top].int()
            out[4][at] = torch.take_along_dim(logp, order[:, :top], 1)
        return tuple(out)
    starts, lens, page = s["starts"].tolist(), s["lengths"].tolist(), case["page"]
    if case["op"] == "norm":
        out, K, V = s["out"].double(), s["K"].double(), s["V"].double()
        half = case["rot"] // 2
        for b in range(case["B"]):
            lo, hi = starts[b], starts[b + 1]
            row = torch.arange(lens[b], lens[b] + hi - lo, device=out.device)
            pos = (row if s["pos"] is None else s["pos"][lo:hi]).double()
            place = s["table"][b].long()[row // page]
            made = []
            for x, w in ((s["Q"][lo:hi].double(), s["qw"]), (s["Kn"][lo:hi].double(), s["kw"])):
                if w is not None:
                    x = w.double() * x * torch.rsqrt(x.square().sum(-1, keepdim=True) / HD + s["eps"])
                y = x.clone()
                if half:
                    turn = torch.polar(torch.ones((), dtype=torch.float64, device=out.device), pos[:, None, None] * s["freq"])
                    if case["inter"]:
                        z = torch.view_as_complex(x[..., :2 * half].reshape(*x.shape[:2], half, 2).contiguous()) * turn
                        y[..., :2 * half] = torch.view_as_real(z).reshape(*x.shape[:2], 2 * half)
                    else:
                        z = torch.complex(x[..., :half], x[..., half:2 * half]) * turn
                        y[..., :half], y[..., half:2 * half] = z.real, z.imag
                made.append(y)
            out[lo:hi] = made[0]
            K[0, place, row % page] = made[1]
            V[0, place, row % page] = s["Vn"][lo:hi].double()
        return out, K, V
    group, W, first = case["Hq"] // case["Hkv"], case["window"], case["first"]
    if work(case)["flops"] > 4e12:
        return None
    outs = [o.double() for o in s["out"]]
    for b in range(case["B"]):
        lo, hi, L = starts[b], starts[b + 1], lens[b]
        n = hi - lo
        # the cache rows that lie in held pages, with their positions; rows in none are nobody's to see
        row = torch.arange(L + n, device=s["table"].device)
        low = max(0, L - W + 1)
        row = row[(row < first) | (row >= low)]
        place = s["table"][b].long()[row // page], row % page
        at, pos = row.clone(), L + torch.arange(n, device=row.device)
        if s["mask"] is not None:
            pos = L + s["depth"][lo:hi]
            at[row >= L] = pos
        hidden = at[None] > pos[:, None]
        if s["mask"] is not None:
            for j in range(n):
                hidden[:, row == L + j] = ((s["mask"][lo:hi] & (1 << j if j < 63 else -(1 << 63))) == 0)[:, None]
        hidden |= (pos[:, None] - at[None] >= W) & (at >= first)[None]
        for q, k, v, out in zip(s["Q"], s["K"], s["V"], outs):
            k, v = k[place].double(), v[place].double()
            for h in range(case["Hq"]):
                score = q[lo:hi, h].double() @ k[:, h // group].T / math.sqrt(HD)
                score[hidden] = -math.inf
                out[lo:hi, h] = torch.softmax(score, -1) @ v[:, h // group]
    return outs
