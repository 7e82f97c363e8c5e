"""Cases and plain forms of the paged-cache operators.

Four operators on a KV cache kept in pages ([pages][page rows][KV heads][128] per layer, one row of page
numbers a sequence):

* ``append``    rotary positions of new Q and K rows, the new K and V rows written into their pages
* ``attend``    attention of the new rows over the pages (causal chunks, draft trees, single tokens)
* ``compact``   the accepted tree rows moved to the end of each sequence, in every layer
* ``turnover``  pages freed, shared by a fork, and reserved again with copies of the shared last pages

``run`` computes a case in its plain form, or, where ``own`` is true, by the framework's calls.
"""
import math
import random

import torch

own = False

HD = 128
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # one request's 64-node draft tree: positions by depth, wavelength-scaled table (latency)
        dict(name="append_tree", op="append", dtype="bf16", B=1, new=64, ragged=False, tree=True, Hq=32, Hkv=8, rot=128,
             inter=False, scaling="wave", theta=500000.0, ctx=4096, ctx_low=4096, page=16, pad=0),
        # prompt chunks far into a long context: interleaved pairs over half of the head, fp16, padded rows behind them
        dict(name="append_far_chunks", op="append", dtype="fp16", B=3, new=1999, ragged=True, tree=False, Hq=64, Hkv=4, rot=64,
             inter=True, scaling="yarn", theta=10000.0, ctx=65536, ctx_low=30000, page=32, pad=37),
        # one sequence decoding over a short prefix (latency)
        dict(name="decode_one", op="attend", dtype="bf16", B=1, new=1, ragged=False, tree=False, Hq=32, Hkv=8, ctx=4096,
             ctx_low=4096, page=16, layers=4, pad=0),
        # a serving batch decoding: 64 sequences of uneven length
        dict(name="decode_batch", op="attend", dtype="bf16", B=64, new=1, ragged=False, tree=False, Hq=32, Hkv=8, ctx=4096,
             ctx_low=512, page=64, layers=2, pad=0),
        # a few tokens at a time over one long document, fp16
        dict(name="few_long", op="attend", dtype="fp16", B=1, new=4, ragged=False, tree=False, Hq=32, Hkv=8, ctx=65536,
             ctx_low=65536, page=32, layers=2, pad=0),
        # one request's 64-node draft tree over a 4096-token prefix
        dict(name="verify_one", op="attend", dtype="bf16", B=1, new=64, ragged=False, tree=True, Hq=32, Hkv=8, ctx=4096,
             ctx_low=4096, page=16, layers=4, pad=0),
        # sixteen requests' draft trees, sixteen query heads a KV head
        dict(name="verify_wide", op="attend", dtype="bf16", B=16, new=64, ragged=False, tree=True, Hq=64, Hkv=4, ctx=8192,
             ctx_low=8192, page=64, layers=1, pad=0),
        # chunked prefill: a ragged batch of prompt chunks, some of them short, padded rows behind them
        dict(name="chunk_ragged", op="attend", dtype="bf16", B=5, new=2048, ragged=True, tree=False, Hq=32, Hkv=8, ctx=6001,
             ctx_low=0, page=16, layers=1, pad=19),
        # after a verify step of 64 requests: accepted rows compacted in every layer
        dict(name="compact_batch", op="compact", dtype="bf16", B=64, new=64, Hq=32, Hkv=8, ctx=128, ctx_low=16, page=16,
             layers=36, acc=6),
        # the same for one request with a long accepted path
        dict(name="compact_one", op="compact", dtype="bf16", B=1, new=64, Hq=32, Hkv=8, ctx=500, ctx_low=500, page=32,
             layers=32, acc=8),
        # parallel samples of 16 prompts: the old samples' pages freed, the prompts forked, room reserved for the next step
        dict(name="turnover_wide", op="turnover", dtype="bf16", parents=16, kids=3, Hkv=8, ctx=250, ctx_low=20, new=64,
             page=16, layers=36),
        # one prompt forked once
        dict(name="turnover_one", op="turnover", dtype="bf16", parents=1, kids=1, Hkv=8, ctx=201, ctx_low=201, new=64,
             page=64, layers=32),
    ]


def _span(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "compact", "turnover"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 3, 4, 8, 16] if Hkv < 8 else [1, 4, 5])
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        tree = rng.random() < 0.4
        new = rng.randint(2, 64) if tree else _span(rng, 1, 2000)
        B = _span(rng, 1, max(1, min(64, 4096 // new)))
        ctx = _span(rng, 64, 65536 if B < 4 else 4096)
        return dict(op=op, dtype=dtype, B=B, new=new, ragged=rng.random() < 0.5, tree=tree, Hq=Hq, Hkv=Hkv,
                    rot=rng.choice([32, 64, 96, 128]), inter=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "wave", "yarn"]), theta=rng.choice([10000.0, 500000.0, 1000000.0]),
                    ctx=ctx, ctx_low=rng.randint(0, ctx), page=page, pad=rng.choice([0, 0, 5, 33]))
    if op == "attend":
        kind = rng.choice(["decode", "tree", "chunk"])
        if kind == "decode":
            new = rng.randint(1, 4)
            B = _span(rng, 1, 64)
            ctx = _span(rng, 16, min(65536, 262144 // B))
        elif kind == "tree":
            new = rng.randint(2, 64)
            B = _span(rng, 1, 16)
            ctx = _span(rng, 16, 8192)
        else:
            new = _span(rng, 5, 1500)
            B = _span(rng, 1, 4)
            ctx = _span(rng, 16, 6000)
        while B * Hq * new * (ctx + new) > 5e8:  # scores that the plain form holds at once
            ctx = max(16, ctx // 2)
            new = max(1, new * 3 // 4)
        low = 0 if rng.random() < 0.3 else rng.randint(ctx // 4, ctx)
        return dict(op=op, dtype=dtype, B=B, new=new, ragged=rng.random() < 0.5, tree=kind == "tree", Hq=Hq, Hkv=Hkv,
                    ctx=ctx, ctx_low=low, page=page, layers=rng.randint(1, 2), pad=rng.choice([0, 0, 7]))
    if op == "compact":
        ctx = _span(rng, 16, 500)
        return dict(op=op, dtype=dtype, B=_span(rng, 1, 64), new=rng.randint(24, 64), Hq=Hq, Hkv=Hkv, ctx=ctx,
                    ctx_low=rng.randint(0, ctx), page=rng.choice([16, 32, 64]), layers=rng.randint(1, 32), acc=rng.randint(1, 8))
    ctx = _span(rng, 16, 300)
    return dict(op=op, dtype=dtype, parents=_span(rng, 1, 16), kids=rng.randint(1, 3), Hkv=Hkv, ctx=ctx,
                ctx_low=rng.randint(0, ctx), new=rng.randint(1, 64), page=rng.choice([16, 32, 64]), layers=rng.randint(1, 32))


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


def _frequencies(case, device):
    """Angular frequency of every rotated pair, in 64 bits, scaled for long contexts; and the factor on both rows."""
    rot, theta = case["rot"], case["theta"]
    i = torch.arange(rot // 2, dtype=torch.float64)
    w = theta ** (-2.0 * i / rot)
    factor = 1.0
    if case["scaling"] == "linear":
        w = w / 4.0
    elif case["scaling"] == "wave":  # long waves stretched by 8, short ones kept, a blend between
        wave = 2 * math.pi / w
        blend = ((8192.0 / wave - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        w = (1 - blend) * w / 8.0 + blend * w
    elif case["scaling"] == "yarn":
        at = [rot * math.log(8192.0 / (2 * math.pi * turns)) / (2 * math.log(theta)) for turns in (32.0, 1.0)]
        low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        ramp = ((i - low) / max(high - low, 1e-3)).clamp(0, 1)
        w = w * (1 - ramp) + w / 16.0 * ramp
        factor = 0.1 * math.log(16.0) + 1.0
    return w.to(device), factor


def _tables(lengths, page, extra, rng, device):
    """Page numbers of sequences that hold `lengths` rows, in shuffled order over a pool with `extra` spare pages."""
    counts = [-(-n // page) for n in lengths]
    total = sum(counts) + extra
    ids = list(range(total))
    rng.shuffle(ids)
    table = torch.full((len(lengths), max(1, max(counts))), -1, dtype=torch.int32)
    at = 0
    for b, c in enumerate(counts):
        table[b, :c] = torch.tensor(ids[at:at + c], dtype=torch.int32)
        at += c
    return table.to(device), counts, total


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    rng = random.Random(seed)
    dt = DTYPES[case["dtype"]]
    i32 = dict(dtype=torch.int32, device=dev)

    def rand(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device=dev, dtype=torch.float32) * scale).to(dt)

    def pool(layers, pages):
        x = torch.empty(layers, pages, case["page"], case["Hkv"], HD, dtype=dt, device=dev)
        x.normal_(generator=g)
        return x

    if case["op"] == "turnover":
        P, kids = case["parents"], case["kids"]
        r = random.Random("%(parents)d %(kids)d %(ctx)d %(ctx_low)d" % case)
        lens = [case["ctx"]] + [r.randint(case["ctx_low"], case["ctx"]) for _ in range(P - 1)]
        rng.shuffle(lens)
        S, page = P * (1 + kids), case["page"]
        room = -(-(case["ctx"] + case["new"]) // page) + 1
        table, counts, used = _tables(lens, page, P * kids * room, rng, dev)
        full = torch.full((S, room), -1, **i32)
        full[:P, :table.shape[1]] = table
        # (the samples of the step before hold pages of their own)
        free = torch.ones(used, dtype=torch.bool)
        free[table[table >= 0].cpu().long()] = False
        spare = torch.nonzero(free).flatten().tolist()
        rng.shuffle(spare)
        full[P:, 0] = torch.tensor(spare[:P * kids], **i32)
        refs = torch.zeros(used, **i32)
        refs[full[full >= 0].long()] = 1
        src = torch.arange(P, **i32).repeat_interleave(kids)
        dst = torch.arange(P, S, **i32)
        new = torch.zeros(S, **i32)
        new[P:] = case["new"]
        return dict(case=case, K=pool(case["layers"], used), V=pool(case["layers"], used), table=full, refs=refs,
                    held=torch.tensor(counts + [1] * (S - P), **i32), lengths=torch.tensor(lens + [page // 2] * (S - P), **i32),
                    src=src, dst=dst, new=new)

    sizes = _sizes(case)
    rng.shuffle(sizes)
    n, lens = [s[0] for s in sizes], [s[1] for s in sizes]
    table, counts, total = _tables([a + b for a, b in sizes], case["page"], 3, rng, dev)
    starts = [0]
    for x in n:
        starts.append(starts[-1] + x)
    N = starts[-1] + case.get("pad", 0)
    s = dict(case=case, table=table, lengths=torch.tensor(lens, **i32), starts=torch.tensor(starts, **i32), N=N,
             max_new=max(n))
    Hq, Hkv = case["Hq"], case["Hkv"]
    depth, masks = [], []
    if case.get("tree"):
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
    if case["op"] == "append":
        s["freq"], s["factor"] = _frequencies(case, dev)
        # Q, K and V as the projection leaves them: columns of one matrix
        qkv = rand(N, (Hq + 2 * Hkv) * HD)
        s["Q"], s["Kn"], s["Vn"] = qkv[:, :Hq * HD], qkv[:, Hq * HD:(Hq + Hkv) * HD], qkv[:, (Hq + Hkv) * HD:]
        s["Q"], s["Kn"], s["Vn"] = s["Q"].view(N, Hq, HD), s["Kn"].view(N, Hkv, HD), s["Vn"].view(N, Hkv, HD)
        s["pos"] = None
        if case["tree"]:
            base = [lens[b] for b in range(len(n)) for _ in range(n[b])]
            s["pos"] = torch.tensor([x + y for x, y in zip(base, depth)] + [0] * (N - len(base)), **i32)
        s["out"] = torch.zeros(N, Hq, HD, dtype=dt, device=dev)
        s["K"], s["V"] = pool(1, total), pool(1, total)
    elif case["op"] == "attend":
        # heads attend more or less sharply
        sharp = torch.rand(Hq, 1, generator=g, device=dev) * 2.5 + 0.5
        s["Q"] = [(torch.randn(N, Hq, HD, generator=g, device=dev) * sharp).to(dt) for _ in range(case["layers"])]
        s["out"] = [torch.zeros(N, Hq, HD, dtype=dt, device=dev) for _ in range(case["layers"])]
        s["K"], s["V"] = pool(case["layers"], total), pool(case["layers"], total)
    else:
        acc, path = [], []
        r = random.Random("%(B)d %(acc)d" % case)
        for c in n:
            a = r.randint(1, case["acc"])
            acc.append(a)
            # the root, then nodes in rising order; none of those among the first `acc` (their rows would be
            # taken over by the first pass, and a pass is to be repeated on its state)
            path.append([0] + sorted(rng.sample(range(case["acc"], c), a - 1)) + [-1] * (c - a))
        s["acc"], s["path"] = torch.tensor(acc, **i32), torch.tensor(path, **i32)
        s["after"] = torch.zeros(len(n), **i32)
        s["K"], s["V"] = pool(case["layers"], total), pool(case["layers"], total)
    return s


# ------------------------------------------------------------------ the framework's calls
def _cache(s):
    """The cache's handle, which a user's program makes once for its pools and tables."""
    if "cache" not in s:
        from tree_verification_gb300.paged import PagedCache
        s["cache"] = PagedCache(list(s["K"]), list(s["V"]), s["table"], s["lengths"], page_refs=s.get("refs"),
                                held=s.get("held"))
    return s["cache"]


def _run_own(s):
    c, op = _cache(s), s["case"]["op"]
    if op == "append":
        c.append(0, s["Q"], s["Kn"], s["Vn"], s["starts"], inv_freq=s["freq"], interleaved=s["case"]["inter"],
                 positions=s["pos"], factor=s["factor"], out=s["out"])
        return s["out"], s["K"], s["V"]
    if op == "attend":
        c.plan(s["starts"], s["N"], s["case"]["Hq"], s["max_new"], tree=s["mask"] is not None)
        for layer, (q, o) in enumerate(zip(s["Q"], s["out"])):
            c.attend(layer, q, HD ** -0.5, mask=s["mask"], out=o)
        return s["out"]
    if op == "compact":
        c.compact(s["path"], s["acc"], lengths_out=s["after"])
        return s["K"], s["V"], s["after"]
    c.free(s["dst"])
    c.fork(s["src"], s["dst"])
    c.reserve(s["new"])
    return s["K"], s["V"], s["table"], s["refs"], s["held"], s["lengths"]


# ------------------------------------------------------------------ the plain forms
def _rows(s):
    """Sequence and place in its chunk of every new row, and which rows are a sequence's."""
    at = torch.arange(s["N"], device=s["starts"].device)
    b = torch.bucketize(at, s["starts"][1:].long(), right=True)
    live = b < s["lengths"].numel()
    b = b.clamp(max=s["lengths"].numel() - 1)
    return b, at - s["starts"].long()[b], live


def _append(s):
    case, page, rot = s["case"], s["case"]["page"], s["case"]["rot"]
    b, i, live = _rows(s)
    row = s["lengths"].long()[b] + i
    pos = row if s["pos"] is None else s["pos"].long()
    angle = pos.double()[:, None] * s["freq"]
    cos, sin = (angle.cos() * s["factor"]).float()[:, None], (angle.sin() * s["factor"]).float()[:, None]

    def turned(x):
        x = x.float()
        part, rest = x[..., :rot], x[..., rot:]
        if case["inter"]:
            x1, x2 = part[..., 0::2], part[..., 1::2]
            part = torch.stack((x1 * cos - x2 * sin, x1 * sin + x2 * cos), -1).flatten(-2)
        else:
            x1, x2 = part[..., :rot // 2], part[..., rot // 2:]
            part = torch.cat((x1 * cos - x2 * sin, x1 * sin + x2 * cos), -1)
        return torch.cat((part, rest), -1).to(s["Q"].dtype)

    s["out"][live] = turned(s["Q"])[live]
    where = s["table"].long()[b, torch.where(live, row, 0) // page][live], (row % page)[live]
    s["K"][0][where] = turned(s["Kn"])[live]
    s["V"][0][where] = s["Vn"][live]
    return s["out"], s["K"], s["V"]


def _attend(s):
    case, page = s["case"], s["case"]["page"]
    b, i, live = _rows(s)
    B, Hq, Hkv = case["B"], case["Hq"], case["Hkv"]
    M, width = s["max_new"], s["table"].shape[1] * page
    n = (s["starts"][1:] - s["starts"][:-1]).long()
    L = s["lengths"].long()
    # padded to [B, M] new rows against every row that the tables can hold
    slot = s["starts"].long()[:-1, None] + torch.arange(M, device=n.device)
    there = torch.arange(M, device=n.device)[None] < n[:, None]
    slot = torch.where(there, slot, 0)
    key = torch.arange(width, device=n.device) - L[:, None]  # a key's place among the new rows, [B, width]
    place = torch.arange(M, device=n.device)
    if s["mask"] is None:
        seen = key[:, None, :] <= place[None, :, None]
    else:
        bits = s["mask"][slot]
        seen = (bits[:, :, None] >> key.clamp(0, 63)[:, None, :] & 1).bool() & (key < 64)[:, None, :] | (key < 0)[:, None, :]
    held = torch.arange(width, device=n.device)[None] < (L + n)[:, None]
    seen = seen & held[:, None, :]
    outs = []
    for q, k, v, out in zip(s["Q"], s["K"], s["V"], s["out"]):
        pages = s["table"].long().clamp(min=0)
        kk = k[pages].view(B, width, Hkv, HD).float().permute(0, 2, 3, 1)
        vv = (v[pages].view(B, width, Hkv, HD) * held[:, :, None, None]).float().permute(0, 2, 1, 3)
        qq = q[slot].float().view(B, M, Hkv, Hq // Hkv, HD).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, HD)
        score = (qq @ kk * HD ** -0.5).view(B, Hkv, Hq // Hkv, M, width)
        score = score.masked_fill(~seen[:, None, None], -math.inf)
        top = score.amax(-1, keepdim=True)
        w = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
        total = w.sum(-1, keepdim=True)
        w = (w / torch.where(total == 0, 1.0, total)).view(B, Hkv, -1, width)
        o = (w @ vv).view(B, Hkv, Hq // Hkv, M, HD).permute(0, 3, 1, 2, 4).reshape(B, M, Hq, HD)
        out[live] = o[b[live], i[live]].to(out.dtype)
        outs.append(out)
    return outs


def _compact(s):
    page = s["case"]["page"]
    path, acc, L = s["path"].long(), s["acc"].long(), s["lengths"].long()
    t = torch.arange(path.shape[1], device=path.device)[None]
    b, t = torch.nonzero(t < acc[:, None], as_tuple=True)
    src, dst = L[b] + path[b, t], L[b] + t
    table = s["table"].long()
    a, z = (table[b, src // page], src % page), (table[b, dst // page], dst % page)
    s["K"][:, z[0], z[1]] = s["K"][:, a[0], a[1]]
    s["V"][:, z[0], z[1]] = s["V"][:, a[0], a[1]]
    s["after"].copy_(L + acc)
    return s["K"], s["V"], s["after"]


def _turnover(s):
    page, table, refs, held, L = s["case"]["page"], s["table"], s["refs"], s["held"], s["lengths"]
    idx = torch.arange(table.shape[1], device=table.device)[None]
    src, dst = s["src"].long(), s["dst"].long()
    # free
    gone = table[dst][idx < held[dst][:, None]].long()
    refs.index_add_(0, gone, torch.full_like(gone, -1, dtype=torch.int32))
    table[dst], held[dst], L[dst] = -1, 0, 0
    # fork
    count = (L[src] + page - 1) // page
    rows = torch.where(idx < count[:, None], table[src], -1)
    shared = rows[rows >= 0].long()
    refs.index_add_(0, shared, torch.ones_like(shared, dtype=torch.int32))
    table[dst], held[dst], L[dst] = rows, count.int(), L[src]
    # reserve: pages that the new rows touch and that are missing or shared, the lowest free ones first
    need = torch.where(s["new"] > 0, (L + s["new"] + page - 1) // page, held)
    first = L // page
    has = idx < held[:, None]
    wanted = (s["new"] > 0)[:, None] & (idx >= first[:, None]) & (idx < need[:, None]) & (~has | (refs[table.clamp(min=0).long()] > 1))
    b, j = torch.nonzero(wanted, as_tuple=True)
    fresh = torch.nonzero(refs == 0).flatten()[:b.numel()]
    was = torch.where(has[b, j], table[b, j], -1).long()
    copied = (was >= 0) & (j == first[b])
    keep = (torch.arange(page, device=table.device)[None] < (L[b] % page)[:, None])[copied]
    for pool in (s["K"], s["V"]):
        old, new = pool[:, was[copied]], pool[:, fresh[copied]]
        pool[:, fresh[copied]] = torch.where(keep[None, :, :, None, None], old, new)
    left = was[was >= 0]
    refs.index_add_(0, left, torch.full_like(left, -1, dtype=torch.int32))
    refs[fresh] = 1
    table[b, j] = fresh.int()
    held.copy_(torch.maximum(held, need))
    return s["K"], s["V"], table, refs, held, L


def run(state):
    if own:
        return _run_own(state)
    return {"append": _append, "attend": _attend, "compact": _compact, "turnover": _turnover}[state["case"]["op"]](state)


def work(case):
    row = case["Hkv"] * HD * 2
    if case["op"] == "turnover":
        r = random.Random("%(parents)d %(kids)d %(ctx)d %(ctx_low)d" % case)
        lens = [case["ctx"]] + [r.randint(case["ctx_low"], case["ctx"]) for _ in range(case["parents"] - 1)]
        rows = sum(x % case["page"] for x in lens) * case["kids"]
        ids = sum(-(-(x + case["new"]) // case["page"]) for x in lens) * case["kids"]
        return {"bytes": rows * row * 2 * 2 * case["layers"] + ids * 4 * 4, "flops": 0}
    sizes = _sizes(case)
    N = sum(a for a, _ in sizes)
    if case["op"] == "append":
        return {"bytes": 2 * N * (case["Hq"] * HD * 2 + 2 * row), "flops": 3 * N * (case["Hq"] + case["Hkv"]) * case["rot"]}
    if case["op"] == "attend":
        # (a tree's node sees about as many of its tree's rows as the tree is deep)
        pairs = sum(a * b + (a * (math.log2(a) + 1) if case["tree"] else a * (a + 1) / 2) for a, b in sizes)
        one = 2 * N * case["Hq"] * HD * 2 + sum(a + b for a, b in sizes) * row * 2
        return {"bytes": case["layers"] * one, "flops": case["layers"] * 4 * HD * case["Hq"] * pairs}
    r = random.Random("%(B)d %(acc)d" % case)
    moved = sum(r.randint(1, case["acc"]) - 1 for _ in range(case["B"]))  # (the root's row stays where it is)
    return {"bytes": max(1, moved) * row * 2 * 2 * case["layers"], "flops": 0}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        out, K, V = s["out"].double(), s["K"].double(), s["V"].double()
        starts, lens = s["starts"].tolist(), s["lengths"].tolist()
        half = case["rot"] // 2
        for b in range(case["B"]):
            lo, hi = starts[b], starts[b + 1]
            row = torch.arange(lens[b], lens[b] + hi - lo, device=out.device)
            pos = (row if s["pos"] is None else s["pos"][lo:hi]).double()
            turn = torch.polar(torch.full((), s["factor"], dtype=torch.float64, device=out.device),
                               pos[:, None, None] * s["freq"])
            place = s["table"][b].long()[row // case["page"]]
            rotated = []
            for x in (s["Q"][lo:hi].double(), s["Kn"][lo:hi].double()):
                y = x.clone()
                if case["inter"]:
                    z = torch.view_as_complex(x[..., :2 * half].reshape(*x.shape[:2], half, 2).contiguous()) * turn
                    y[..., :2 * half] = torch.view_as_real(z).reshape(*x.shape[:2], 2 * half)
                else:
                    z = torch.complex(x[..., :half], x[..., half:2 * half]) * turn
                    y[..., :half], y[..., half:2 * half] = z.real, z.imag
                rotated.append(y)
            out[lo:hi] = rotated[0]
            K[0, place, row % case["page"]] = rotated[1]
            V[0, place, row % case["page"]] = s["Vn"][lo:hi].double()
        return out, K, V
    if case["op"] == "attend":
        if work(case)["flops"] > 6e12:
            return None
        starts, lens, group = s["starts"].tolist(), s["lengths"].tolist(), case["Hq"] // case["Hkv"]
        outs = [o.double() for o in s["out"]]
        for b in range(case["B"]):
            lo, hi, L = starts[b], starts[b + 1], lens[b]
            n = hi - lo
            row = torch.arange(L + n, device=s["table"].device)
            place = s["table"][b].long()[row // case["page"]], row % case["page"]
            unseen = torch.zeros(n, L + n, dtype=torch.bool, device=row.device)
            if s["mask"] is None:
                unseen[:, L:] = torch.ones(n, n, dtype=torch.bool, device=row.device).triu(1)
            else:
                for j in range(n):
                    unseen[:, L + j] = (s["mask"][lo:hi] & (1 << j if j < 63 else -(1 << 63))) == 0
            for q, k, v, out in zip(s["Q"], s["K"], s["V"], outs):
                k, v = k[place].double(), v[place].double()
                for h in range(case["Hq"]):
                    score = q[lo:hi, h].double() @ k[:, h // group].T / math.sqrt(HD)
                    score[unseen] = -math.inf
                    out[lo:hi, h] = torch.softmax(score, -1) @ v[:, h // group]
        return outs
    if case["op"] == "compact":
        for pool in (s["K"], s["V"]):
            for b, (L, a) in enumerate(zip(s["lengths"].tolist(), s["acc"].tolist())):
                table, path = s["table"][b].tolist(), s["path"][b].tolist()
                for t in range(a):
                    x, y = L + path[t], L + t
                    pool[:, table[y // case["page"]], y % case["page"]] = pool[:, table[x // case["page"]], x % case["page"]]
        return s["K"].double(), s["V"].double(), s["lengths"] + s["acc"]
    page, refs, held, lens = case["page"], s["refs"].tolist(), s["held"].tolist(), s["lengths"].tolist()
    table = s["table"].tolist()
    for d in s["dst"].tolist():
        for j in range(held[d]):
            refs[table[d][j]] -= 1
        table[d], held[d], lens[d] = [-1] * len(table[d]), 0, 0
    for a, d in zip(s["src"].tolist(), s["dst"].tolist()):
        held[d], lens[d] = -(-lens[a] // page), lens[a]
        for j in range(held[d]):
            table[d][j] = table[a][j]
            refs[table[a][j]] += 1
    free = [p for p, r in enumerate(refs) if r == 0]
    before = list(refs)
    for b, n in enumerate(s["new"].tolist()):
        if n == 0:
            continue
        need = -(-(lens[b] + n) // page)
        for j in range(lens[b] // page, need):
            old = table[b][j] if j < held[b] else -1
            if old >= 0 and before[old] == 1:
                continue
            new = free.pop(0)
            refs[new], table[b][j] = 1, new
            if old >= 0:
                refs[old] -= 1
                rows = lens[b] - j * page
                if rows > 0:
                    s["K"][:, new, :rows] = s["K"][:, old, :rows].clone()
                    s["V"][:, new, :rows] = s["V"][:, old, :rows].clone()
        held[b] = max(held[b], need)
    i32 = dict(dtype=torch.int32, device=s["table"].device)
    return (s["K"].double(), s["V"].double(), torch.tensor(table, **i32), torch.tensor(refs, **i32),
            torch.tensor(held, **i32), torch.tensor(lens, **i32))
