"""The paged K/V cache, case by case: inputs, plain forms, 64-bit values.

Four operators of a serving loop whose cache is cut into pages:

  rope    norms of the queries' and keys' heads, the rotation by position, the rows into pages
  attn    attention of a draft tree (one node: ordinary decoding) over the pages
  assign  which pages a sequence holds: forks, reorders, new rows, pages given back
  commit  the accepted path's rows moved behind the committed ones, in every layer

Pages are k_pages, v_pages [layers, N, Hkv, page, d] in bf16 (one layer of them: without the
first dimension); row r of sequence b lies in page page_table[b, r // page], row r % page.
`run` gives the plain form, in torch operations and 32 bits, or with `own` the library's calls on
the same state.
"""
import math
import random

import torch

own = False

D = 128          # head dimension


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one new token of a small batch: the latency of the call
        dict(name="rope_decode", op="rope", B=8, n=1, q_min=1, q_max=1, pos_max=8000, Hq=32, Hkv=8, page=64, norm=True, rot=128,
             pairs="halves", dest="pages", lens=1),
        # the nodes of a full batch's draft trees, straight into the pages
        dict(name="rope_trees", op="rope", B=64, n=60, q_min=60, q_max=60, pos_max=4096, Hq=32, Hkv=8, page=64, norm=False, rot=128,
             pairs="halves", dest="pages", lens=2),
        # a server's mixed batch of prompts: rows packed for the prompt's attention, and into the pages
        dict(name="rope_prompts", op="rope", B=24, n=0, q_min=5, q_max=4096, pos_max=0, Hq=32, Hkv=8, page=64, norm=True, rot=128,
             pairs="halves", dest="both", lens=3),
        # plain decoding, one long sequence, small pages: the work has to be split over its length
        dict(name="decode_one", op="attn", B=1, n=1, L_min=20011, L_max=20011, Hq=32, Hkv=8, page=16, lens=4),
        # plain decoding of a ragged batch with long sequences in it
        dict(name="decode_ragged", op="attn", B=48, n=1, L_min=100, L_max=30000, Hq=64, Hkv=8, page=64, lens=5),
        # the verify step's own shape: 60-node trees at 4096 committed tokens
        dict(name="tree_b64", op="attn", B=64, n=60, L_min=4096, L_max=4096, Hq=32, Hkv=8, page=64, lens=6),
        # trees over sequences of very different lengths, small pages
        dict(name="tree_ragged", op="attn", B=16, n=48, L_min=33, L_max=16000, Hq=64, Hkv=8, page=16, lens=7),
        # room for the next step's rows: numbers alone, nothing is copied
        dict(name="assign_grow", op="assign", kind="grow", layers=32, B=64, L_min=100, L_max=2000, grow=60, Hkv=8, page=64, spare=140, lens=8),
        # one prompt continued in every slot
        dict(name="assign_fork", op="assign", kind="fork", layers=32, B=32, L_min=3000, L_max=3000, grow=1, Hkv=8, page=64, spare=70, lens=9),
        # a beam search's step: slots continue one another, some end
        dict(name="assign_reorder", op="assign", kind="reorder", layers=32, B=64, L_min=10, L_max=700, grow=8, Hkv=8, page=32, spare=300, lens=10),
        # one step of one sequence, all layers
        dict(name="commit_one", op="commit", layers=32, B=1, n=60, depth=6, L_min=2048, L_max=2048, Hkv=8, page=64, lens=11),
        # one step of a full batch, all layers
        dict(name="commit_b64", op="commit", layers=32, B=64, n=60, depth=8, L_min=20, L_max=500, Hkv=8, page=64, lens=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    return rng.choice([(32, 8), (64, 8), (40, 40), (32, 32), (8, 2), (28, 4), (40, 8), (6, 2), (16, 1), (1, 1)])


def draw(rng):
    op = rng.choice(["rope", "attn", "attn", "assign", "commit"])
    lens = rng.randrange(1 << 20)
    Hq, Hkv = _heads(rng)
    page = rng.choice([16, 32, 64, 128])
    if op == "rope":
        while True:
            B, hi = _log_int(rng, 1, 64), _log_int(rng, 1, 4096)
            n = rng.choice([0, 1, rng.randint(2, 64)])
            lo, hi = (n, n) if n else (_log_int(rng, 1, hi), hi)
            if B * hi * (Hq + Hkv) <= 24 * 1400 * 40:
                return dict(op=op, B=B, n=n, q_min=lo, q_max=hi, pos_max=rng.choice([0, _log_int(rng, 1, 130000)]), Hq=Hq, Hkv=Hkv,
                            page=page, norm=rng.random() < 0.5, rot=rng.choice([128, 128, 64, 32, 96]),
                            pairs=rng.choice(["halves", "halves", "neighbours"]), dest=rng.choice(["pages", "packed", "both"]), lens=lens)
    if op == "attn":
        while True:
            B, n, hi = _log_int(rng, 1, 64), rng.choice([1, 1, 2, _log_int(rng, 3, 64), rng.randint(3, 64)]), _log_int(rng, 1, 32000)
            if B * Hkv * hi <= 64 * 8 * 4096 and B * Hq * n * hi <= 64 * 32 * 60 * 4096:
                return dict(op=op, B=B, n=n, L_min=_log_int(rng, 1, hi) - 1, L_max=hi, Hq=Hq, Hkv=Hkv, page=page, lens=lens)
    layers, B = _log_int(rng, 1, 48), _log_int(rng, 1, 64)
    if op == "assign":
        while True:
            hi = _log_int(rng, 1, 3000)
            kind = rng.choice(["grow", "fork", "reorder"])
            case = dict(op=op, kind=kind, layers=layers, B=B, L_min=_log_int(rng, 1, hi) - 1, L_max=hi, grow=_log_int(rng, 1, 200), Hkv=Hkv,
                        page=page, lens=lens)
            case["spare"] = 4 + 2 * B * (2 + case["grow"] // page)
            if layers * Hkv * page * (case["spare"] + B * (hi // page + 1)) <= 32 * 8 * 64 * 1700:
                return case
            layers = max(1, layers // 2)
    while True:
        n, hi = rng.randint(1, 64), _log_int(rng, 1, 2000)
        if layers * B * Hkv * (hi + 70) <= 32 * 64 * 8 * 576:
            return dict(op=op, layers=layers, B=B, n=n, depth=min(n - 1, rng.randint(0, 10)), L_min=_log_int(rng, 1, hi) - 1, L_max=hi,
                        Hkv=Hkv, page=page, lens=lens)
        layers = max(1, layers // 2)


def _tree(rng, n):
    """Parents of n nodes: one of the nodes before, near ones more often."""
    return [-1] + [max(0, i - 1 - int(rng.expovariate(1 / 4))) for i in range(1, n)]


def _counts(case):
    """The case's lengths: dict of lists of B numbers, from the case alone."""
    rng = random.Random(case["lens"])
    B, op = case["B"], case["op"]
    if op == "rope":
        new = [_log_int(rng, case["q_min"], case["q_max"]) for _ in range(B)]
        if B > 1:
            new[0], new[-1] = case["q_max"], case["q_min"]
        pos = [rng.randint(0, case["pos_max"]) for _ in new]
        parent = [_tree(rng, case["n"]) for _ in new] if case["n"] else None
        return {"new": new, "pos": pos, "parent": parent}
    lo, hi = case["L_min"], case["L_max"]
    L = [min(hi, _log_int(rng, lo + 1, hi + 1) - 1) for _ in range(B)]
    L[0] = hi
    if lo == hi:
        L = [hi] * B
    if op == "attn":
        return {"L": L, "parent": [_tree(rng, case["n"]) for _ in range(B)]}
    if op == "assign":
        if case["kind"] == "grow":
            src = list(range(B))
        elif case["kind"] == "fork":
            src, L = [0] * B, [L[0]] + [0] * (B - 1)
        else:
            src = [rng.randrange(-1, B) if rng.random() < 0.7 else b for b in range(B)]
        return {"L": L, "src": src, "grow": [rng.randint((case["grow"] + 1) // 2, case["grow"]) for _ in range(B)]}
    acc = [rng.randint(0, case["depth"]) for _ in range(B)]
    path = [[0] + sorted(rng.sample(range(1, case["n"]), a)) + [-1] * (case["depth"] - a) for a in acc]
    return {"L": L, "acc": acc, "path": path}


def _depths(parent):
    d = []
    for p in parent:
        d.append(0 if p < 0 else d[p] + 1)
    return d


def _copies(case, c):
    """Rows that the assignment copies (of one layer and kv head, of K)."""
    rows, kept = 0, set()
    for b in sorted(range(case["B"]), key=lambda b: c["src"][b] != b):       # a slot that continues itself comes first
        s = c["src"][b]
        if s >= 0 and s in kept:
            rows += c["L"][s] % case["page"]
        kept.add(s)
    return rows


def work(case):
    c = _counts(case)
    op, Hkv = case["op"], case["Hkv"]
    if op == "rope":
        T, Hq = sum(c["new"]), case["Hq"]
        outs = {"pages": Hq + 2 * Hkv, "packed": Hq + Hkv, "both": Hq + 3 * Hkv}[case["dest"]]
        ins = Hq + (Hkv if case["dest"] == "packed" else 2 * Hkv)
        return {"bytes": 2 * D * T * (ins + outs), "flops": 8 * D * T * (Hq + Hkv)}
    if op == "attn":
        Hq, B, n = case["Hq"], case["B"], case["n"]
        seen = sum(n * L + sum(_depths(p)) + n for L, p in zip(c["L"], c["parent"]))
        return {"bytes": 4 * D * (sum(L + n for L in c["L"]) * Hkv + B * n * Hq), "flops": 4 * D * Hq * seen}
    if op == "assign":
        page = case["page"]
        pages = sum(-(-((c["L"][s] if s >= 0 else 0) + g) // page) for s, g in zip(c["src"], c["grow"]))
        return {"bytes": 8 * pages + 20 * case["B"] + case["layers"] * 2 * Hkv * _copies(case, c) * 2 * 2 * D, "flops": 0}
    moved = sum(sum(p != t for t, p in enumerate(path[:a + 1])) for path, a in zip(c["path"], c["acc"]))
    return {"bytes": case["layers"] * 2 * Hkv * moved * 2 * 2 * D + 4 * case["B"] * (case["depth"] + 4), "flops": 0}


# ---------------------------------------------------------------- inputs
def _rows(shape, gen, gain=0.3):
    """bf16 rows as projections leave them: normal, with channels of different strength."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)
    return x.mul_(torch.exp(gain * torch.randn(shape[-1], generator=gen, device="cuda")).bfloat16())


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _table(rows, page, width, ids, first=None):
    """[B, width] page numbers, taken from ids, for rows first[b] .. rows[b] - 1 of each sequence; -1 elsewhere."""
    out = []
    for b, r in enumerate(rows):
        t0, t1 = (first[b] // page if first else 0), -(-r // page)
        out.append([-1] * t0 + [next(ids) for _ in range(t0, t1)] + [-1] * (width - t1))
    return out


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    c = _counts(case)
    op, B, Hkv, page = case["op"], case["B"], case["Hkv"], case["page"]
    order = random.Random(seed)
    s = dict(case, scale=D ** -0.5)

    def shuffled(n):
        ids = list(range(n))
        order.shuffle(ids)
        return iter(ids)

    if op == "rope":
        T, Hq, rot = sum(c["new"]), case["Hq"], case["rot"]
        qkv = _rows((T, (Hq + 2 * Hkv) * D), gen)                 # one projection's output, cut in three
        q, k, v = qkv.split([Hq * D, Hkv * D, Hkv * D], 1)
        s.update(q=q.unflatten(1, (Hq, D)), k=k.unflatten(1, (Hkv, D)), v=v.unflatten(1, (Hkv, D)))
        if case["norm"]:
            s.update(q_weight=_rows((D,), gen, 0.0).add_(2.0), k_weight=_rows((D,), gen, 0.0).add_(2.0))
        else:
            s.update(q_weight=None, k_weight=None)
        base = 10000.0 if seed % 2 else 500000.0
        s["inv_freq"] = (base ** -(torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)).float()
        s["pos"] = _ints(c["pos"])
        s["q_out"] = torch.empty((T, Hq, D), dtype=torch.bfloat16, device="cuda")
        s["k_out"] = None if case["dest"] == "pages" else torch.empty((T, Hkv, D), dtype=torch.bfloat16, device="cuda")
        if case["n"]:
            s["parent"], s["cu"] = _ints(c["parent"]), None
        else:
            cu = [0]
            for m in c["new"]:
                cu.append(cu[-1] + m)
            s["parent"], s["cu"] = None, _ints(cu)
        s["k_pages"] = s["v_pages"] = s["page_table"] = None
        if case["dest"] != "packed":
            end = [p + m for p, m in zip(c["pos"], c["new"])]
            N = sum(-(-e // page) - p // page for e, p in zip(end, c["pos"])) + 3
            s["page_table"] = _ints(_table(end, page, -(-max(end) // page), shuffled(N), c["pos"]))
            s["k_pages"], s["v_pages"] = _rows((N, Hkv, page, D), gen), _rows((N, Hkv, page, D), gen)
    elif op == "attn":
        n, rows = case["n"], [L + case["n"] for L in c["L"]]
        N = sum(-(-r // page) for r in rows) + 3
        s.update(q=_rows((B, n, case["Hq"], D), gen), kv_len=_ints(c["L"]), parent=_ints(c["parent"]))
        s["page_table"] = _ints(_table(rows, page, -(-max(rows) // page), shuffled(N)))
        s["k_pages"], s["v_pages"] = _rows((N, Hkv, page, D), gen), _rows((N, Hkv, page, D), gen)
    elif op == "assign":
        held = [-(-L // page) for L in c["L"]]
        N = sum(held) + case["spare"]
        table = _table(c["L"], page, -(-(max(c["L"]) + case["grow"]) // page), shuffled(N))
        refs = [0] * N
        for row in table:
            for p in row:
                if p >= 0:
                    refs[p] += 1
        s.update(page_table=_ints(table), held=_ints(held), refs=_ints(refs), kv_len=_ints(c["L"]), grow=_ints(c["grow"]),
                 src=None if case["kind"] == "grow" else _ints(c["src"]))
        s["k_pages"], s["v_pages"] = (_rows((case["layers"], N, Hkv, page, D), gen) for _ in range(2))
    else:
        n, rows = case["n"], [L + case["n"] for L in c["L"]]
        N = sum(-(-r // page) for r in rows) + 3
        s.update(kv_len=_ints(c["L"]), new_len=torch.empty(B, dtype=torch.int32, device="cuda"), path=_ints(c["path"]), acc=_ints(c["acc"]))
        s["page_table"] = _ints(_table(rows, page, -(-max(rows) // page), shuffled(N)))
        s["k_pages"], s["v_pages"] = (_rows((case["layers"], N, Hkv, page, D), gen) for _ in range(2))
    return s


# ---------------------------------------------------------------- plain forms
def _sees(parent):
    """[B, n, n]: node j is i or above it, by squaring the one-step relation."""
    n = parent.shape[1]
    par = parent.long()
    step = torch.eye(n, device="cuda").expand(len(par), n, n) + torch.nn.functional.one_hot(par.clamp(min=0), n) * (par >= 0)[..., None]
    for _ in range(6):
        step = (step @ step).clamp(max=1.0)
    return step > 0


def _plain_rope(s):
    T, rot = s["q"].shape[0], s["rot"]
    t = torch.arange(T, device="cuda")
    if s["n"]:
        b, row = t // s["n"], t % s["n"]
        ahead = _sees(s["parent"]).sum(-1).view(-1) - 1                              # a node's depth
    else:
        cu = s["cu"].long()
        b = torch.searchsorted(cu[1:], t, right=True)
        ahead = row = t - cu[b]
    pos = s["pos"].long()[b]
    angle = (pos + ahead).double()[:, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turned(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()
        if s["pairs"] == "halves":
            x0, x1, rest = x.split([rot // 2, rot // 2, D - rot], -1)
            return torch.cat([x0 * cos - x1 * sin, x1 * cos + x0 * sin, rest], -1).bfloat16()
        x0, x1 = x[..., 0:rot:2], x[..., 1:rot:2]
        return torch.cat([torch.stack([x0 * cos - x1 * sin, x1 * cos + x0 * sin], -1).flatten(-2), x[..., rot:]], -1).bfloat16()

    s["q_out"].copy_(turned(s["q"], s["q_weight"]))
    k = turned(s["k"], s["k_weight"])
    if s["k_out"] is not None:
        s["k_out"].copy_(k)
    if s["page_table"] is not None:
        at = pos + row
        p = s["page_table"].long()[b, at // s["page"]]
        s["k_pages"][p, :, at % s["page"]] = k
        s["v_pages"][p, :, at % s["page"]] = s["v"]
    return [x for x in (s["q_out"], s["k_out"], s["k_pages"], s["v_pages"]) if x is not None]


def _plain_attn(s):
    B, n, Hq, Hkv, page = s["B"], s["n"], s["Hq"], s["Hkv"], s["page"]
    G, width = Hq // Hkv, s["page_table"].shape[1]
    K = width * page
    sees_tree = _sees(s["parent"])
    out = torch.empty_like(s["q"])
    step = max(1, (1 << 29) // (Hkv * max(K * D, G * n * K)))
    for b0 in range(0, B, step):                                                     # as many sequences as fit
        bs = slice(b0, min(B, b0 + step))
        m = bs.stop - b0
        ids = s["page_table"][bs].long().clamp(min=0)
        L = s["kv_len"][bs].long()[:, None, None]
        at = torch.arange(K, device="cuda") - L                                      # [m, 1, K], from 0 on: the tree's rows
        sees = (at < 0) | (sees_tree[bs].gather(2, at.clamp(0, n - 1).expand(m, n, K)) & (at < n))
        rows = lambda x: x[ids].float().transpose(1, 2).reshape(m, Hkv, K, D)  # noqa: E731
        q = s["q"][bs].float().view(m, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(m, Hkv, G * n, D)
        x = (q @ rows(s["k_pages"]).transpose(-1, -2)).mul_(s["scale"]).view(m, Hkv, G, n, K)
        x.masked_fill_(~sees[:, None, None], -math.inf)
        x.sub_(x.amax(-1, keepdim=True)).exp_()
        l = x.sum(-1, keepdim=True)
        o = (x.view(m, Hkv, G * n, K) @ rows(s["v_pages"])).view(m, Hkv, G, n, D) / l
        out[bs] = o.permute(0, 3, 1, 2, 4).reshape(m, n, Hq, D).bfloat16()
    return out


def _plain_assign(s):
    B, page = s["B"], s["page"]
    table, refs, L, N = s["page_table"].long(), s["refs"], s["kv_len"].long(), s["refs"].shape[0]
    me, col = torch.arange(B, device="cuda"), torch.arange(s["page_table"].shape[1], device="cuda")
    src = me if s["src"] is None else s["src"].long()
    of = src.clamp(min=0)
    length = torch.where(src < 0, 0, L[of])
    full, part = length // page, length % page
    need = (length + s["grow"].long() + page - 1) // page
    theirs = table[of]
    last = theirs.gather(1, full.clamp(max=len(col) - 1)[:, None])[:, 0]            # the partly filled page
    # of the slots that continue s one goes on in that page: s itself, else the first; none if it is shared
    key = torch.where(src == me, -1, me)
    first = torch.full((B,), B, device="cuda").scatter_reduce(0, of, torch.where(src < 0, B, key), "amin")
    stays = (key == first[of]) & (refs[last.clamp(min=0)] <= 1)
    copy = (src >= 0) & (part > 0) & ~stays
    # a slot that continues itself keeps what it holds behind its rows, unless it is shared
    more = (src == me)[:, None] & (col >= full[:, None]) & (col < s["held"][:, None]) & (refs[theirs.clamp(min=0)] <= 1)
    there = (src >= 0)[:, None] & ((col < full[:, None]) | ((col == full[:, None]) & ((part > 0) & ~copy)[:, None]) | more)
    fresh = (col < need[:, None]) & ~there
    free = torch.argsort((refs != 0).int(), stable=True)                            # free pages first, by number
    rank = (fresh.view(-1).cumsum(0) - 1).view_as(fresh).clamp(0, N - 1)
    now = torch.where(fresh, free[rank], theirs)
    now = torch.where(col < need[:, None], now, torch.where(col < s["held"][:, None], -1, table))
    # the copies; a slot that copies nothing repeats one that does (page 0 onto itself, if none does)
    i = copy.int().argmax()
    one = torch.where(copy, me, i)
    to = now.gather(1, full.clamp(max=len(col) - 1)[:, None])[:, 0]
    frm_, to_, rows = (torch.where(copy.any(), x[one], 0) for x in (last, to, part))
    keep = (torch.arange(page, device="cuda") < rows[:, None])[:, None, :, None]
    for pages in (s["k_pages"], s["v_pages"]):
        for layer in pages:
            layer[to_] = torch.where(keep, layer[frm_], layer[to_])
    hit = (col < need[:, None]).int().view(-1)
    s["refs"].copy_(torch.zeros_like(refs).index_add_(0, now.clamp(min=0).view(-1), hit))
    s["page_table"].copy_(now)
    s["held"].copy_(need)
    s["kv_len"].copy_(length)
    return s["page_table"], s["held"], s["refs"], s["kv_len"], s["k_pages"], s["v_pages"]


def _plain_commit(s):
    page, L, acc = s["page"], s["kv_len"].long(), s["acc"].long()
    # a place behind the accepted path repeats the path's first row, which stays where it is
    t = torch.arange(s["depth"] + 1, device="cuda")
    t = torch.where(t <= acc[:, None], t, 0)
    seq = torch.arange(s["B"], device="cuda")[:, None]
    table = s["page_table"].long()
    place = lambda row: (table[seq, row // page].view(-1), (row % page).view(-1))  # noqa: E731
    p0, r0 = place(L[:, None] + s["path"].long().gather(1, t))
    p1, r1 = place(L[:, None] + t)
    for pages in (s["k_pages"], s["v_pages"]):
        for layer in pages:
            layer[p1, :, r1] = layer[p0, :, r0]
    torch.add(s["kv_len"], s["acc"] + 1, out=s["new_len"])
    return s["k_pages"], s["v_pages"], s["new_len"]


# ---------------------------------------------------------------- the library's calls
def _own(s):
    import eagle_tree_speculative_gb300 as E
    if s["op"] == "rope":
        E.eagle_qkv_rope(s["q"], s["k"], s["v"], s["inv_freq"], s["pos"], cu=s["cu"], parent=s["parent"], q_weight=s["q_weight"],
                         k_weight=s["k_weight"], eps=1e-6, interleaved=s["pairs"] != "halves", k_pages=s["k_pages"], v_pages=s["v_pages"],
                         page_table=s["page_table"], q_out=s["q_out"], k_out=s["k_out"])
        return [x for x in (s["q_out"], s["k_out"], s["k_pages"], s["v_pages"]) if x is not None]
    if s["op"] == "attn":
        return E.eagle_tree_attn_paged(s["q"], s["k_pages"], s["v_pages"], s["page_table"], s["kv_len"], s["parent"], scale=s["scale"])
    if s["op"] == "assign":
        E.eagle_pages_assign(s["k_pages"], s["v_pages"], s["page_table"], s["held"], s["refs"], s["kv_len"], s["grow"], src=s["src"])
        return s["page_table"], s["held"], s["refs"], s["kv_len"], s["k_pages"], s["v_pages"]
    E.eagle_pages_commit(s["k_pages"], s["v_pages"], s["page_table"], s["kv_len"], s["path"], s["acc"], s["depth"], kv_len_out=s["new_len"])
    return s["k_pages"], s["v_pages"], s["new_len"]


def run(state):
    if own:
        return _own(state)
    return {"rope": _plain_rope, "attn": _plain_attn, "assign": _plain_assign, "commit": _plain_commit}[state["op"]](state)


# ---------------------------------------------------------------- 64 bits, from the definitions
def _exact_rope(s, c):
    rot, start = s["rot"], 0
    outs = {"q": [], "k": []}
    kp, vp = (None if x is None else x.double() for x in (s["k_pages"], s["v_pages"]))
    table = None if s["page_table"] is None else s["page_table"].tolist()
    for b, m in enumerate(c["new"]):
        ahead = _depths(c["parent"][b]) if c["parent"] else range(m)
        angle = torch.tensor([c["pos"][b] + a for a in ahead], dtype=torch.float64, device="cuda")[:, None] * s["inv_freq"].double()
        turn = torch.polar(torch.ones_like(angle), angle)[:, None]                  # e^(i angle)
        for name in ("q", "k"):
            x = s[name][start:start + m].double()
            if s[name + "_weight"] is not None:
                x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + 1e-6) * s[name + "_weight"].double()
            head = x[..., :rot]
            z = head.unflatten(-1, (2, rot // 2)).transpose(-1, -2) if s["pairs"] == "halves" else head.unflatten(-1, (rot // 2, 2))
            z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn)
            z = z.transpose(-1, -2) if s["pairs"] == "halves" else z
            outs[name].append(torch.cat([z.flatten(-2), x[..., rot:]], -1))
        if table:
            r = 0
            while r < m:                                                            # page by page
                at = c["pos"][b] + r
                p, i = table[b][at // s["page"]], at % s["page"]
                k = min(m - r, s["page"] - i)
                kp[p, :, i:i + k] = outs["k"][b][r:r + k].transpose(0, 1)
                vp[p, :, i:i + k] = s["v"][start + r:start + r + k].double().transpose(0, 1)
                r += k
        start += m
    k_out = torch.cat(outs["k"]) if s["k_out"] is not None else None
    return [x for x in (torch.cat(outs["q"]), k_out, kp, vp) if x is not None]


def _exact_attn(s, c):
    out = torch.empty((s["B"], s["n"], s["Hq"], D), dtype=torch.float64, device="cuda")
    G, n, table = s["Hq"] // s["Hkv"], s["n"], s["page_table"].tolist()
    for b, (L, parent) in enumerate(zip(c["L"], c["parent"])):
        sees = torch.zeros((n, L + n), dtype=torch.bool)
        sees[:, :L] = True
        for i in range(n):
            j = i
            while j >= 0:
                sees[i, L + j] = True
                j = parent[j]
        sees = sees.cuda()
        ids = [p for p in table[b] if p >= 0]
        for h in range(s["Hkv"]):
            k, v = (x[ids, h].reshape(-1, D)[:L + n].double() for x in (s["k_pages"], s["v_pages"]))
            q = s["q"][b, :, h * G:(h + 1) * G].double().transpose(0, 1)
            w = torch.softmax(torch.where(sees, q @ k.T * s["scale"], -math.inf), -1)
            out[b, :, h * G:(h + 1) * G] = (w @ v).transpose(0, 1)
    return out


def _exact_assign(s, c):
    """Slot by slot, page by page."""
    B, page, old = s["B"], s["page"], s["page_table"].tolist()
    refs, held = s["refs"].tolist(), s["held"].tolist()
    free = sorted(p for p, r in enumerate(refs) if r == 0)
    pages = [x.clone() for x in (s["k_pages"], s["v_pages"])]
    table, lengths, moves = [], [], []
    for b in range(B):
        t = c["src"][b]
        L = c["L"][t] if t >= 0 else 0
        need = -(-(L + c["grow"][b]) // page)
        row = old[t][:L // page] if t >= 0 else []
        for x in range(L // page, need):
            alone = t >= 0 and x < held[t] and refs[old[t][x]] == 1
            if x == L // page and L % page:                       # the page that the rows end in
                heirs = [y for y in range(B) if c["src"][y] == t]
                stays = alone and b == (t if t in heirs else heirs[0])
                if not stays:
                    moves.append((old[t][x], free[0], L % page))
            else:
                stays = alone and t == b
            row = row + [old[t][x] if stays else free.pop(0)]
        table.append(row + [-1 if x < held[b] else old[b][x] for x in range(need, len(old[b]))])
        lengths.append(L)
    for a, z, r in moves:
        for x in pages:
            x[:, z, :, :r] = x[:, a, :, :r]
    count = [0] * len(refs)
    need = [-(-(L + g) // page) for L, g in zip(lengths, c["grow"])]
    for row, m in zip(table, need):
        for p in row[:m]:
            count[p] += 1
    return _ints(table), _ints(need), _ints(count), _ints(lengths), *(x.double() for x in pages)


def _exact_commit(s, c):
    page, table = s["page"], s["page_table"].tolist()
    new = [x.clone() for x in (s["k_pages"], s["v_pages"])]
    for b, (L, a, path) in enumerate(zip(c["L"], c["acc"], c["path"])):
        for t in range(a + 1):
            (p0, r0), (p1, r1) = ((table[b][r // page], r % page) for r in (L + path[t], L + t))
            for x, was in zip(new, (s["k_pages"], s["v_pages"])):
                x[:, p1, :, r1] = was[:, p0, :, r0]
    return *(x.double() for x in new), _ints([L + a + 1 for L, a in zip(c["L"], c["acc"])])


def exact(case, seed):
    c = _counts(case)
    s = prepare(case, seed)
    return {"rope": _exact_rope, "attn": _exact_attn, "assign": _exact_assign, "commit": _exact_commit}[case["op"]](s, c)
