"""The prompt attention and the 8-bit cache, case by case: inputs, plain forms, 64-bit values.

Four operators that a serving loop runs around one verify step:

  prompt   causal attention of packed prompts (queries may stand behind a prefix)
  append   prompt rows quantised into the 8-bit K/V cache of one layer
  tree     attention of a draft tree (one node: ordinary decoding) over that cache
  commit   the accepted path's rows of every layer quantised into the cache

The cache holds e4m3 codes [.., B, Hkv, Lmax, d] and one power-of-two scale per 32 rows and
kv head; a row is code * scale.  `run` gives the plain form, in torch operations and 32 bits,
or with `own` the library's calls on the same state.
"""
import math
import random

import torch

own = False

D = 128          # head dimension
BLOCK = 32       # cache rows that share a scale
E_MIN = -64      # the smallest scale is 2^-64


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one short prompt: the latency of the call
        dict(name="prompt_one_short", op="prompt", B=1, q_min=37, q_max=37, prefix=0, Hq=32, Hkv=8, lens=1),
        # a server's mixed batch of prompts, lengths from a few tokens on
        dict(name="prompt_ragged", op="prompt", B=16, q_min=5, q_max=4096, prefix=0, Hq=32, Hkv=8, lens=2),
        # chunks of long prompts behind what has been computed already, eight heads a group
        dict(name="prompt_chunks", op="prompt", B=3, q_min=500, q_max=1100, prefix=7000, Hq=64, Hkv=8, lens=3),
        # one long document
        dict(name="prompt_long", op="prompt", B=1, q_min=16384, q_max=16384, prefix=0, Hq=32, Hkv=8, lens=4),
        # a few tokens each, into partly filled blocks
        dict(name="append_few", op="append", B=8, q_min=1, q_max=9, pos_max=1000, Lmax=1024, Hkv=8, lens=5),
        # the prompts of a full batch
        dict(name="append_prompts", op="append", B=64, q_min=16, q_max=2048, pos_max=100, Lmax=2200, Hkv=8, lens=6),
        # plain decoding, one sequence, every head its own keys
        dict(name="decode_one", op="tree", B=1, n=1, L_min=1777, L_max=1777, Lmax=2048, Hq=40, Hkv=40, lens=7),
        # plain decoding of a ragged batch with long sequences in it
        dict(name="decode_ragged", op="tree", B=48, n=1, L_min=100, L_max=30000, Lmax=32768, Hq=64, Hkv=8, lens=8),
        # the verify step's own shape: 60-node trees at 4096 committed tokens
        dict(name="tree_b64", op="tree", B=64, n=60, L_min=4096, L_max=4096, Lmax=4160, Hq=32, Hkv=8, lens=9),
        # trees over sequences of very different lengths
        dict(name="tree_ragged", op="tree", B=16, n=48, L_min=33, L_max=16000, Lmax=16384, Hq=64, Hkv=8, lens=10),
        # one step of one sequence, all layers
        dict(name="commit_one", op="commit", layers=32, B=1, n=60, depth=6, L_min=2048, L_max=2048, Lmax=2112, Hkv=8, lens=11),
        # one step of a full batch, all layers
        dict(name="commit_b64", op="commit", layers=32, B=64, n=60, depth=8, L_min=20, L_max=500, Lmax=576, Hkv=8, lens=12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    return rng.choice([(32, 8), (64, 8), (40, 40), (32, 32), (8, 2), (28, 4), (40, 8), (6, 2), (16, 1), (1, 1)])


def draw(rng):
    op = rng.choice(["prompt", "append", "tree", "tree", "commit"])
    lens = rng.randrange(1 << 20)
    Hq, Hkv = _heads(rng)
    if op == "prompt":
        while True:
            B, hi = _log_int(rng, 1, 24), _log_int(rng, 1, 16384)
            lo, prefix = _log_int(rng, 1, hi), rng.choice([0, 0, _log_int(rng, 1, 8192)])
            case = dict(op=op, B=B, q_min=lo, q_max=hi, prefix=prefix, Hq=Hq, Hkv=Hkv, lens=lens)
            if B * Hq * hi * (hi + prefix) <= 32 * 16384 * 8192 and work(case)["flops"] > 1e6:
                return case
    if op == "append":
        while True:
            B, hi, pos = _log_int(rng, 1, 64), _log_int(rng, 1, 4096), rng.choice([0, _log_int(rng, 1, 4096)])
            if B * hi * Hkv <= 64 * 2048 * 8 and B * (hi + pos) * Hkv <= 64 * 2200 * 8:
                return dict(op=op, B=B, q_min=_log_int(rng, 1, hi), q_max=hi, pos_max=pos, Lmax=hi + pos + rng.randrange(70),
                            Hkv=Hkv, lens=lens)
    if op == "tree":
        while True:
            B, n, hi = _log_int(rng, 1, 64), rng.choice([1, 2, _log_int(rng, 3, 64), rng.randint(3, 64)]), _log_int(rng, 1, 32000)
            if B * Hkv * hi <= 64 * 8 * 4096 and B * Hq * n * hi <= 64 * 32 * 60 * 4096:
                return dict(op=op, B=B, n=n, L_min=_log_int(rng, 1, hi) - 1, L_max=hi, Lmax=hi + rng.randint(0, 200), Hq=Hq, Hkv=Hkv,
                            lens=lens)
    while True:
        layers, B, n, hi = _log_int(rng, 1, 48), _log_int(rng, 1, 64), rng.randint(1, 64), _log_int(rng, 1, 2000)
        if layers * B * Hkv * (hi + 70) <= 32 * 64 * 8 * 576:
            return dict(op=op, layers=layers, B=B, n=n, depth=min(n - 1, rng.randint(0, 10)), L_min=_log_int(rng, 1, hi) - 1, L_max=hi,
                        Lmax=hi + 66, Hkv=Hkv, lens=lens)


def _counts(case):
    """The case's lengths: dict of lists of B numbers, from the case alone."""
    rng = random.Random(case["lens"])
    B, op = case["B"], case["op"]
    if op in ("prompt", "append"):
        new = [_log_int(rng, case["q_min"], case["q_max"]) for _ in range(B)]
        if B > 1:
            new[0], new[-1] = case["q_max"], case["q_min"]
        if op == "prompt":
            return {"q": new, "k": [m + rng.randint((case["prefix"] + 1) // 2, case["prefix"]) for m in new]}
        return {"new": new, "pos": [rng.randint(0, case["pos_max"]) for _ in new]}
    L = [min(case["L_max"], _log_int(rng, case["L_min"] + 1, case["L_max"] + 1) - 1) for _ in range(B)]
    if B > 1:
        L[0] = case["L_max"]
    if case["L_min"] == case["L_max"]:
        L = [case["L_max"]] * B
    if op == "tree":
        # parent of node i: one of the nodes before it, near ones more often
        parent = [[-1] + [max(0, i - 1 - int(rng.expovariate(1 / 4))) for i in range(1, case["n"])] for _ in range(B)]
        return {"L": L, "parent": parent}
    acc = [rng.randint(0, case["depth"]) for _ in range(B)]
    path = [[0] + sorted(rng.sample(range(1, case["n"]), a)) + [-1] * (case["depth"] - a) for a in acc]
    return {"L": L, "acc": acc, "path": path}


def _depths(parent):
    d = []
    for p in parent:
        d.append(0 if p < 0 else d[p] + 1)
    return d


def work(case):
    c = _counts(case)
    op, Hkv = case["op"], case["Hkv"]
    blocks = lambda pos, m: (pos + m + BLOCK - 1) // BLOCK - pos // BLOCK  # noqa: E731  scales of rows pos .. pos + m - 1
    if op == "prompt":
        Hq, Tq, Tk = case["Hq"], sum(c["q"]), sum(c["k"])
        seen = sum(q * (k - q) + q * (q + 1) // 2 for q, k in zip(c["q"], c["k"]))
        return {"bytes": 2 * D * (2 * Tq * Hq + 2 * Tk * Hkv) + 4 * Tq * Hq, "flops": 4 * D * Hq * seen}
    if op == "append":
        rows = sum(c["new"])
        return {"bytes": 2 * Hkv * (rows * D * 3 + 4 * sum(blocks(p, m) for p, m in zip(c["pos"], c["new"]))), "flops": 0}
    if op == "tree":
        Hq, B, n = case["Hq"], case["B"], case["n"]
        seen = sum(n * L + sum(_depths(p)) + n for L, p in zip(c["L"], c["parent"]))
        cache = sum(2 * Hkv * (L * D + 4 * blocks(0, L)) for L in c["L"])
        return {"bytes": cache + 2 * B * n * D * (2 * Hq + 2 * Hkv), "flops": 4 * D * Hq * seen}
    rows = sum(a + 1 for a in c["acc"])
    return {"bytes": case["layers"] * 2 * Hkv * (rows * D * 3 + 4 * sum(blocks(L, a + 1) for L, a in zip(c["L"], c["acc"]))), "flops": 0}


# ---------------------------------------------------------------- inputs
def _rows(shape, gen, gain=0.3):
    """bf16 rows as projections leave them: normal, with channels of different strength."""
    x = torch.randn(shape, generator=gen, device="cuda")
    return (x * torch.exp(gain * torch.randn(shape[-1], generator=gen, device="cuda"))).bfloat16()


def _scale_of(amax):
    """2^e with the least e >= E_MIN for which amax <= 448 * 2^e."""
    m, e = torch.frexp(amax)                       # amax = m 2^e, 0.5 <= m < 1;  448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(amax > 0, e, E_MIN).clamp(min=E_MIN)
    return torch.ldexp(torch.ones_like(amax), e)


def _cache(shape, gen, strength=1.0):
    """Codes and scales of a cache full of rows [.., Lmax, D]."""
    lead, Lmax = shape[:-2], shape[-2]
    nb = (Lmax + BLOCK - 1) // BLOCK
    gain = torch.exp(0.3 * torch.randn(D, generator=gen, device="cuda")) * strength
    codes = torch.empty((*lead, nb * BLOCK, D), dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty((*lead, nb), device="cuda")
    flat_c, flat_s = codes.view(-1, nb, BLOCK, D), scales.view(-1, nb)
    step = max(1, (1 << 28) // (nb * BLOCK * D))
    for at in range(0, flat_c.shape[0], step):
        x = torch.randn((min(step, flat_c.shape[0] - at), nb, BLOCK, D), generator=gen, device="cuda") * gain
        s = _scale_of(x.abs().amax((-2, -1)))
        flat_s[at:at + step] = s
        flat_c[at:at + step] = (x / s[..., None, None]).to(torch.float8_e4m3fn)
    return codes[..., :Lmax, :].contiguous(), scales


def _starts(m):
    out = [0]
    for v in m:
        out.append(out[-1] + v)
    return torch.tensor(out, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    c = _counts(case)
    op, B, Hkv = case["op"], case["B"], case["Hkv"]
    s = dict(case, scale=D ** -0.5)
    if op == "prompt":
        Tq, Tk = sum(c["q"]), sum(c["k"])
        s.update(q=_rows((Tq, case["Hq"], D), gen), k=_rows((Tk, Hkv, D), gen), v=_rows((Tk, Hkv, D), gen),
                 cu_q=_starts(c["q"]), cu_k=_starts(c["k"]), max_q=max(c["q"]), max_k=max(c["k"]))
    elif op == "append":
        T, Lmax = sum(c["new"]), case["Lmax"]
        s.update(k=_rows((T, Hkv, D), gen), v=_rows((T, Hkv, D), gen), cu=_starts(c["new"]), pos=ints(c["pos"]))
        s["k8"], s["k_scale"] = _cache((B, Hkv, Lmax, D), gen, 0.8)
        s["v8"], s["v_scale"] = _cache((B, Hkv, Lmax, D), gen, 0.8)
    elif op == "tree":
        n = case["n"]
        s.update(q=_rows((B, n, case["Hq"], D), gen), k_tree=_rows((B, n, Hkv, D), gen), v_tree=_rows((B, n, Hkv, D), gen),
                 kv_len=ints(c["L"]), parent=ints(c["parent"]))
        s["k8"], s["k_scale"] = _cache((B, Hkv, case["Lmax"], D), gen)
        s["v8"], s["v_scale"] = _cache((B, Hkv, case["Lmax"], D), gen)
    else:
        layers, n = case["layers"], case["n"]
        s.update(k_tree=_rows((layers, B, n, Hkv, D), gen), v_tree=_rows((layers, B, n, Hkv, D), gen),
                 kv_len=ints(c["L"]), new_len=torch.empty(B, dtype=torch.int32, device="cuda"), path=ints(c["path"]), acc=ints(c["acc"]))
        s["k8"], s["k_scale"] = _cache((layers, B, Hkv, case["Lmax"], D), gen, 0.8)
        s["v8"], s["v_scale"] = _cache((layers, B, Hkv, case["Lmax"], D), gen, 0.8)
    return s


# ---------------------------------------------------------------- plain forms
def _plain_prompt(s):
    """Every sequence padded to the longest, scores as one batched product."""
    B, Hq, Hkv, nq, nk = s["B"], s["Hq"], s["Hkv"], s["max_q"], s["max_k"]
    G = Hq // Hkv
    cq, ck = s["cu_q"].long(), s["cu_k"].long()
    lq, lk = cq[1:] - cq[:-1], ck[1:] - ck[:-1]
    iq = torch.arange(nq, device="cuda")
    ik = torch.arange(nk, device="cuda")
    at_q = (cq[:-1, None] + iq).clamp(max=s["q"].shape[0] - 1)
    at_k = (ck[:-1, None] + ik).clamp(max=s["k"].shape[0] - 1)
    q = s["q"].float()[at_q].view(B, nq, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * nq, D)
    k = s["k"].float()[at_k].permute(0, 2, 3, 1)
    v = s["v"].float()[at_k].permute(0, 2, 1, 3)
    x = (q @ k).mul_(s["scale"]).view(B, Hkv, G, nq, nk)
    sees = (ik < lk[:, None])[:, None, :] & (ik <= (iq + (lk - lq)[:, None])[:, :, None])       # [B, nq, nk]
    x.masked_fill_(~sees[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    base = torch.where(m > -math.inf, m, 0.0)
    x.sub_(base).exp_()
    l = x.sum(-1, keepdim=True)
    o = (x.view(B, Hkv, G * nq, nk) @ v).view(B, Hkv, G, nq, D) / torch.where(l > 0, l, 1.0)
    lse = (l.log() + base)[..., 0]
    t = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(cq[1:], t, right=True)
    i = t - cq[b]
    return o.permute(0, 3, 1, 2, 4)[b, i].reshape(-1, Hq, D).bfloat16(), lse.permute(0, 3, 1, 2)[b, i].reshape(-1, Hq)


def _plain_write(x, b, p, pos, codes, scales):
    """Rows x [R, N, Hkv, D] (R layers; row n goes to sequence b[n], cache row p[n]) into codes [R, B, Hkv, Lmax, D]
    and scales [R, B, Hkv, NB]; pos [B]: rows that the sequences hold already."""
    R, B, Hkv, Lmax = codes.shape[:4]
    nb = scales.shape[-1]
    x = x.float()
    at = b * nb + p // BLOCK
    need = torch.zeros((R, B * nb, Hkv), device="cuda")
    need.scatter_reduce_(1, at[None, :, None].expand(R, -1, Hkv), x.abs().amax(-1), "amax")
    need = _scale_of(need).view(R, B, nb, Hkv).permute(0, 1, 3, 2)                             # [R, B, Hkv, NB]
    hit = torch.zeros(B * nb, dtype=torch.bool, device="cuda").index_fill_(0, at, True).view(B, nb)
    held = hit & (torch.arange(nb, device="cuda") * BLOCK < pos[:, None])                      # touched, and not empty before
    old = scales.clone()
    new = torch.where(hit[:, None], torch.where(held[:, None], torch.maximum(need, old), need), old)
    scales.copy_(new)
    # the rows that the block of row pos holds already, brought to its new scale
    first = (pos // BLOCK).clamp(max=nb - 1)
    rows = first[:, None] * BLOCK + torch.arange(BLOCK, device="cuda")                          # [B, BLOCK]
    at_row = rows.clamp(max=Lmax - 1)[:, None]
    take = first[:, None, None].expand(B, Hkv, 1)[None].expand(R, -1, -1, -1)
    by = (old.gather(-1, take) / new.gather(-1, take))[..., None]                               # [R, B, Hkv, 1, 1]
    seq = torch.arange(B, device="cuda")[:, None, None]
    head = torch.arange(Hkv, device="cuda")[None, :, None]
    bits = codes.view(torch.uint8)
    was = bits[:, seq, head, at_row]                                                            # [R, B, Hkv, BLOCK, D]
    now = (was.view(torch.float8_e4m3fn).float() * by).to(torch.float8_e4m3fn).view(torch.uint8)
    keep = (rows < pos[:, None]) & held.gather(1, first[:, None])
    bits[:, seq, head, at_row] = torch.where(keep[None, :, None, :, None], now, was)
    # the new rows
    b_, p_, h_ = b[:, None], p[:, None], torch.arange(Hkv, device="cuda")[None]
    s_ = new[:, b_, h_, p_ // BLOCK]                                                            # [R, N, Hkv]
    bits[:, b_, h_, p_] = (x / s_[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_append(s):
    cu, pos = s["cu"].long(), s["pos"].long()
    t = torch.arange(s["k"].shape[0], device="cuda")
    b = torch.searchsorted(cu[1:], t, right=True)
    p = pos[b] + t - cu[b]
    _plain_write(s["k"][None], b, p, pos, s["k8"][None], s["k_scale"][None])
    _plain_write(s["v"][None], b, p, pos, s["v8"][None], s["v_scale"][None])
    return s["k8"], s["v8"], s["k_scale"], s["v_scale"]


def _plain_tree(s):
    B, n, Hq, Hkv, Lmax = s["B"], s["n"], s["Hq"], s["Hkv"], s["Lmax"]
    G = Hq // Hkv
    # anc[b, i, j]: node j is i or above it, by squaring the one-step relation
    par = s["parent"].long()
    step = torch.eye(n, device="cuda").expand(B, n, n) + torch.nn.functional.one_hot(par.clamp(min=0), n) * (par >= 0)[..., None]
    for _ in range(6):
        step = (step @ step).clamp(max=1.0)
    blk = torch.arange(Lmax, device="cuda") // BLOCK
    rows = lambda c, sc: (c.float() * sc[..., blk, None])  # noqa: E731
    there = torch.arange(Lmax, device="cuda") < s["kv_len"][:, None]                            # [B, Lmax]
    q = s["q"].float().view(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
    kt, vt = s["k_tree"].float().permute(0, 2, 3, 1), s["v_tree"].float().permute(0, 2, 1, 3)
    x = torch.cat([q @ rows(s["k8"], s["k_scale"]).transpose(-1, -2), q @ kt], -1).mul_(s["scale"]).view(B, Hkv, G, n, Lmax + n)
    sees = torch.cat([there[:, None].expand(B, n, Lmax), step > 0], -1)
    x.masked_fill_(~sees[:, None, None], -math.inf)
    x.sub_(x.amax(-1, keepdim=True)).exp_()
    l = x.sum(-1, keepdim=True)
    x = x.view(B, Hkv, G * n, Lmax + n)
    v = torch.where(there[:, None, :, None], rows(s["v8"], s["v_scale"]), 0.0)
    o = (x[..., :Lmax] @ v + x[..., Lmax:] @ vt).view(B, Hkv, G, n, D) / l
    return o.permute(0, 3, 1, 2, 4).reshape(B, n, Hq, D).bfloat16()


def _plain_commit(s):
    B, n = s["B"], s["n"]
    pos, acc = s["kv_len"].long(), s["acc"].long()
    # a place behind the accepted path repeats the path's first row, at the first row's place
    t = torch.arange(s["depth"] + 1, device="cuda")
    t = torch.where(t <= acc[:, None], t, 0)
    seq = torch.arange(B, device="cuda")[:, None]
    src = (seq * n + s["path"].long().gather(1, t)).view(-1)
    p = (pos[:, None] + t).view(-1)
    b = seq.expand_as(t).reshape(-1)
    _plain_write(s["k_tree"].flatten(1, 2)[:, src], b, p, pos, s["k8"], s["k_scale"])
    _plain_write(s["v_tree"].flatten(1, 2)[:, src], b, p, pos, s["v8"], s["v_scale"])
    torch.add(s["kv_len"], s["acc"] + 1, out=s["new_len"])
    return s["k8"], s["v8"], s["k_scale"], s["v_scale"], s["new_len"]


# ---------------------------------------------------------------- the library's calls
def _own(s):
    import eagle_tree_speculative_gb300 as E
    if s["op"] == "prompt":
        return E.eagle_prompt_attn(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], scale=s["scale"], return_lse=True)
    if s["op"] == "append":
        E.eagle_kv8_append(s["k"], s["v"], s["cu"], s["pos"], s["k8"], s["v8"], s["k_scale"], s["v_scale"])
        return s["k8"], s["v8"], s["k_scale"], s["v_scale"]
    if s["op"] == "tree":
        return E.eagle_tree_attn_kv8(s["q"], s["k8"], s["v8"], s["k_scale"], s["v_scale"], s["k_tree"], s["v_tree"], s["kv_len"],
                                     s["parent"], scale=s["scale"])
    E.eagle_kv8_commit(s["k_tree"], s["v_tree"], s["k8"], s["v8"], s["k_scale"], s["v_scale"], s["kv_len"], s["path"], s["acc"],
                       s["depth"], kv_len_out=s["new_len"])
    return s["k8"], s["v8"], s["k_scale"], s["v_scale"], s["new_len"]


def run(state):
    if own:
        return _own(state)
    return {"prompt": _plain_prompt, "append": _plain_append, "tree": _plain_tree, "commit": _plain_commit}[state["op"]](state)


# ---------------------------------------------------------------- 64 bits, from the definitions
def _exact_rows(q, k, v, sees, scale):
    """softmax over the keys that `sees` [rows, keys] allows, of q [G, rows, D], k, v [keys, D], all float64."""
    x = (q @ k.T) * scale
    x = torch.where(sees, x, -math.inf)
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - torch.where(torch.isfinite(lse), lse, 0.0)[..., None])
    return p @ v, lse


def _exact_prompt(s, c):
    out = torch.empty((s["q"].shape[0], s["Hq"], D), dtype=torch.float64, device="cuda")
    lse = torch.empty(out.shape[:2], dtype=torch.float64, device="cuda")
    G, q0, k0 = s["Hq"] // s["Hkv"], 0, 0
    for nq, nk in zip(c["q"], c["k"]):
        for h in range(s["Hkv"]):
            hs = slice(h * G, (h + 1) * G)
            for i0 in range(0, nq, 2048):
                i1 = min(nq, i0 + 2048)
                end = nk - nq + i1                                # no query of the chunk sees a key from here on
                sees = torch.arange(end, device="cuda") <= torch.arange(nk - nq + i0, nk - nq + i1, device="cuda")[:, None]
                o, z = _exact_rows(s["q"][q0 + i0:q0 + i1, hs].double().transpose(0, 1), s["k"][k0:k0 + end, h].double(),
                                   s["v"][k0:k0 + end, h].double(), sees, s["scale"])
                out[q0 + i0:q0 + i1, hs], lse[q0 + i0:q0 + i1, hs] = o.transpose(0, 1), z.T
        q0, k0 = q0 + nq, k0 + nk
    return out, lse


def _exact_block(old_codes, old_scale, rows):
    """One block of one head: the codes of its rows (those held, then the new ones) and its scale."""
    top = float(rows.abs().max())
    e = E_MIN if top == 0.0 else max(E_MIN, math.ceil(math.log2(top / 448.0)))
    e = e if top <= 448.0 * 2.0 ** e else e + 1
    e = e - 1 if e > E_MIN and top <= 448.0 * 2.0 ** (e - 1) else e
    scale = 2.0 ** e if old_codes.shape[0] == 0 else max(2.0 ** e, old_scale)
    held = old_codes.double() * (old_scale / scale)
    return torch.cat([_e4m3(held), _e4m3(rows / scale)]), scale


def _e4m3(x):
    """The nearest e4m3 value, ties to the even one, of float64 |x| <= 448."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -40))).clamp(min=-6)
    e = torch.where(x.abs() >= torch.exp2(e + 1), e + 1, e)
    q = torch.exp2(e - 3)
    return torch.round(x / q) * q


def _exact_write(rows, pos, codes, scales):
    """rows[b]: [m, Hkv, D] new rows of sequence b (float64); codes [B, Hkv, Lmax, D], scales [B, Hkv, NB] (float64), in place."""
    for b, (x, at) in enumerate(zip(rows, pos)):
        for p0 in range(at // BLOCK * BLOCK, at + x.shape[0], BLOCK):
            lo, hi = max(at, p0), min(at + x.shape[0], p0 + BLOCK)
            for h in range(codes.shape[1]):
                held = codes[b, h, p0:lo]
                got, sc = _exact_block(held, float(scales[b, h, p0 // BLOCK]), x[lo - at:hi - at, h])
                codes[b, h, p0:hi], scales[b, h, p0 // BLOCK] = got, sc


def _exact_tree(s, c):
    out = torch.empty((s["B"], s["n"], s["Hq"], D), dtype=torch.float64, device="cuda")
    G, n = s["Hq"] // s["Hkv"], s["n"]
    for b, (L, parent) in enumerate(zip(c["L"], c["parent"])):
        sees = torch.zeros((n, L + n), dtype=torch.bool)
        sees[:, :L] = True
        for i in range(n):
            j = i
            while j >= 0:
                sees[i, L + j] = True
                j = parent[j]
        sees = sees.cuda()
        of = torch.arange(L, device="cuda") // BLOCK
        for h in range(s["Hkv"]):
            rows = lambda x8, sc, tree: torch.cat([x8[b, h, :L].double() * sc[b, h].double()[of, None], tree[b, :, h].double()])  # noqa: E731
            out[b, :, h * G:(h + 1) * G] = _exact_rows(s["q"][b, :, h * G:(h + 1) * G].double().transpose(0, 1), rows(s["k8"], s["k_scale"], s["k_tree"]),
                                                       rows(s["v8"], s["v_scale"], s["v_tree"]), sees, s["scale"])[0].transpose(0, 1)
    return out


def exact(case, seed):
    c = _counts(case)
    op = case["op"]
    if op in ("append", "commit"):  # block by block on the host: small cases only
        rows = sum(c["new"]) if op == "append" else sum(a + 1 for a in c["acc"]) * case["layers"]
        if rows * case["Hkv"] > 20000 or case.get("layers", 1) * case["B"] * case["Hkv"] > 4000:
            return None
    s = prepare(case, seed)
    if op == "prompt":
        return _exact_prompt(s, c)
    if op == "tree":
        return _exact_tree(s, c)
    host = lambda t: t.cpu().double()  # noqa: E731
    k8, v8, ks, vs = host(s["k8"]), host(s["v8"]), host(s["k_scale"]), host(s["v_scale"])
    if op == "append":
        cut = lambda x: host(x).split(c["new"])  # noqa: E731
        _exact_write(cut(s["k"]), c["pos"], k8, ks)
        _exact_write(cut(s["v"]), c["pos"], v8, vs)
        return k8, v8, ks, vs
    for layer in range(case["layers"]):
        for tree, codes, scales in ((s["k_tree"], k8, ks), (s["v_tree"], v8, vs)):
            t = host(tree[layer])
            rows = [t[b, p[:a + 1]] for b, (p, a) in enumerate(zip(c["path"], c["acc"]))]
            _exact_write(rows, c["L"], codes[layer], scales[layer])
    return k8, v8, ks, vs, None
