"""Plain 64-bit CPU forms of the calls on the paged K/V cache, written from their definitions
(Python and torch float64 on the CPU, one sequence, head or row at a time).

The two calls that compute also return, per output element, how far a result may be off.
"""
from __future__ import annotations

import math

import torch

from .prompt_kv8 import HALF_BF16, _softmax_rows


def depths(parent):
    """Depth of every node of one tree; None if it is none."""
    d = []
    for i, p in enumerate(parent):
        if (p != -1) if i == 0 else not 0 <= p < i:
            return None
        d.append(0 if i == 0 else d[p] + 1)
    return d


def places(table, page, rows):
    """(page number, row in it) of the given rows of one sequence."""
    return [(int(table[r // page]), r % page) for r in rows]


# ---------------------------------------------------------------- norms and rotation
def turned(x, w, inv_freq, position, eps, interleaved):
    """One token's heads x [H, d] (bf16 values): out [H, d] and tolerance [H, d].

    fp32 work on the way: the norm's factor (128 squares, their sum in 7 levels, rsqrt within 2 ulp)
    and its two products, at most 14 * 2^-24 of y; the angle to 2^-29 of a turn, its sine and cosine
    within 2 ulp and 2^-24, together 2^-21 of the pair; two products and a sum.  All in all below
    2^-19 of |y_i| + |y_j|, beside the one rounding to bf16 (half a step, 2^-8)."""
    x = x.double()
    H, d = x.shape
    y = x.clone()
    if w is not None:
        y = x / torch.sqrt((x * x).sum(1, keepdim=True) / d + eps) * w.double()
    f = inv_freq.double()
    half = f.numel()
    out, size = y.clone(), y.abs()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = math.cos(position * float(f[i])), math.sin(position * float(f[i]))
        out[:, a] = y[:, a] * c - y[:, b] * s
        out[:, b] = y[:, b] * c + y[:, a] * s
        size[:, a] = size[:, b] = y[:, a].abs() + y[:, b].abs()
    tol = HALF_BF16 * out.abs() + 2.0 ** -19 * size
    # from half a step above the largest bf16 value, 2^128 (1 - 2^-8), on, rounding gives infinity
    return torch.where(out.abs() >= 2.0 ** 128 * (1 - 2.0 ** -9), torch.copysign(torch.full_like(out, torch.inf), out), out), tol


def qkv_rope(q, k, v, q_weight, k_weight, inv_freq, pos, cu, parent, eps, interleaved, page, N, table):
    """q [T, Hq, d], k / v [T, Hkv, d]; cu or parent as lists.  Returns per token (None where nothing is
    written) a dict of q, k (out, tolerance), v and place (None, or page number and row)."""
    out = [None] * q.shape[0]
    for b, p in enumerate(pos):
        if parent is None:
            rows = list(range(cu[b], cu[b + 1]))
            ahead = list(range(len(rows)))
        else:
            n = len(parent[b])
            rows = list(range(b * n, b * n + n))
            ahead = depths(parent[b])
        room = 2 ** 31 - 1 if table is None else table.shape[1] * page
        if ahead is None or p < 0 or p + len(rows) > room:
            continue
        for i, t in enumerate(rows):
            at = None
            if table is not None:
                at = places(table[b], page, [p + i])[0]
                at = at if 0 <= at[0] < N else None
            out[t] = dict(q=turned(q[t], q_weight, inv_freq, p + ahead[i], eps, interleaved),
                          k=turned(k[t], k_weight, inv_freq, p + ahead[i], eps, interleaved), v=v[t], place=at)
    return out


# ---------------------------------------------------------------- attention
def tree_attn_paged(q, k_pages, v_pages, table, kv_len, parent, scale):
    """q [B, n, Hq, d], pages [N, Hkv, page, d] (bf16 values), table / parent int arrays.  A refused
    sequence gives zeros.  The weights are rounded to bf16 (half a step: 2^-8)."""
    B, n, Hq, d = q.shape
    N, Hkv, page, _ = k_pages.shape
    G = Hq // Hkv
    out = torch.zeros(B, n, Hq, d, dtype=torch.float64)
    tol = torch.zeros_like(out)
    for b in range(B):
        L, par = int(kv_len[b]), [int(x) for x in parent[b]]
        if depths(par) is None or L < 0 or L + n > table.shape[1] * page:
            continue
        sees = torch.zeros(n, L + n, dtype=torch.bool)
        sees[:, :L] = True
        for i in range(n):
            j = i
            while j >= 0:
                sees[i, L + j] = True
                j = par[j]
        at = places(table[b], page, range(L + n))
        ids = torch.tensor([p for p, _ in at])
        rows = torch.tensor([r for _, r in at])
        there = (ids >= 0) & (ids < N)
        for h in range(Hkv):
            k, v = (torch.where(there[:, None], x[ids.clamp(0, N - 1), h, rows].double(), 0.0) for x in (k_pages, v_pages))
            for g in range(h * G, h * G + G):
                out[b, :, g], _, tol[b, :, g] = _softmax_rows(q[b, :, g].double(), k, v, sees, scale, HALF_BF16, 0.0)
    return out, tol


# ---------------------------------------------------------------- which pages a slot holds
def pages_assign(table, held, refs, kv_len, grow, src, page):
    """Lists in, the new (table, held, refs, kv_len) and the copies [(from, to, rows)] out; None if the call
    is refused."""
    B, P, N = len(held), len(table[0]), len(refs)
    src = list(range(B)) if src is None else list(src)
    free = [p for p in range(N) if refs[p] == 0]
    new, lens, copies = [], [], []
    for b in range(B):
        s = src[b]
        if not -1 <= s < B or grow[b] < 0:
            return None
        L = kv_len[s] if s >= 0 else 0
        if L < 0 or (s >= 0 and L > held[s] * page) or -(-(L + grow[b]) // page) > P:
            return None
        need, row = -(-(L + grow[b]) // page), []
        for t in range(need):
            mine = None                                   # the page that stays
            if t < L // page:
                mine = table[s][t]
            elif s >= 0 and t < held[s] and refs[table[s][t]] <= 1:
                ends_here = t == L // page and L % page
                if s == b or (ends_here and src[s] != s and b == min(x for x in range(B) if src[x] == s)):
                    mine = table[s][t]
            if mine is None:
                if not free:
                    return None
                mine = free.pop(0)
                if t == L // page and L % page:
                    copies.append((table[s][t], mine, L % page))
            row.append(mine)
        new.append(row)
        lens.append(L)
    out, count = [], list(refs)
    for b in range(B):
        for t in range(held[b]):
            count[table[b][t]] -= 1
        for p in new[b]:
            count[p] += 1
        m = len(new[b])
        out.append(new[b] + [-1 if t < held[b] else table[b][t] for t in range(m, P)])
    return out, [len(r) for r in new], count, lens, copies


def pages_commit(pages, table, kv_len, path, accept_len, max_depth, page, N):
    """pages: tensors [layers, N, Hkv, page, d], in place; returns the new lengths."""
    lens = []
    for b, (L, a) in enumerate(zip(kv_len, accept_len)):
        p = [int(x) for x in path[b][:max(a, -1) + 1]]
        cap = len(table[b]) * page
        ok = 0 <= a <= max_depth and L >= 0 and L + a + 1 <= cap and p[0] == 0 and all(y > x for x, y in zip(p, p[1:]))
        ok = ok and L + p[-1] < cap
        if ok:
            moves = [t for t in range(a + 1) if p[t] != t]
            frm, to = places(table[b], page, [L + p[t] for t in moves]), places(table[b], page, [L + t for t in moves])
            ok = all(0 <= x < N for x, _ in frm + to)
        if not ok:
            lens.append(L)
            continue
        for x in pages:
            rows = [x[:, i, :, r].clone() for i, r in frm]
            for (i, r), row in zip(to, rows):
                x[:, i, :, r] = row
        lens.append(L + a + 1)
    return lens
