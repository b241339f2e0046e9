"""Plain 64-bit CPU forms of the prompt attention and of the calls on the 8-bit K/V cache,
written from their definitions (torch float64 on the CPU, one sequence and head at a time).

The attention forms also return, per output element, how far a result may be off when the
softmax weights are rounded before they are multiplied with V: with the weights p_j = exp(s_j
- max s) and a rounding error of at most w_j on p_j,

    |error| <= half |out|  +  sum_j (w_j + c p_j) |v_j| / sum_j p_j

where half = 2^-8 is the output's own rounding to bf16 (half a step) and c covers fp32: the
scores are sums of 128 products (each product exact, 128 additions of 2^-24 relative to the
sum of magnitudes A), so a weight is off by a factor of exp(2^-17 A) or so; the exponential
(2^-21) and the sum of the weights (2^-24 a term) come on top, once in the weight and once in
the sum.
"""
from __future__ import annotations

import numpy as np
import torch

KV8_BLOCK = 32
E_MIN = -64
HALF_BF16 = 2.0 ** -8


def _softmax_rows(q, k, v, sees, scale, w_rel, w_abs, extra=0.0):
    """q [R, d], k / v [N, d] float64, sees bool [R, N] -> out [R, d], lse [R], tolerance [R, d].
    Weights are rounded by at most max(w_rel p, w_abs); `extra`: a further error of a score,
    relative to scale * max|q| * sum|k|."""
    R = q.shape[0]
    s = torch.where(sees, (q @ k.T) * scale, -torch.inf)
    some = sees.any(1)
    m = torch.where(some, s.amax(1) if k.shape[0] else torch.full((R,), -torch.inf).double(), 0.0)
    p = torch.where(sees, torch.exp(s - m[:, None]), 0.0)
    l = p.sum(1)
    safe = torch.where(l > 0, l, 1.0)
    out = (p @ v) / safe[:, None]
    lse = torch.where(some, m + torch.log(safe), -torch.inf)
    A = (q.abs() @ k.abs().T) * scale
    ds = 2.0 ** -17 * A + extra * scale * q.abs().amax(1)[:, None] * k.abs().sum(1)[None]
    ds = torch.where(sees, ds, 0.0)
    ds_max = ds.amax(1, keepdim=True) if k.shape[0] else torch.zeros(R, 1).double()
    n = sees.sum(1, keepdim=True).double()
    c = 2.0 * (torch.expm1(ds_max) + 2.0 ** -21 + n * 2.0 ** -24)
    w = torch.maximum(w_rel * p, torch.full_like(p, w_abs) * sees) + c * p
    tol = HALF_BF16 * out.abs() + (w @ v.abs()) / safe[:, None]
    return out, lse, tol


def prompt_attn(q, k, v, cu_q, cu_k, scale):
    """q [Tq, Hq, d], k / v [Tk, Hkv, d] (bf16 values), cu_q / cu_k lists of B + 1.  Rows of
    no sequence come back as NaN.  The weights are rounded to bf16 (half a step: 2^-8)."""
    q, k, v = (t.double().cpu() for t in (q, k, v))
    Tq, Hq, d = q.shape
    G = Hq // k.shape[1]
    out = torch.full((Tq, Hq, d), torch.nan).double()
    lse = torch.full((Tq, Hq), torch.nan).double()
    tol = torch.zeros(Tq, Hq, d).double()
    for b in range(len(cu_q) - 1):
        q0, q1, k0, k1 = int(cu_q[b]), int(cu_q[b + 1]), int(cu_k[b]), int(cu_k[b + 1])
        nq, nk = q1 - q0, k1 - k0
        sees = torch.arange(nk)[None] <= (nk - nq + torch.arange(nq))[:, None]
        for h in range(Hq):
            o, z, t = _softmax_rows(q[q0:q1, h], k[k0:k1, h // G], v[k0:k1, h // G], sees, scale,
                                    HALF_BF16, 0.0)
            out[q0:q1, h], lse[q0:q1, h], tol[q0:q1, h] = o, z, t
    return out, lse, tol


def scale_of(amax: float) -> float:
    """The least 2^e, e >= E_MIN, with amax <= 448 * 2^e (exact: e4m3's largest value times a
    power of two is a double)."""
    e = E_MIN
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


# every finite e4m3 value with its code, in order of the value
_CODES = np.array([c for c in range(256) if c & 0x7F != 0x7F], np.uint8)
_VALUES = torch.from_numpy(_CODES.copy()).view(torch.float8_e4m3fn).double().numpy()


def e4m3(x: np.ndarray) -> np.ndarray:
    """The codes of the nearest e4m3 values, ties to the even code, beyond 448 to +-448,
    NaN to NaN; by search over all values."""
    pos = np.sort(_VALUES[_VALUES >= 0])[1:]             # one zero, then the codes 0 .. 126 in order
    a = np.minimum(np.abs(x), 448.0)
    a = np.where(np.isnan(x), 0.0, a)
    hi = np.searchsorted(pos, a).clip(max=126)
    lo = np.where(pos[hi] == a, hi, np.maximum(hi - 1, 0))
    d_lo, d_hi = a - pos[lo], pos[hi] - a
    code = np.where((d_hi < d_lo) | ((d_hi == d_lo) & (lo % 2 == 1)), hi, lo).astype(np.uint8)
    code = np.where(np.isnan(x), 0x7F, code).astype(np.uint8)
    return code | (np.signbit(x).astype(np.uint8) << 7)


def _value(codes: np.ndarray) -> np.ndarray:
    return torch.from_numpy(np.ascontiguousarray(codes)).view(torch.float8_e4m3fn).double().numpy()


def write_rows(x, at, codes, scales):
    """Rows x [m, d] (float64) of one head behind its first `at` rows: codes uint8 [Lmax, d],
    scales float64 [NB], in place."""
    m = x.shape[0]
    for blk in range(at // KV8_BLOCK, -(-(at + m) // KV8_BLOCK) if m else 0):
        r0 = blk * KV8_BLOCK
        lo, hi = max(at, r0), min(at + m, r0 + KV8_BLOCK)
        new = x[lo - at:hi - at]
        fin = np.abs(new[np.isfinite(new)])
        sc = scale_of(float(fin.max()) if fin.size else 0.0)
        if lo > r0:
            sc = max(sc, scales[blk])
            if sc > scales[blk]:
                codes[r0:lo] = e4m3(_value(codes[r0:lo]) * (scales[blk] / sc))
        codes[lo:hi] = e4m3(new / sc)
        scales[blk] = sc


def kv8_append(x, cu, pos, codes, scales):
    """x [T, Hkv, d] (float64), codes uint8 [B, Hkv, Lmax, d], scales float64 [B, Hkv, NB]."""
    for b in range(len(pos)):
        rows = x[int(cu[b]):int(cu[b + 1])]
        for h in range(codes.shape[1]):
            write_rows(rows[:, h], int(pos[b]), codes[b, h], scales[b, h])


def kv8_commit(x, kv_len, path, acc, codes, scales):
    """x [layers, B, n, Hkv, d] (float64); codes and scales with a leading layers."""
    for layer in range(x.shape[0]):
        for b in range(x.shape[1]):
            if acc[b] >= 0:
                rows = x[layer, b, [int(i) for i in path[b][:int(acc[b]) + 1]]]
                for h in range(codes.shape[2]):
                    write_rows(rows[:, h], int(kv_len[b]), codes[layer, b, h], scales[layer, b, h])


def _tree_sees(n, L, parent):
    """bool [n, L + n]: the cache's L rows, then the tree's."""
    sees = torch.zeros(n, L + n, dtype=torch.bool)
    sees[:, :L] = True
    for i in range(n):
        j = i
        while j >= 0:
            sees[i, L + j] = True
            j = int(parent[j])
    return sees


def _key_rows(codes, scales, tree, b, h, L):
    """float64 [L + n, d]: rows of the cache, then the tree's."""
    blk = np.arange(L) // KV8_BLOCK
    return torch.cat([torch.from_numpy(_value(codes[b, h, :L]) * scales[b, h][blk][:, None]), tree[b, :, h]])


def tree_attn_kv8(q, codes, scales, v_codes, v_scales, k_tree, v_tree, kv_len, parent, scale):
    """q [B, n, Hq, d], k_tree / v_tree [B, n, Hkv, d] (bf16 values); codes uint8 [B, Hkv, Lmax,
    d], scales float64.  The tolerance is a loose one, that of weights held in two 4-bit digits
    (2^-8 of the weight, and for small ones 2^-10 on a scale where the largest is at least 2^6);
    tree_attn_kv8_tight has the kernel's own."""
    q, kt, vt = (t.double().cpu() for t in (q, k_tree, v_tree))
    B, n, Hq, d = q.shape
    Hkv = kt.shape[2]
    G = Hq // Hkv
    out = torch.zeros(B, n, Hq, d).double()
    tol = torch.zeros(B, n, Hq, d).double()
    for b in range(B):
        L = int(kv_len[b])
        sees = _tree_sees(n, L, parent[b])
        for h in range(Hkv):
            k, v = _key_rows(codes, scales, kt, b, h, L), _key_rows(v_codes, v_scales, vt, b, h, L)
            top = v[L:].abs().amax(1, keepdim=True) * 2.0 ** -17
            slack = torch.cat([torch.zeros(L, 1), top]).double()
            for g in range(G):
                o, _, t = _softmax_rows(q[b, :, h * G + g], k, v, sees, scale, HALF_BF16, 2.0 ** -16,
                                        extra=2.0 ** -16)
                out[b, :, h * G + g], tol[b, :, h * G + g] = o, t + slack.max()
    return out, tol


KV8_SPREAD = 8        # a larger spread of V exponents: weights in bf16


def _row_exponents(v):
    """The exponents e that bring each row's largest magnitude to [128, 256); NaN for a row below
    2^-120, which counts as zeros."""
    top = v.abs().amax(1)
    e = torch.floor(torch.log2(torch.where(top >= 2.0 ** -120, top, torch.nan))) - 7
    return e


def tree_attn_kv8_tight(q, codes, scales, v_codes, v_scales, k_tree, v_tree, kv_len, parent, scale):
    """As tree_attn_kv8, with the tolerance of the roundings that the kernel makes.  With scores s
    in log2 units, weights p = 2^(s - max s) and ev the exponent of a V row (its block's scale, or that
    which brings a tree row's largest magnitude to [128, 256)):

      query    two 4-bit digits of each element on a scale where the row's largest is in [128, 256).
               Elements from 2^-2 on are exact; below, each digit is off by half a step of 2^-9 at
               most: together 2^-16 of the row's largest.  The tree's keys the same.
      scores   256 products (two digits), each addition off by 2^-24 of the sum of magnitudes A:
               2^-16 A; the factor, the product with it and the subtraction of the maximum: 2^-22 of
               the largest A.
      weights  fp16 P = 2^(s + ev - m + 6 or more), m at most the largest s + ev: half a step is 2^-11
               of P, and 2^-25 where P is below 2^-14, which is 2^(m - max s - ev - 31) of p.  Where the
               exponents spread over more than KV8_SPREAD (or one is below -64), bf16: 2^-8 of P; a
               part of the keys may still be within the spread and in fp16, off by 2^(KV8_SPREAD - 31).
      V        codes are exact; of the tree's rows elements far below the largest are fp16 subnormals:
               2^-25 on the scale 2^ev.
      sums, exponential, output  as above, and 2^-8 of the result."""
    q, kt, vt = (t.double().cpu() for t in (q, k_tree, v_tree))
    B, n, Hq, d = q.shape
    Hkv = kt.shape[2]
    G = Hq // Hkv
    log2e = 1.4426950408889634
    out = torch.zeros(B, n, Hq, d).double()
    tol = torch.zeros(B, n, Hq, d).double()
    for b in range(B):
        L = int(kv_len[b])
        sees = _tree_sees(n, L, parent[b])
        blk = np.arange(L) // KV8_BLOCK
        tree = torch.arange(L + n) >= L
        for h in range(Hkv):
            k, v = _key_rows(codes, scales, kt, b, h, L), _key_rows(v_codes, v_scales, vt, b, h, L)
            ev = torch.cat([torch.from_numpy(np.log2(v_scales[b, h][blk])), _row_exponents(v[L:])])
            known = ev[~torch.isnan(ev)]
            wide = known.numel() > 0 and (float(known.max() - known.min()) > KV8_SPREAD or float(known.min()) < E_MIN)
            ev = torch.where(torch.isnan(ev), float(E_MIN), ev)
            v_off = torch.where(tree, torch.exp2(ev - 25), 0.0)[:, None]
            for g in range(G):
                x = q[b, :, h * G + g]
                s = torch.where(sees, (x @ k.T) * (scale * log2e), -torch.inf)
                top = s.amax(1, keepdim=True)
                p = torch.exp2(s - top)
                l = p.sum(1, keepdim=True)
                A = (x.abs() @ k.abs().T) * scale
                xm, km = x.abs().amax(1)[:, None], k.abs().amax(1)[None]
                ds = 2.0 ** -16 * A + 2.0 ** -16 * scale * (xm * k.abs().sum(1)[None] + torch.where(
                    tree, x.abs().sum(1)[:, None] * km + 2.0 ** -16 * d * xm * km, 0.0))
                ds = torch.where(sees, ds, 0.0).amax(1, keepdim=True)
                ds = ds + 2.0 ** -22 * torch.where(sees, A, 0.0).amax(1, keepdim=True)
                c = 2.0 * (torch.expm1(ds) + 2.0 ** -21 + sees.sum(1, keepdim=True).double() * 2.0 ** -24)
                if wide:
                    w = 2.0 ** -8 * p + 2.0 ** (KV8_SPREAD - 31) * sees
                else:
                    m = (s + ev).amax(1, keepdim=True)
                    w = torch.maximum(2.0 ** -11 * p, torch.exp2(m - top - ev - 31) * sees)
                o = (p @ v) / l
                out[b, :, h * G + g] = o
                tol[b, :, h * G + g] = HALF_BF16 * o.abs() + ((w + c * p) @ v.abs() + p @ v_off.expand(-1, d)) / l
    return out, tol
