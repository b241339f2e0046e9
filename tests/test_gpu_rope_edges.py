"""The norms and the rotation at the edges of what their arguments allow, against the 64-bit form of oracle/paged.py."""
import numpy as np
import pytest
import torch

from oracle import paged as ref

pytestmark = pytest.mark.gpu
D = 128


def _E():
    import eagle_tree_speculative_gb300 as E
    return E


def _bf16(shape, seed, gain=0.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * torch.exp(gain * torch.randn(shape[-1], generator=g))).bfloat16()


def _dev(x):
    return torch.as_tensor(np.asarray(x)).to(torch.int32).cuda().contiguous()


def _freq(rot=D):
    return (10000.0 ** -(torch.arange(0, rot, 2).double() / rot)).float()


def _within(got, want, tol):
    """Every value within its bound, NaN and infinities where they are due."""
    g = got.double().cpu()
    same = (g == want) | (torch.isnan(g) & torch.isnan(want))
    return bool((same | ((g - want).abs() <= tol)).all())


def _norms(size, weight, eps, seed=1):
    """Five tokens of 3 / 1 heads, `size` and `weight` times an ordinary one's values and weights."""
    T, Hq, Hkv = 5, 3, 1
    q, k = _bf16((T, Hq, D), seed) * size, _bf16((T, Hkv, D), seed + 1) * size
    qw, kw = (_bf16((D,), seed + 2) + 1) * weight, (_bf16((D,), seed + 3) + 1) * weight
    f = _freq()
    a, b = _E().eagle_qkv_rope(q.cuda(), k.cuda(), None, f.cuda(), _dev([7]), cu=_dev([0, T]), q_weight=qw.cuda(), k_weight=kw.cuda(), eps=eps)
    for t in range(T):
        assert _within(a[t], *ref.turned(q[t], qw, f, 7 + t, eps, False)), t
        assert _within(b[t], *ref.turned(k[t], kw, f, 7 + t, eps, False)), t


@pytest.mark.parametrize("size,weight,eps", [(2.0 ** 58, 2.0 ** -90, 1e-6), (2.0 ** 58, 2.0 ** -60, 1e-6), (2.0 ** -55, 2.0 ** 100, 2.0 ** -115)])
def test_weights_far_from_one_over_heads_far_from_one(size, weight, eps):
    """The factor of a head times its weight leaves fp32 where the normed head times its weight does not."""
    _norms(size, weight, eps)


@pytest.mark.parametrize("size,eps", [(2.0 ** 62, 2.0 ** 123), (2.0 ** 66, 2.0 ** 127), (1.0, 2.0 ** 127), (2.0 ** -70, 2.0 ** -140),
                                      (2.0 ** -75, 2.0 ** -149), (2.0 ** -50, 2.0 ** -100), (2.0 ** -52, 2.0 ** -101)])
def test_eps_beside_squares_at_the_ends_of_fp32(size, eps):
    """Squares that overflow beside an eps that counts, squares that are denormal or zero beside one that does not."""
    _norms(size, 1.0, eps)


@pytest.mark.parametrize("n", [0, 1, 9])
def test_an_empty_batch_of_trees(n):
    E = _E()
    q, k = (torch.empty(0, H, D, dtype=torch.bfloat16, device="cuda") for H in (4, 2))
    kp, vp, table, _, _ = E.paged_cache(1, 5, 2, 16, 0, 3)
    parent = _dev(np.zeros((0, n)))
    a, b = E.eagle_qkv_rope(q, k, None, _freq().cuda(), _dev([]), parent=parent)
    assert a.shape == q.shape and b.shape == k.shape
    a, b = E.eagle_qkv_rope(q, k, k, _freq().cuda(), _dev([]), parent=parent, k_pages=kp[0], v_pages=vp[0], page_table=table)
    assert a.shape == q.shape and b is None
    with pytest.raises((TypeError, ValueError)):
        E.eagle_qkv_rope(q, k, None, _freq().cuda(), _dev([]), parent=_dev([]))


@pytest.mark.parametrize("Hq,Hkv,norm", [(6, 2, True), (3, 1, False)])
def test_a_call_that_streams(Hq, Hkv, norm):
    """Enough tokens for the launch of long calls (four a warp with 12 warps an SM), a tail behind the whole ones that
    the warps share, more than 32 sequences (empty ones among them), rows both packed and into pages, strided."""
    E, page = _E(), 64
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rng = np.random.default_rng(Hq)
    B, least = 70, sms * 3 * 4 * 4
    lens = [int(x) for x in rng.integers(0, 2 * least // B, B)]
    lens[5] = lens[33] = lens[69] = 0
    lens[40] += max(0, least - sum(lens)) + 801
    T, pos = sum(lens), [int(x) for x in rng.integers(0, 500, B)]
    assert T >= least and T % (sms * 12)
    cu = [0] + [int(x) for x in np.cumsum(lens)]
    need = [-(-(p + m) // page) - p // page for p, m in zip(pos, lens)]
    N = sum(need) + 2
    ids = list(rng.permutation(N))
    table = np.full((B, max(-(-(p + m) // page) for p, m in zip(pos, lens))), -1, np.int64)
    for b, (p, m) in enumerate(zip(pos, need)):
        table[b, p // page:p // page + m] = [ids.pop() for _ in range(m)]
    qkv = _bf16((T, (Hq + 2 * Hkv) * D + 8), 1)
    q, k, v = (x.unflatten(1, (-1, D)) for x in qkv[:, :(Hq + 2 * Hkv) * D].split([Hq * D, Hkv * D, Hkv * D], 1))
    qw, kw = ((_bf16((D,), 2) + 1), (_bf16((D,), 3) + 1)) if norm else (None, None)
    f = _freq()
    kp, vp = _bf16((N, Hkv, page, D), 4), _bf16((N, Hkv, page, D), 5)
    gq, gk, gv = (x.unflatten(1, (-1, D)) for x in qkv.cuda()[:, :(Hq + 2 * Hkv) * D].split([Hq * D, Hkv * D, Hkv * D], 1))
    gkp, gvp, k_out = kp.cuda(), vp.cuda(), torch.empty(T, Hkv, D, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    a, b = E.eagle_qkv_rope(gq, gk, gv, f.cuda(), _dev(pos), cu=_dev(cu), q_weight=None if qw is None else qw.cuda(),
                            k_weight=None if kw is None else kw.cuda(), k_pages=gkp, v_pages=gvp, page_table=_dev(table), k_out=k_out, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    a, b = a.cpu(), b.cpu()
    seq = np.repeat(np.arange(B), lens)
    row = np.concatenate([np.arange(m) for m in lens])
    at = np.array(pos)[seq] + row
    ids, r = torch.as_tensor(table[seq, at // page]), torch.as_tensor(at % page)
    for t in sorted({*range(0, T, 211), *(c for c in cu if c < T), *(c - 1 for c in cu if c > 0), *range(T - 30, T)}):
        assert _within(a[t], *ref.turned(q[t], qw, f, int(at[t]), 1e-6, False)), t
        assert _within(b[t], *ref.turned(k[t], kw, f, int(at[t]), 1e-6, False)), t
    # every row of every page: the rows of the sequences, and as they were elsewhere
    kp[ids, :, r], vp[ids, :, r] = b, v
    assert torch.equal(gkp.cpu(), kp) and torch.equal(gvp.cpu(), vp)
    # every token, by the same call over few of them
    for t0 in range(0, T, 1500):
        some = slice(t0, min(T, t0 + 1500))
        part = [0] + [int(min(max(c - t0, 0), some.stop - t0)) for c in cu[1:]]
        begins = [p + max(0, min(t0, c1) - c0) for p, c0, c1 in zip(pos, cu, cu[1:])]
        x, y = E.eagle_qkv_rope(gq[some], gk[some], None, f.cuda(), _dev(begins), cu=_dev(part), q_weight=None if qw is None else qw.cuda(),
                                k_weight=None if kw is None else kw.cuda())
        assert torch.equal(x.cpu(), a[some]) and torch.equal(y.cpu(), b[some]), t0
