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
