"""Attention over pages with refused sequences so long that many pieces of the work hold a part of them: what they
write goes through the workspace and the merging, beside sequences that are done."""
import numpy as np
import pytest
import torch

from oracle import paged as ref

pytestmark = pytest.mark.gpu
D = 128
BAD_TREE, CAPACITY = 0x01, 0x10


def _bf16(shape, seed, gain=0.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * torch.exp(gain * torch.randn(shape[-1], generator=g))).bfloat16()


def _dev(x):
    return torch.as_tensor(np.asarray(x)).to(torch.int32).cuda().contiguous()


@pytest.mark.parametrize("n,Hq,Hkv", [(1, 8, 1), (4, 4, 1), (60, 4, 1), (60, 8, 2), (40, 8, 1), (64, 5, 1)])
@pytest.mark.parametrize("bad", [0, 1, 2])
def test_long_sequences_with_invalid_trees_are_zeros(n, Hq, Hkv, bad):
    """Single row tiles, pairs, and three row tiles; the refused sequence first, in the middle, last."""
    import eagle_tree_speculative_gb300 as E
    rng, page = np.random.default_rng(n), 64
    L = [300, 300, 300]
    L[bad] = 20000
    L[(bad + 1) % 3] = 5000
    need = [-(-(x + n) // page) for x in L]
    N = sum(need) + 1
    ids = list(rng.permutation(N))
    table = np.full((3, max(need)), -1, np.int64)
    for b, m in enumerate(need):
        table[b, :m] = [ids.pop() for _ in range(m)]
    parent = [[-1] + [int(rng.integers(max(0, i - 6), i)) for i in range(1, n)] for _ in L]
    parent[bad][n // 2] = n // 2                              # (a root whose parent is 0, where there is one node)
    q, kp, vp = _bf16((3, n, Hq, D), 1), _bf16((N, Hkv, page, D), 2), _bf16((N, Hkv, page, D), 3)
    size = E.tree_attn_paged_workspace_size(3, n, Hq, Hkv, D, page, table.shape[1])
    ws = torch.full((size,), 0xff, dtype=torch.uint8, device="cuda")
    out = torch.full((3, n, Hq, D), torch.nan, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (q.cuda(), kp.cuda(), vp.cuda(), _dev(table), _dev(L), _dev(parent))
    E.eagle_tree_attn_paged(*args, out=out, workspace=ws, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == BAD_TREE
    got = out.double().cpu()
    assert not bool(got[bad].any()) and not bool(torch.isnan(got).any())
    want, tol = ref.tree_attn_paged(q, kp, vp, table, L, parent, D ** -0.5)
    assert bool(((got - want).abs() <= tol).all())
    # the parts that the call before left in the workspace do not show
    again = torch.full_like(out, torch.nan)
    E.eagle_tree_attn_paged(*args, out=again, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(again, out)
