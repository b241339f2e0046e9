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


def test_calls_behind_a_refused_assignment_write_into_nobody_else_s_pages():
    """No page is free: the fork and the room for a tree are refused, and what runs on with the old table stores the rows
    that the slots have pages for, in pages of their own; the shared ones stay."""
    import eagle_tree_speculative_gb300 as E
    B, page, N, n, Hq, Hkv, depth = 3, 16, 6, 20, 4, 2, 3
    _, _, table, held, refs = E.paged_cache(0, N, Hkv, page, B, 8)
    kp, vp = _bf16((1, N, Hkv, page, D), 1).cuda(), _bf16((1, N, Hkv, page, D), 2).cuda()
    kv_len, st = _dev([0] * B), torch.zeros(1, dtype=torch.int32, device="cuda")
    E.eagle_pages_assign(kp, vp, table, held, refs, kv_len, _dev([40, 20, 0]), dev_status=st)
    kv_len.copy_(_dev([40, 20, 0]))
    E.eagle_pages_assign(kp, vp, table, held, refs, kv_len, _dev([0] * B), src=_dev([0, 1, 0]), dev_status=st)
    assert int(st.item()) == 0 and refs.tolist() == [2, 2, 1, 1, 1, 1] and held.tolist() == [3, 2, 3]
    was = [x.clone() for x in (table, held, refs, kv_len, kp, vp)]
    E.eagle_pages_assign(kp, vp, table, held, refs, kv_len, _dev([n] * B), src=_dev([1, 1, 0]), dev_status=st)
    assert int(st.item()) == CAPACITY
    assert all(torch.equal(x, y) for x, y in zip((table, held, refs, kv_len, kp, vp), was))
    L, parent = kv_len.tolist(), [[-1] + [(i - 1) // 2 for i in range(1, n)]] * B
    q, k, v = _bf16((B * n, Hq, D), 3).cuda(), _bf16((B * n, Hkv, D), 4).cuda(), _bf16((B * n, Hkv, D), 5).cuda()
    f = (10000.0 ** -(torch.arange(0, D, 2).double() / D)).float().cuda()
    k_out = torch.empty_like(k)
    st.zero_()
    qr, _ = E.eagle_qkv_rope(q, k, v, f, kv_len, parent=_dev(parent), k_pages=kp[0], v_pages=vp[0], page_table=table, k_out=k_out, dev_status=st)
    assert int(st.item()) == CAPACITY                          # rows without a page
    E.eagle_tree_attn_paged(qr.view(B, n, Hq, D), kp[0], vp[0], table, kv_len, _dev(parent))
    want = [x.clone() for x in was[4:]]
    rows = table.tolist()
    for b in range(B):
        for i in range(n):
            at = L[b] + i
            if rows[b][at // page] >= 0:
                want[0][0, rows[b][at // page], :, at % page], want[1][0, rows[b][at // page], :, at % page] = k_out[b * n + i], v[b * n + i]
    assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])
    assert all(torch.equal(x[:, :2], y[:, :2]) for x, y in zip((kp, vp), was[4:]))
    # the path of slot 0 lies in rows that it has, those of the others do not: they are skipped
    st.zero_()
    E.eagle_pages_commit(kp, vp, table, kv_len, _dev([[0, 2, 5, 7], [0, 2, 13, 14], [0, 1, 3, 9]]), _dev([3, 3, 3]), depth, dev_status=st)
    assert int(st.item()) == CAPACITY and kv_len.tolist() == [44, 20, 40]
    for x, w in zip((kp, vp), want):
        own = w[0, rows[0][2]].clone()
        for t, p in ((1, 2), (2, 5), (3, 7)):
            own[:, 8 + t] = w[0, rows[0][2], :, 8 + p]
        w[0, rows[0][2]] = own
        assert torch.equal(x, w)
