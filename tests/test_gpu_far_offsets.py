"""Prompt attention and the 8-bit cache's calls where offsets pass 32 bits: a cache of more than 4 GB and token rows
spread over more than 2^32 elements."""
import numpy as np
import pytest
import torch

from oracle import prompt_kv8 as ref

pytestmark = pytest.mark.gpu
D = 128


def _E():
    import eagle_tree_speculative_gb300 as E
    return E


def _dev(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _bf16(shape, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * torch.exp(0.5 * torch.randn(shape[-1], generator=g))).bfloat16()


def _room(gb):
    if torch.cuda.mem_get_info()[0] < gb * 2 ** 30:
        pytest.skip(f"needs {gb} GB")


def test_cache_of_more_than_4_gb():
    """300 sequences of 128 heads and 1000 rows (4.9 GB of K codes, as much of V): rows are appended to the last
    sequence, attended and followed by a committed path; nothing else changes."""
    _room(24)
    E = _E()
    B, Hkv, Lmax, n, depth = 300, 128, 1000, 3, 2
    k8, v8, ks, vs = E.kv8_cache(1, B, Hkv, Lmax)
    assert k8.numel() > 2 ** 32
    m, at = 70, 900
    x, y = _bf16((m, Hkv, D), 1), _bf16((m, Hkv, D), 2)
    cu, pos, kv_len = np.zeros(B + 1), np.zeros(B), np.zeros(B)
    cu[B], pos[B - 1], kv_len[B - 1] = m, at, at + m
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    E.eagle_kv8_append(x.cuda(), y.cuda(), _dev(cu), _dev(pos), k8[0], v8[0], ks[0], vs[0], dev_status=st)
    want = []
    for t in (x, y):
        codes, scales = np.zeros((1, Hkv, Lmax, D), np.uint8), np.ones((1, Hkv, -(-Lmax // 32)))
        ref.kv8_append(t.double().numpy(), [0, m], [at], codes, scales)
        want.append((codes, scales))
    host = lambda t: t[0, B - 1:].view(torch.uint8).cpu().numpy()  # noqa: E731
    for got, sc, (codes, scales) in ((k8, ks, want[0]), (v8, vs, want[1])):
        assert np.array_equal(host(got), codes) and np.array_equal(sc[0, B - 1:].double().cpu().numpy(), scales)
        assert int(torch.count_nonzero(got.view(torch.uint8)[0, :B - 1].view(torch.int64))) == 0
    q, kt, vt = torch.zeros(B, n, Hkv, D).bfloat16(), torch.zeros(B, n, Hkv, D).bfloat16(), torch.zeros(B, n, Hkv, D).bfloat16()
    for i, t in enumerate((q, kt, vt)):
        t[B - 1:] = _bf16((1, n, Hkv, D), 3 + i)
    parent = np.tile([-1, 0, 0], (B, 1))
    out = E.eagle_tree_attn_kv8(q.cuda(), k8[0], v8[0], ks[0], vs[0], kt.cuda(), vt.cuda(), _dev(kv_len), _dev(parent), dev_status=st)
    torch.cuda.synchronize()
    o, tol = ref.tree_attn_kv8_tight(q[B - 1:], *want[0], *want[1], kt[B - 1:], vt[B - 1:], [at + m], parent[:1], D ** -0.5)
    assert ((out[B - 1:].double().cpu() - o).abs() <= tol).all() and int(torch.count_nonzero(out[:B - 1])) == 0
    acc, path = np.full(B, -1), np.zeros((B, depth + 1))
    acc[B - 1], path[B - 1, 1] = 1, 2
    new = E.eagle_kv8_commit(kt[None].cuda(), vt[None].cuda(), k8, v8, ks, vs, _dev(kv_len), _dev(path), _dev(acc), depth, dev_status=st)
    for t, got, (codes, scales) in ((kt, k8, want[0]), (vt, v8, want[1])):
        ref.kv8_commit(t[None, B - 1:].double().numpy(), [at + m], path[B - 1:], [1], codes[None], scales[None])
        assert np.array_equal(host(got), codes)
    assert int(st.item()) == 0 and new.tolist() == [0] * (B - 1) + [at + m + 2]


def test_token_rows_spread_over_more_than_32_bits():
    """q, k and v as columns of rows of 2^21 elements, 2100 of them: the last tokens lie beyond 2^32."""
    _room(24)
    E = _E()
    T, W, Hq, Hkv = 2100, 2 ** 21, 4, 2
    wide = torch.empty(T, W // D, D, dtype=torch.bfloat16, device="cuda")
    assert wide.numel() > 2 ** 32
    q, k, v = wide[:, :Hq], wide[:, 5000:5000 + Hkv], wide[:, -Hkv:]
    parts = [_bf16((T, h, D), s) for h, s in ((Hq, 11), (Hkv, 12), (Hkv, 13))]
    for view, x in zip((q, k, v), parts):
        view.copy_(x.cuda())
    lens, st = [1999, 101], torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = _dev([0, 1999, T])
    out, lse = E.eagle_prompt_attn(q, k, v, cu, return_lse=True, dev_status=st)
    k8, v8, ks, vs = (t[0] for t in E.kv8_cache(1, 2, Hkv, 2048))
    E.eagle_kv8_append(k, v, cu, _dev([3, 60]), k8, v8, ks, vs, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    o, z, tol = ref.prompt_attn(parts[0][1950:], parts[1], parts[2], [0, 49, 150], [0, 1999, T], D ** -0.5)
    assert ((out[1950:].double().cpu() - o).abs() <= tol).all()
    for t, got, sc in ((parts[1], k8, ks), (parts[2], v8, vs)):
        codes, scales = np.zeros((2, Hkv, 2048, D), np.uint8), np.ones((2, Hkv, 64))
        ref.kv8_append(t.double().numpy(), [0, lens[0], T], [3, 60], codes, scales)
        assert np.array_equal(got.view(torch.uint8).cpu().numpy(), codes)
