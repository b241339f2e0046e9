"""The paged cache's calls at their edges: offsets past 32 bits, empty batches, graphs, streams, memory that other work
still uses, many slots and pages, what the binding refuses."""
import numpy as np
import pytest
import torch

from oracle import paged as ref

pytestmark = pytest.mark.gpu
D = 128


def _E():
    import eagle_tree_speculative_gb300 as E
    return E


def _dev(x):
    return torch.as_tensor(np.asarray(x)).to(torch.int32).cuda().contiguous()


def _bf16(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).bfloat16()


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _freq():
    return (10000.0 ** -(torch.arange(0, D, 2).double() / D)).float()


def _close(got, want, tol):
    return bool(((got.double().cpu() - want).abs() <= tol).all())


def test_pages_beyond_32_bit_offsets():
    """70 000 pages of 4 heads and 64 rows (2.3 G elements of K, as much of V): the last pages hold a sequence that is
    rotated into, attended, committed and forked, the first ones are not touched."""
    if torch.cuda.mem_get_info()[0] < 30 * 2 ** 30:
        pytest.skip("needs 30 GB")
    E, N, Hkv, Hq, page, n, depth = _E(), 70000, 4, 8, 64, 5, 3
    k = torch.zeros(1, N, Hkv, page, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    assert k.numel() > 2 ** 31
    P = 4
    refs = torch.ones(N, dtype=torch.int32, device="cuda")
    refs[-10:] = 0                                         # whatever else there is, is taken
    table, held, kv_len, st = _dev(np.full((2, P), -1)), _dev([0, 0]), _dev([0, 0]), _status()
    L = 100
    E.eagle_pages_assign(k, v, table, held, refs, kv_len, _dev([L, 0]), dev_status=st)
    assert table.tolist() == [[N - 10, N - 9, -1, -1], [-1] * P]
    x = _bf16((L, (Hq + 2 * Hkv) * D), 1).cuda()
    q, kk, vv = (t.unflatten(1, (-1, D)) for t in x.split([Hq * D, Hkv * D, Hkv * D], 1))
    f = _freq()
    E.eagle_qkv_rope(q, kk, vv, f.cuda(), kv_len, cu=_dev([0, L, L]), k_pages=k[0], v_pages=v[0], page_table=table, dev_status=st)
    kv_len.copy_(_dev([L, 0]))
    rows = lambda t, m: torch.cat([t[0, i, :, :] for i in range(N - 10, N)], 1)[:, :m].transpose(0, 1).cpu()  # noqa: E731
    for t in (0, 63, 64, 99):
        assert _close(rows(k, L)[t], *ref.turned(kk[t].cpu(), None, f, t, 1e-6, False))
    assert torch.equal(rows(v, L), vv.cpu())
    # slot 1 goes on with slot 0, both get a tree
    E.eagle_pages_assign(k, v, table, held, refs, kv_len, _dev([n, n]), src=_dev([0, 0]), dev_status=st)
    assert table[:, :2].tolist() == [[N - 10, N - 9], [N - 10, N - 8]] and kv_len.tolist() == [L, L]
    assert torch.equal(k[0, N - 8, :, :L - 64], k[0, N - 9, :, :L - 64])
    parent = [[-1, 0, 0, 1, 3]] * 2
    x = _bf16((2 * n, (Hq + 2 * Hkv) * D), 2).cuda()
    q, kk, vv = (t.unflatten(1, (-1, D)) for t in x.split([Hq * D, Hkv * D, Hkv * D], 1))
    qr, _ = E.eagle_qkv_rope(q, kk, vv, f.cuda(), kv_len, parent=_dev(parent), k_pages=k[0], v_pages=v[0], page_table=table, dev_status=st)
    out = E.eagle_tree_attn_paged(qr.view(2, n, Hq, D), k[0], v[0], table, kv_len, _dev(parent), dev_status=st)
    tail = [t[0, N - 10:].cpu() for t in (k, v)]           # the same pages as a small pool
    small = table.cpu().numpy() - (N - 10)
    assert _close(out, *ref.tree_attn_paged(qr.view(2, n, Hq, D).cpu(), *tail, small, [L, L], parent, D ** -0.5))
    path, acc = [[0, 2, -1, -1], [0, 1, 3, 4]], [1, 3]
    E.eagle_pages_commit(k, v, table, kv_len, _dev(path), _dev(acc), depth, dev_status=st)
    tail = [t[None] for t in tail]
    assert kv_len.tolist() == ref.pages_commit(tail, small, [L, L], path, acc, depth, page, 10)
    assert torch.equal(k[0, N - 10:].cpu(), tail[0][0]) and torch.equal(v[0, N - 10:].cpu(), tail[1][0])
    assert not bool(k[0, :N - 10].any()) and not bool(v[0, :N - 10].any()) and int(st.item()) == 0


def test_empty_batches():
    E = _E()
    kp, vp, table, held, refs = E.paged_cache(2, 5, 2, 16, 0, 3)
    none, f = _dev([]), _freq().cuda()
    assert table.shape == (0, 3)
    E.eagle_pages_assign(kp, vp, table, held, refs, none, none)
    assert E.eagle_pages_commit(kp, vp, table, none, _dev(np.zeros((0, 4))), none, 3) is none
    q, k = torch.empty(0, 4, D, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 2, D, dtype=torch.bfloat16, device="cuda")
    a, b = E.eagle_qkv_rope(q, k, k, f, none, cu=_dev([0]), k_pages=kp[0], v_pages=vp[0], page_table=table)
    assert a.shape == q.shape and b is None
    a, b = E.eagle_qkv_rope(q, k, None, f, _dev([3, 4]), cu=_dev([0, 0, 0]))
    assert a.shape == q.shape and b.shape == k.shape
    out = E.eagle_tree_attn_paged(q.view(0, 1, 4, D), kp[0], vp[0], table, none, _dev(np.zeros((0, 1))))
    assert out.shape == (0, 1, 4, D)
    kp, vp, table, held, refs = E.paged_cache(0, 9, 2, 16, 2, 3)         # no layers: numbers alone
    E.eagle_pages_assign(kp, vp, table, held, refs, _dev([0, 0]), _dev([20, 1]))
    assert table.tolist() == [[0, 1, -1], [2, -1, -1]]
    torch.cuda.synchronize()


@pytest.mark.parametrize("B,N,P,page", [(1100, 9000, 4, 16), (3, 300000, 5, 64), (2, 9000, 4000, 16)])
def test_assign_many_slots_and_pages(B, N, P, page):
    """More slots than warps and lanes, long refs, wide tables."""
    E, rng = _E(), np.random.default_rng(N)
    kp, vp, table, held, refs = E.paged_cache(0, N, 1, page, B, P)
    lens = [0] * B
    want = [[-1] * P] * B, [0] * B, [0] * N, lens
    kv_len, st = _dev(lens), _status()
    for step in range(4):
        src = None if step == 0 else [int(x) for x in rng.integers(-1, B, B)]
        now = [want[3][b] if src is None else (want[3][src[b]] if src[b] >= 0 else 0) for b in range(B)]
        grow = [int(rng.integers(0, min(P * page - x, 4 * page if B > 9 else P * page) + 1)) for x in now]
        got = ref.pages_assign(*want, grow, src, page)
        E.eagle_pages_assign(kp, vp, table, held, refs, kv_len, _dev(grow), src=None if src is None else _dev(src), dev_status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == (0x10 if got is None else 0)
        if got is None:
            st.zero_()
            continue
        want = [list(x) for x in got[:4]]
        assert table.tolist() == want[0] and held.tolist() == want[1] and refs.tolist() == want[2] and kv_len.tolist() == want[3]
        want[3] = [min(P * page, x + g // 2) for x, g in zip(want[3], grow)]
        kv_len.copy_(_dev(want[3]))


def _step_inputs(seed, B=6, n=7, Hq=8, Hkv=2, page=16, layers=3, depth=3):
    rng = np.random.default_rng(seed)
    L = [int(x) for x in rng.integers(0, 90, B)]
    parent = [[-1] + [int(rng.integers(0, i)) for i in range(1, n)] for _ in range(B)]
    acc = [int(rng.integers(0, depth + 1)) for _ in range(B)]
    path = [[0] + sorted(int(x) for x in rng.choice(np.arange(1, n), a, replace=False)) + [-1] * (depth - a) for a in acc]
    x = _bf16((B * n, (Hq + 2 * Hkv) * D), seed).cuda()
    q, k, v = (t.unflatten(1, (-1, D)) for t in x.split([Hq * D, Hkv * D, Hkv * D], 1))
    return dict(B=B, n=n, Hq=Hq, L=L, parent=_dev(parent), acc=_dev(acc), path=_dev(path), depth=depth, q=q, k=k, v=v, f=_freq().cuda(),
                kp=_bf16((layers, 90, Hkv, page, D), seed + 1).cuda(), vp=_bf16((layers, 90, Hkv, page, D), seed + 2).cuda(),
                src=_dev(rng.integers(0, B, B)), page=page)


def _cache(s):
    """The cache's numbers with L rows in each slot, and its pages."""
    E = _E()
    _, _, table, held, refs = E.paged_cache(0, 90, 1, s["page"], s["B"], 7)
    kv_len = _dev([0] * s["B"])
    c = dict(kp=s["kp"].clone(), vp=s["vp"].clone(), table=table, held=held, refs=refs, len=kv_len)
    E.eagle_pages_assign(c["kp"], c["vp"], table, held, refs, kv_len, _dev(s["L"]))
    kv_len.copy_(_dev(s["L"]))
    return c


def _step(s, c, stream=None, dev_status=None):
    """What a server does in a step: fork, rotate into the pages, attend, commit."""
    E, kw = _E(), dict(stream=stream, dev_status=dev_status)
    E.eagle_pages_assign(c["kp"], c["vp"], c["table"], c["held"], c["refs"], c["len"], s["grow"], src=s["src"], **kw)
    outs = []
    for l in range(len(c["kp"])):
        q, _ = E.eagle_qkv_rope(s["q"], s["k"], s["v"], s["f"], c["len"], parent=s["parent"], k_pages=c["kp"][l], v_pages=c["vp"][l],
                                page_table=c["table"], **kw)
        outs.append(E.eagle_tree_attn_paged(q.view(s["B"], s["n"], s["Hq"], D), c["kp"][l], c["vp"][l], c["table"], c["len"], s["parent"], **kw))
    E.eagle_pages_commit(c["kp"], c["vp"], c["table"], c["len"], s["path"], s["acc"], s["depth"], **kw)
    return outs


def test_a_captured_step_replays_like_eager_ones():
    """A whole step in one graph; every replay goes on where the last one left the cache."""
    s = _step_inputs(1)
    s["grow"] = _dev([s["n"]] * s["B"])
    s["src"] = _dev([0, 0, 2, 2, 4, 4])
    eager, mine = _cache(s), _cache(s)
    st = _status()
    want = []
    for _ in range(3):
        want.append([o.clone() for o in _step(s, eager)] + [eager[x].clone() for x in ("table", "held", "refs", "len", "kp", "vp")])
    torch.cuda.synchronize()
    keep = {k: v.clone() for k, v in mine.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = _step(s, mine, dev_status=st)
    for k, v in keep.items():
        mine[k].copy_(v)
    for w in want:
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs + [mine[x] for x in ("table", "held", "refs", "len", "kp", "vp")], w):
            assert torch.equal(a, b)
    assert int(st.item()) == 0


def test_steps_on_two_streams_at_once():
    """Two caches, two streams, each call's scratch from its own stream's pool, while the current stream is busy with
    memory that it has just given back."""
    ins = [_step_inputs(i, B=4 + i) for i in (2, 3)]
    for s in ins:
        s["grow"] = _dev([s["n"]] * s["B"])
    want = []
    for s in ins:
        c = _cache(s)
        want.append(_step(s, c) + [c[x] for x in ("table", "held", "refs", "len", "kp", "vp")])
    caches = [_cache(s) for s in ins]
    streams = [torch.cuda.Stream() for _ in ins]
    torch.cuda.synchronize()
    junk = torch.full((1 << 24,), 3.0, device="cuda")
    for _ in range(20):
        junk = junk * 1.0 + 1.0                            # frees and takes memory of the current stream
    got = [_step(s, c, stream=st) + [c[x] for x in ("table", "held", "refs", "len", "kp", "vp")] for s, c, st in zip(ins, caches, streams)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_a_caller_s_workspace():
    E = _E()
    s = _step_inputs(4)
    c = _cache(s)
    s["grow"] = _dev([s["n"]] * s["B"])
    B, P = c["table"].shape
    ws = torch.full((E.pages_workspace_size(B, 90, P),), 255, dtype=torch.uint8, device="cuda")
    args = (c["kp"], c["vp"], c["table"], c["held"], c["refs"], c["len"], s["grow"])
    E.eagle_pages_assign(*args, workspace=ws)
    with pytest.raises(E.EagleError) as e:
        E.eagle_pages_assign(*args, workspace=ws[:64])
    assert e.value.code == 3
    q = s["q"].contiguous().view(B, s["n"], s["Hq"], D)
    need = E.tree_attn_paged_workspace_size(B, s["n"], s["Hq"], 2, D, 16, P)
    want = E.eagle_tree_attn_paged(q, c["kp"][0], c["vp"][0], c["table"], c["len"], s["parent"])
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")              # NaN: no initialisation needed
    got = E.eagle_tree_attn_paged(q, c["kp"][0], c["vp"][0], c["table"], c["len"], s["parent"], workspace=ws)
    assert torch.equal(got, want)
    with pytest.raises(E.EagleError):
        E.eagle_tree_attn_paged(q, c["kp"][0], c["vp"][0], c["table"], c["len"], s["parent"], workspace=ws[:need - 16])


@pytest.mark.parametrize("L", [40, 9000])
def test_results_and_scratch_at_odd_multiples_of_16_bytes(L):
    E = _E()
    q, kp, vp = _bf16((2, 3, 8, D), 1).cuda(), _bf16((160, 2, 64, D), 2).cuda(), _bf16((160, 2, 64, D), 3).cuda()
    table, lens = _dev(np.arange(320).reshape(2, 160) % 160), _dev([L, L - 7])
    parent = _dev([[-1, 0, 1]] * 2)
    want = E.eagle_tree_attn_paged(q, kp, vp, table, lens, parent)
    need = E.tree_attn_paged_workspace_size(2, 3, 8, 2, D, 64, 160)
    room, ws = torch.zeros(q.numel() + 8, dtype=torch.bfloat16, device="cuda"), torch.zeros(need + 16, dtype=torch.uint8, device="cuda")
    out = room[8:].view(q.shape)
    E.eagle_tree_attn_paged(q, kp, vp, table, lens, parent, out=out, workspace=ws[16:])
    assert out.data_ptr() % 32 == 16 and torch.equal(out, want) and not bool(room[:8].any())


def test_what_the_binding_refuses():
    E = _E()
    s = _step_inputs(5)
    c = _cache(s)
    B, n, kp, vp, table = s["B"], s["n"], c["kp"], c["vp"], c["table"]
    grow = _dev([1] * B)
    ok = dict(k_pages=kp, v_pages=vp, page_table=table, held=c["held"], refs=c["refs"], kv_len=c["len"], grow=grow)
    for change in (dict(k_pages=kp[0]), dict(v_pages=vp[:2]), dict(v_pages=vp.float()), dict(page_table=table.long()), dict(page_table=table[0]),
                   dict(held=c["held"][:-1]), dict(refs=c["refs"][1:]), dict(kv_len=c["len"].cpu()), dict(grow=grow[None]),
                   dict(src=grow[:2]), dict(grow=None), dict(k_pages=None), dict(page_table=[[1]]), dict(v_pages=vp.transpose(0, 1))):
        with pytest.raises((TypeError, ValueError)):
            E.eagle_pages_assign(**{**ok, **change})
    ok = dict(k_pages=kp, v_pages=vp, page_table=table, kv_len=c["len"], path=s["path"], accept_len=s["acc"], max_depth=s["depth"])
    for change in (dict(max_depth=2), dict(path=s["path"][:2]), dict(accept_len=None), dict(kv_len_out=c["len"][:2]), dict(k_pages=kp[0])):
        with pytest.raises((TypeError, ValueError)):
            E.eagle_pages_commit(**{**ok, **change})
    ok = dict(q=s["q"], k=s["k"], v=s["v"], inv_freq=s["f"], pos=c["len"], parent=s["parent"], k_pages=kp[0], v_pages=vp[0], page_table=table)
    cu = _dev([0] + [B * n] * B)
    for change in (dict(q=s["q"].float()), dict(k=s["k"][1:]), dict(v=s["v"][1:]), dict(v=None), dict(cu=cu), dict(parent=None), dict(parent=s["parent"][:, 1:]),
                   dict(k_pages=kp), dict(k_pages=None), dict(page_table=None), dict(inv_freq=s["f"].double()), dict(pos=c["len"].cpu()),
                   dict(q_weight=s["f"]), dict(k_weight=s["f"].bfloat16()), dict(k_out=s["k"]), dict(q_out=s["q"][:3]),
                   dict(parent=None, cu=cu[1:])):
        with pytest.raises((TypeError, ValueError)):
            E.eagle_qkv_rope(**{**ok, **change})
    with pytest.raises(E.EagleError):
        E.eagle_qkv_rope(**{**ok, "inv_freq": s["f"][:4]})                       # eight dimensions
    q = s["q"].contiguous().view(B, n, s["Hq"], D)
    ok = dict(q=q, k_pages=kp[0], v_pages=vp[0], page_table=table, kv_len=c["len"], parent=s["parent"])
    for change in (dict(q=s["q"]), dict(q=q.transpose(0, 1)), dict(k_pages=kp), dict(v_pages=vp[0, 1:]), dict(page_table=table[1:]),
                   dict(kv_len=c["len"].long()), dict(parent=s["parent"][0]), dict(out=q.float()), dict(page_table=None), dict(k_pages=None)):
        with pytest.raises((TypeError, ValueError)):
            E.eagle_tree_attn_paged(**{**ok, **change})
