"""GPU parity of the 8-bit cache's calls with the 64-bit forms of oracle/prompt_kv8.py.

eagle_kv8_append and eagle_kv8_commit are compared bit for bit (codes, scales, and every byte
they must not touch); eagle_tree_attn_kv8 to the bound derived there, per output element.
"""
import numpy as np
import pytest
import torch

import workloads as W
from oracle import prompt_kv8 as ref

pytestmark = pytest.mark.gpu
D = 128


def _E():
    import eagle_tree_speculative_gb300 as E
    return E


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _bf16(shape, seed, gain=0.5):
    g = _gen(seed)
    return (torch.randn(shape, generator=g) * torch.exp(gain * torch.randn(shape[-1], generator=g))).bfloat16()


def _dev(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x)).to(dtype).cuda().contiguous()


def _random_cache(lead, Lmax, seed, spread=3):
    """Random codes (NaN codes left out) and powers of two around 1/64."""
    g = _gen(seed)
    codes = torch.randint(0, 256, (*lead, Lmax, D), generator=g, dtype=torch.int32)
    codes = torch.where((codes & 0x7F) == 0x7F, codes - 1, codes).to(torch.uint8).numpy()
    nb = -(-Lmax // ref.KV8_BLOCK)
    scales = torch.exp2(torch.randint(-6 - spread, -6 + spread + 1, (*lead, nb), generator=g).double()).numpy()
    return codes, scales


def _put(codes, scales):
    return (torch.from_numpy(codes.copy()).cuda().view(torch.float8_e4m3fn),
            torch.from_numpy(scales).float().cuda())


def _same(dev_codes, dev_scales, codes, scales):
    got = dev_codes.view(torch.uint8).cpu().numpy()
    assert np.array_equal(dev_scales.double().cpu().numpy(), scales), "scales"
    bad = got != codes
    assert not bad.any(), f"{int(bad.sum())} codes differ, first at {tuple(int(i[0]) for i in np.nonzero(bad))}"


# ---------------------------------------------------------------- append
def _append(x, y, lens, pos, Hkv, Lmax, seed, k_dev=None, v_dev=None, status=0):
    E = _E()
    B = len(lens)
    kc, ks = _random_cache((B, Hkv), Lmax, seed)
    vc, vs = _random_cache((B, Hkv), Lmax, seed + 1)
    k8, kd = _put(kc, ks)
    v8, vd = _put(vc, vs)
    cu = [0] + list(np.cumsum(lens))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    E.eagle_kv8_append(x.cuda() if k_dev is None else k_dev, y.cuda() if v_dev is None else v_dev, _dev(cu),
                       _dev(pos), k8, v8, kd, vd, dev_status=st)
    torch.cuda.synchronize()
    ref.kv8_append(x.double().numpy(), cu, pos, kc, ks)
    ref.kv8_append(y.double().numpy(), cu, pos, vc, vs)
    _same(k8, kd, kc, ks)
    _same(v8, vd, vc, vs)
    assert int(st.item()) == status


@pytest.mark.parametrize("m", [1, 2, 31, 32, 33, 64, 65, 100])
@pytest.mark.parametrize("pos", [0, 1, 31, 32, 40, 63])
def test_append_every_way_into_a_block(m, pos):
    x, y = _bf16((m, 2, D), 100 * m + pos), _bf16((m, 2, D), 100 * m + pos + 7)
    _append(x, y, [m], [pos], 2, pos + m + (m % 5), m + pos)


@pytest.mark.parametrize("size", [2.0 ** -70, 2.0 ** -20, 1.0, 2.0 ** 30, 2.0 ** 119])
def test_append_magnitudes(size):
    """Far smaller and far larger rows than the block holds: the old codes stay, or are
    rounded again to the new scale (most of them to subnormals or zero)."""
    x = (_bf16((20, 3, D), 5).double() * size).bfloat16()
    y = torch.zeros(20, 3, D).bfloat16()
    _append(x, y, [20], [17], 3, 64, 6)


def test_append_scale_borders():
    """amax at 448 * 2^e, one bf16 step above and below, and ties of the e4m3 rounding."""
    rows = torch.zeros(7 * 32, 1, D)
    for i, top in enumerate([448.0, 450.0, 446.0, 7.0, 7.03125, 2.0 ** -56 * 448, 0.0]):
        rows[32 * i:32 * (i + 1)] = torch.linspace(-1, 1, D) * top
        rows[32 * i, 0, 5] = top
        rows[32 * i + 1, 0, :8] = torch.tensor([17.0, 19.0, 21.0, 23.0, -17.0, 0.0009765625, 0.0029296875, -0.0]) * top / 448
    x = rows.bfloat16()
    _append(x, -x, [7 * 32], [0], 1, 7 * 32, 8)


def test_append_ragged_batch_and_strided_tokens():
    """More sequences than lanes, empty ones among them, from a fused projection's slice."""
    rng = np.random.default_rng(4)
    lens = [int(v) for v in rng.integers(0, 50, 70)]
    lens[0] = lens[33] = lens[69] = 0
    pos = [int(v) for v in rng.integers(0, 60, 70)]
    Hkv, T = 3, sum(lens)
    qkv = _bf16((T, 4 + 2 * Hkv, D), 9).cuda()
    k, v = qkv[:, 4:4 + Hkv], qkv[:, 4 + Hkv:]
    _append(k.cpu(), v.cpu(), lens, pos, Hkv, 120, 10, k_dev=k, v_dev=v)


def test_append_non_finite_elements():
    """Infinities become +-448 codes, NaN the NaN code; the finite ones set the scale."""
    x, y = _bf16((40, 2, D), 11), _bf16((40, 2, D), 12)
    x[3, 0, 7], x[3, 1, 9], x[39, 1, 0] = float("inf"), float("-inf"), float("nan")
    y[20] = float("inf")
    _append(x, y, [40], [5], 2, 64, 13, status=_E().EAGLE_DEV_NONFINITE)


@pytest.mark.parametrize("cu,pos,whole", [([0, 4, 2, 9], [0, 0, 0], True), ([0, 4, 6, 10], [0, 0, 0], True),
                                          ([-1, 4, 6, 9], [0, 0, 0], True), ([0, 4, 6, 9], [-1, 0, 0], False),
                                          ([0, 4, 6, 9], [61, 0, 0], False)])
def test_append_bad_lengths(cu, pos, whole):
    """Bad offsets write nothing; a sequence that would leave its cache is skipped alone."""
    E = _E()
    kc, ks = _random_cache((3, 1), 64, 14)
    k8, kd = _put(kc, ks)
    v8, vd = _put(kc, ks)
    x = _bf16((9, 1, D), 15)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    E.eagle_kv8_append(x.cuda(), x.cuda(), _dev(cu), _dev(pos), k8, v8, kd, vd, dev_status=st)
    torch.cuda.synchronize()
    if not whole:
        for b in (1, 2):
            ref.write_rows(x[cu[b]:cu[b + 1], 0].double().numpy(), pos[b], kc[b, 0], ks[b, 0])
    _same(k8, kd, kc, ks)
    _same(v8, vd, kc, ks)
    assert int(st.item()) == E.EAGLE_DEV_CAPACITY


# ---------------------------------------------------------------- commit
@pytest.mark.parametrize("B,layers,Hkv,n,depth", [(1, 3, 2, 1, 0), (5, 2, 3, 20, 6), (3, 1, 8, 64, 63), (40, 2, 1, 30, 40)])
def test_commit_paths(B, layers, Hkv, n, depth):
    E = _E()
    rng = np.random.default_rng(B + n)
    depth_max = depth
    acc = [int(rng.integers(0, min(depth, n - 1) + 1)) for _ in range(B)]
    acc[-1] = min(depth, n - 1)
    if B > 2:
        acc[1] = -1
    path = np.full((B, depth_max + 1), -1, np.int32)
    for b, a in enumerate(acc):
        if a >= 0:
            path[b, :a + 1] = [0] + sorted(rng.choice(np.arange(1, n), a, replace=False))
    L = [int(v) for v in rng.integers(0, 70, B)]
    L[0] = 32
    Lmax = max(L) + 65
    kc, ks = _random_cache((layers, B, Hkv), Lmax, 21)
    vc, vs = _random_cache((layers, B, Hkv), Lmax, 22)
    k8, kd = _put(kc, ks)
    v8, vd = _put(vc, vs)
    x, y = _bf16((layers, B, n, Hkv, D), 23), _bf16((layers, B, n, Hkv, D), 24)
    kv_len, out_len = _dev(L), torch.full((B,), -9, dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    E.eagle_kv8_commit(x.cuda(), y.cuda(), k8, v8, kd, vd, kv_len, _dev(path), _dev(acc), depth_max,
                       kv_len_out=out_len, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    ref.kv8_commit(x.double().numpy(), L, path, acc, kc, ks)
    ref.kv8_commit(y.double().numpy(), L, path, acc, vc, vs)
    _same(k8, kd, kc, ks)
    _same(v8, vd, vc, vs)
    assert kv_len.tolist() == L and out_len.tolist() == [l + a + 1 for l, a in zip(L, acc)]
    # in place: the same again from the same lengths leaves the cache and advances kv_len
    E.eagle_kv8_commit(x.cuda(), y.cuda(), k8, v8, kd, vd, kv_len, _dev(path), _dev(acc), depth_max)
    assert kv_len.tolist() == out_len.tolist()
    _same(k8, kd, kc, ks)


@pytest.mark.parametrize("what", ["depth", "room", "negative", "start", "order", "node"])
def test_commit_bad_sequences_are_skipped_alone(what):
    E = _E()
    n, Dp, Lmax = 6, 3, 64
    L, acc = [10, 20], [2, 1]
    path = np.array([[0, 2, 4, -1], [0, 3, -1, -1]], np.int32)
    bit = E.EAGLE_DEV_BAD_TREE
    if what == "depth":
        acc[0], bit = 4, E.EAGLE_DEV_CAPACITY
    elif what == "room":
        L[0], bit = 62, E.EAGLE_DEV_CAPACITY
    elif what == "negative":
        L[0], bit = -1, E.EAGLE_DEV_CAPACITY
    elif what == "start":
        path[0, 0] = 1
    elif what == "order":
        path[0, 2] = 2
    else:
        path[0, 2] = 6
    kc, ks = _random_cache((1, 2, 1), Lmax, 31)
    k8, kd = _put(kc, ks)
    v8, vd = _put(kc, ks)
    x = _bf16((1, 2, n, 1, D), 32)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    new = E.eagle_kv8_commit(x.cuda(), x.cuda(), k8, v8, kd, vd, _dev(L), _dev(path), _dev(acc), Dp, dev_status=st)
    torch.cuda.synchronize()
    ref.write_rows(x[0, 1, [0, 3], 0].double().numpy(), 20, kc[0, 1, 0], ks[0, 1, 0])
    _same(k8, kd, kc, ks)
    _same(v8, vd, kc, ks)
    assert int(st.item()) == bit and new.tolist() == [L[0], 22]


# ---------------------------------------------------------------- tree attention
def _quantised(lead, L, Lmax, seed, gain=0.5, junk=True):
    """A cache of rows as the calls write them; rows from L[b] on hold NaN codes."""
    g = _gen(seed)
    ch = torch.exp(gain * torch.randn(D, generator=g))
    x = (torch.randn(*lead, Lmax, D, generator=g) * ch).bfloat16().double().numpy()
    codes = np.full((*lead, Lmax, D), 0x7F, np.uint8)
    scales = np.full((*lead, -(-Lmax // ref.KV8_BLOCK)), np.nan)
    for b in range(lead[0]):
        for h in range(lead[1]):
            ref.write_rows(x[b, h, :L[b]], 0, codes[b, h], scales[b, h])
            if not junk:
                codes[b, h, L[b]:] = 0
    return codes, scales


def _tree_check(B, n, Hq, Hkv, L, Lmax, seed, parent=None, scale=None, cache=None, gain=0.5):
    E = _E()
    if parent is None:
        parent = np.stack([W.random_tree(n, 12, seed, b) if n > 1 else np.array([-1], np.int32) for b in range(B)])
    q, kt, vt = _bf16((B, n, Hq, D), seed, gain), _bf16((B, n, Hkv, D), seed + 1), _bf16((B, n, Hkv, D), seed + 2)
    (kc, ks), (vc, vs) = cache or (_quantised((B, Hkv), L, Lmax, seed + 3), _quantised((B, Hkv), L, Lmax, seed + 4))
    k8, kd = _put(kc, ks)
    v8, vd = _put(vc, vs)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = E.eagle_tree_attn_kv8(q.cuda(), k8, v8, kd, vd, kt.cuda(), vt.cuda(), _dev(L), _dev(parent), scale=scale,
                                dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    o, tol = ref.tree_attn_kv8(q, kc, ks, vc, vs, kt, vt, L, parent, scale or D ** -0.5)
    worst = ((out.double().cpu() - o).abs() / (tol + 1e-30)).max()
    assert worst <= 1.0, f"output off by {float(worst):.3g} times the bound"
    return float(worst)


@pytest.mark.parametrize("L", [0, 1, 31, 32, 33, 127, 128, 129, 160, 255, 256, 257, 300, 384, 500, 1000])
@pytest.mark.parametrize("n", [1, 5])
def test_tree_attention_every_length(L, n):
    _tree_check(1, n, 4, 2, [L], max(L, 1) + L % 7, 10 * L + n)


@pytest.mark.parametrize("Hq,Hkv,n", [(1, 1, 1), (1, 1, 64), (2, 2, 60), (6, 2, 43), (5, 1, 26), (7, 1, 64), (8, 1, 64),
                                      (8, 2, 32), (8, 2, 33), (16, 1, 60), (3, 1, 2), (32, 1, 1), (130, 1, 1), (64, 1, 5)])
def test_tree_attention_heads_and_trees(Hq, Hkv, n):
    _tree_check(2, n, Hq, Hkv, [300, 77], 320, 1000 + Hq + n)


def test_tree_attention_ragged_batch():
    L = [0, 1, 700, 64, 129, 31, 2000, 513]
    _tree_check(8, 11, 8, 2, L, 2048, 41)


def test_tree_attention_decode_many_sequences():
    L = [int(v) for v in np.random.default_rng(5).integers(0, 1500, 20)]
    _tree_check(20, 1, 8, 1, L, 1500, 43)


def test_tree_attention_64_node_chain():
    _tree_check(1, 64, 4, 1, [400], 400, 45, parent=W.chain_tree(64)[None])


def test_tree_attention_sharp_and_flat_softmax():
    _tree_check(1, 20, 4, 1, [900], 1000, 47, scale=1.5)
    _tree_check(1, 20, 4, 1, [900], 1000, 48, scale=1e-3)


def test_tree_attention_blocks_of_very_different_scale():
    """Scales from 2^-30 to 2^6 from block to block (and heads): K rows of any size, and V blocks
    whose weight is all of the output or nothing of it."""
    L, Lmax = [700], 704
    kc, ks = _quantised((1, 2), L, Lmax, 51)
    vc, vs = _quantised((1, 2), L, Lmax, 52)
    g = np.random.default_rng(6)
    vs = vs * 2.0 ** g.integers(-30, 7, vs.shape)
    ks = ks * 2.0 ** g.integers(-30, 1, ks.shape)
    _tree_check(1, 9, 4, 2, L, Lmax, 53, cache=((kc, ks), (vc, vs)))


def test_tree_attention_late_large_keys():
    """Each block's keys are larger than the last one's: the running maximum keeps moving."""
    L, Lmax = [1024], 1024
    kc, ks = _quantised((1, 1), L, Lmax, 55)
    ks = ks * 2.0 ** np.floor(np.linspace(-5, 2, ks.shape[-1]))
    _tree_check(1, 30, 4, 1, L, Lmax, 57, cache=((kc, ks), _quantised((1, 1), L, Lmax, 56)))


def test_tree_attention_queries_of_any_size():
    """Queries from 2^-60 to 2^20 and an all-zero one: digits are taken per row."""
    E = _E()
    n = 8
    L = [200]
    cache = _quantised((1, 1), L, 200, 61), _quantised((1, 1), L, 200, 62)
    (kc, ks), (vc, vs) = cache
    q = _bf16((1, n, 2, D), 63)
    for i, e in enumerate([-60, -20, -8, 0, 2, 4, 5]):
        q[0, i] = (q[0, i].double() * 2.0 ** e).bfloat16()
    q[0, 7] = 0
    kt, vt = _bf16((1, n, 1, D), 64), _bf16((1, n, 1, D), 65)
    parent = W.chain_tree(n)[None]
    k8, kd = _put(kc, ks)
    v8, vd = _put(vc, vs)
    out = E.eagle_tree_attn_kv8(q.cuda(), k8, v8, kd, vd, kt.cuda(), vt.cuda(), _dev(L), _dev(parent))
    o, tol = ref.tree_attn_kv8(q, kc, ks, vc, vs, kt, vt, L, parent, D ** -0.5)
    assert ((out.double().cpu() - o).abs() <= tol).all()


def test_tree_attention_bad_sequences_give_zeros():
    E = _E()
    B, n, L, Lmax = 5, 6, [40, 65, -1, 64, 10], 64
    parent = np.stack([W.random_tree(n, 4, 71, b) for b in range(B)])
    parent[0, 3] = 3
    parent[4, 0] = 0
    ok_L = [max(0, min(v, Lmax)) for v in L]
    kc, ks = _quantised((B, 1), ok_L, Lmax, 72, junk=False)
    vc, vs = _quantised((B, 1), ok_L, Lmax, 73, junk=False)
    q, kt, vt = _bf16((B, n, 2, D), 74), _bf16((B, n, 1, D), 75), _bf16((B, n, 1, D), 76)
    k8, kd = _put(kc, ks)
    v8, vd = _put(vc, vs)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = E.eagle_tree_attn_kv8(q.cuda(), k8, v8, kd, vd, kt.cuda(), vt.cuda(), _dev(L), _dev(parent), dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == E.EAGLE_DEV_BAD_TREE | E.EAGLE_DEV_CAPACITY
    assert (out[[0, 1, 2, 4]] == 0).all()
    one = slice(3, 4)
    o, tol = ref.tree_attn_kv8(q[one], kc[one], ks[one], vc[one], vs[one], kt[one], vt[one], L[3:4], parent[one], D ** -0.5)
    assert ((out[one].double().cpu() - o).abs() <= tol).all()


def test_tree_attention_in_a_captured_graph_and_on_a_side_stream():
    """Bit-equal results on a side stream and in a graph replayed after the lengths grew."""
    E = _E()
    B, n, Hq, Hkv, Lmax = 3, 20, 8, 2, 1100
    L = [1000, 300, 0]
    kc, ks = _quantised((B, Hkv), [Lmax] * B, Lmax, 81)
    vc, vs = _quantised((B, Hkv), [Lmax] * B, Lmax, 82)
    k8, kd = _put(kc, ks)
    v8, vd = _put(vc, vs)
    parent = _dev(np.stack([W.random_tree(n, 6, 83, b) for b in range(B)]))
    q, kt, vt = (_bf16((B, n, h, D), s).cuda() for h, s in ((Hq, 84), (Hkv, 85), (Hkv, 86)))
    kv_len = _dev(L)
    ws = [torch.empty(max(1, E.tree_attn_kv8_workspace_size(B, n, Hq, Hkv, D, Lmax)), dtype=torch.uint8, device="cuda")
          for _ in range(2)]
    call = lambda **kw: E.eagle_tree_attn_kv8(q, k8, v8, kd, vd, kt, vt, kv_len, parent, **kw)  # noqa: E731
    first = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    second = call(stream=side)
    side.synchronize()
    assert torch.equal(first, second)
    out = torch.empty_like(first)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out=out, workspace=ws[0])
    for grown in ([1100, 301, 1], [0, 1100, 640]):
        kv_len.copy_(_dev(grown))
        graph.replay()
        want = call(workspace=ws[1])
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_full_size_verify_shape():
    """The B = 64 step's layer (60 nodes, 32/8 heads, 4096 rows): two sequences checked whole."""
    E = _E()
    B, n, Hq, Hkv, L = 64, 60, 32, 8, 4096
    gen = torch.Generator(device="cuda").manual_seed(9)
    mk = lambda *s: torch.randn(*s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    k8, v8, kd, vd = (t[0] for t in E.kv8_cache(1, B, Hkv, L))
    kv = mk(B * L, 2 * Hkv, D)
    cu = _dev(np.arange(B + 1) * L)
    E.eagle_kv8_append(kv[:, :Hkv], kv[:, Hkv:], cu, _dev(np.zeros(B)), k8, v8, kd, vd)
    q, kt, vt = mk(B, n, Hq, D), mk(B, n, Hkv, D), mk(B, n, Hkv, D)
    parent = np.stack([W.random_tree(n, 8, 91, b) for b in range(B)])
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = E.eagle_tree_attn_kv8(q, k8, v8, kd, vd, kt, vt, _dev([L] * B), _dev(parent), dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    host = lambda t, b: t[b:b + 1].cpu()  # noqa: E731
    for b in (0, 61):
        codes = [host(t, b).view(torch.uint8).numpy() for t in (k8, v8)]
        sc = [host(t, b).double().numpy() for t in (kd, vd)]
        o, tol = ref.tree_attn_kv8(host(q, b), codes[0], sc[0], codes[1], sc[1], host(kt, b), host(vt, b), [L],
                                   parent[b:b + 1], D ** -0.5)
        assert ((host(out, b).double() - o).abs() <= tol).all()


# ---------------------------------------------------------------- the calls together
def test_prompt_then_steps():
    """As a serving loop runs them, one layer: a packed prompt through eagle_prompt_attn and
    into the cache, then three steps of tree attention, verify and commit, in one stream.  The
    cache, the lengths and each step's attention equal the 64-bit forms fed with the same
    bf16 rows; the accepted paths come from eagle_verify_accept."""
    E = _E()
    B, n, Hq, Hkv, V, Dp = 3, 12, 8, 2, 64, 4
    lens = [45, 1, 100]
    Lmax = 160
    T = sum(lens)
    cu = [0] + list(np.cumsum(lens))
    q, k, v = _bf16((T, Hq, D), 1), _bf16((T, Hkv, D), 2), _bf16((T, Hkv, D), 3)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache = E.kv8_cache(1, B, Hkv, Lmax)
    k8, v8, kd, vd = cache
    out = E.eagle_prompt_attn(q.cuda(), k.cuda(), v.cuda(), _dev(cu), dev_status=st)
    E.eagle_kv8_append(k.cuda(), v.cuda(), _dev(cu), _dev([0] * B), k8[0], v8[0], kd[0], vd[0], dev_status=st)
    o, _, tol = ref.prompt_attn(q, k, v, cu, cu, D ** -0.5)
    assert ((out.double().cpu() - o).abs() <= tol).all()
    codes = [np.zeros((1, B, Hkv, Lmax, D), np.uint8) for _ in range(2)]
    scales = [np.ones((1, B, Hkv, -(-Lmax // 32))) for _ in range(2)]
    for x, c, s in ((k, codes[0], scales[0]), (v, codes[1], scales[1])):
        ref.kv8_append(x.double().numpy(), cu, [0] * B, c[0], s[0])
    L = list(lens)
    kv_len = _dev(L)
    for step in range(3):
        parent = np.stack([W.random_tree(n, Dp, 100 + step, b) for b in range(B)])
        tq, tk, tv = _bf16((B, n, Hq, D), 10 + step), _bf16((B, n, Hkv, D), 20 + step), _bf16((B, n, Hkv, D), 30 + step)
        got = E.eagle_tree_attn_kv8(tq.cuda(), k8[0], v8[0], kd[0], vd[0], tk.cuda(), tv.cuda(), kv_len, _dev(parent),
                                    dev_status=st)
        target = W.per_seq_normal(B, (n, V), 2.0, 200 + step, W.TAG_TARGET)
        tokens = np.random.default_rng(step).integers(0, V, (B, n)).astype(np.int32)
        for b in range(B):                           # half of the nodes carry their parent's greedy token
            for i in range(1, n, 2):
                tokens[b, i] = int(np.argmax(target[b, parent[b, i]]))
        acc, path, _ = E.eagle_verify_accept(torch.from_numpy(target).cuda(), None, _dev(tokens), _dev(parent), Dp, 0.0,
                                             5, dev_status=st)
        E.eagle_kv8_commit(tk[None].cuda(), tv[None].cuda(), k8, v8, kd, vd, kv_len, path, acc, Dp, dev_status=st)
        torch.cuda.synchronize()
        o, tol = ref.tree_attn_kv8(tq, codes[0][0], scales[0][0], codes[1][0], scales[1][0], tk, tv, L, parent, D ** -0.5)
        assert ((got.double().cpu() - o).abs() <= tol).all(), step
        acc, path = acc.cpu().numpy(), path.cpu().numpy()
        assert (acc >= 0).all()
        for x, c, s in ((tk, codes[0], scales[0]), (tv, codes[1], scales[1])):
            ref.kv8_commit(x[None].double().numpy(), L, path, acc, c, s)
        L = [l + int(a) + 1 for l, a in zip(L, acc)]
        assert kv_len.tolist() == L
        _same(k8, kd, codes[0], scales[0])
        _same(v8, vd, codes[1], scales[1])
    assert int(st.item()) == 0 and max(L) > max(lens)


# ---------------------------------------------------------------- further calls
@pytest.mark.parametrize("where", [(0,), (31,), (32, 33), (70, 3, 40)])
@pytest.mark.parametrize("value", ["inf", "nan"])
def test_append_non_finite_rows_anywhere_in_a_block(where, value):
    """A whole row without a finite element beside others that set the scale; a block of nothing else."""
    x, y = _bf16((75, 1, D), 111), _bf16((75, 1, D), 112)
    for t in where:
        x[t] = float(value)
    y[5:37, 0, 64:] = float(value)
    _append(x, y, [75], [17], 1, 96, 113, status=_E().EAGLE_DEV_NONFINITE)


@pytest.mark.parametrize("start", [0, 9, 31])
def test_commit_non_finite_elements_of_long_paths(start):
    """Paths longer than the rows a warp holds at once, an infinity and a NaN in them."""
    E = _E()
    n, depth, Lmax = 40, 30, 64
    x = _bf16((2, 1, n, 2, D), 114)
    x[0, 0, 3, 1, 5], x[1, 0, 25, 0, 100] = float("inf"), float("nan")
    path = np.array([[0] + list(range(2, 32))], np.int32)
    kc, ks = _random_cache((2, 1, 2), Lmax, 115)
    k8, kd = _put(kc, ks)
    v8, vd = _put(kc, ks)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    E.eagle_kv8_commit(x.cuda(), x.cuda(), k8, v8, kd, vd, _dev([start]), _dev(path), _dev([depth]), depth, dev_status=st)
    torch.cuda.synchronize()
    ref.kv8_commit(x.double().numpy(), [start], path, [depth], kc, ks)
    _same(k8, kd, kc, ks)
    _same(v8, vd, kc, ks)
    assert int(st.item()) == E.EAGLE_DEV_NONFINITE


def _attention_inputs(B, n, Hq, Hkv, L, Lmax, seed):
    kc, ks = _quantised((B, Hkv), L, Lmax, seed)
    vc, vs = _quantised((B, Hkv), L, Lmax, seed + 1)
    parent = _dev(np.stack([W.random_tree(n, 6, seed, b) if n > 1 else np.array([-1], np.int32) for b in range(B)]))
    q, kt, vt = (_bf16((B, n, h, D), seed + 2 + i).cuda() for i, h in enumerate((Hq, Hkv, Hkv)))
    return (q, *sum(zip(_put(kc, ks), _put(vc, vs)), ()), kt, vt, _dev(L), parent)


def test_tree_attention_on_two_streams_at_once():
    """Calls of different shapes that run at the same time, a workspace each."""
    E = _E()
    shapes = [(3, 20, 8, 2, [1000, 300, 0], 1100), (2, 1, 16, 4, [2000, 77], 2048)]
    args = [_attention_inputs(*s, seed=121 + 10 * i) for i, s in enumerate(shapes)]
    want = [E.eagle_tree_attn_kv8(*a) for a in args]
    streams = [torch.cuda.Stream() for _ in shapes]
    ws = [torch.empty(max(1, E.tree_attn_kv8_workspace_size(*s[:4], D, s[5])), dtype=torch.uint8, device="cuda") for s in shapes]
    outs = [[torch.zeros_like(w) for _ in range(20)] for w in want]
    torch.cuda.synchronize()
    for k in range(20):
        for i, st in enumerate(streams):
            E.eagle_tree_attn_kv8(*args[i], out=outs[i][k], workspace=ws[i], stream=st)
    torch.cuda.synchronize()
    for i, w in enumerate(want):
        assert all(torch.equal(o, w) for o in outs[i])


@pytest.mark.parametrize("B,n,Hq,Hkv,L", [(1, 1, 8, 8, 2000), (2, 3, 4, 2, 5), (1, 1, 1, 1, 0), (16, 30, 8, 2, 700)])
def test_work_queued_behind_the_attention_sees_its_output(B, n, Hq, Hkv, L):
    """A copy right behind the call, with nothing between, and the output cleared before it."""
    E = _E()
    args = _attention_inputs(B, n, Hq, Hkv, [L] * B, 2048, seed=141)
    want = E.eagle_tree_attn_kv8(*args)
    torch.cuda.synchronize()
    out = torch.empty_like(want)
    got = [torch.empty_like(want) for _ in range(50)]
    ws = torch.empty(max(1, E.tree_attn_kv8_workspace_size(B, n, Hq, Hkv, D, 2048)), dtype=torch.uint8, device="cuda")
    for g in got:
        out.fill_(float("nan"))
        E.eagle_tree_attn_kv8(*args, out=out, workspace=ws)
        g.copy_(out)
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)


def test_tree_attention_reports_value_scales_out_of_range():
    """2^44 is the largest V scale; a larger one sets the status bit, in the cache or in the tree."""
    E = _E()
    B, n, Hq, Hkv, L, Lmax = 1, 4, 4, 1, [100], 128
    args = list(_attention_inputs(B, n, Hq, Hkv, L, Lmax, seed=151))
    for block, exp, bit in ((0, 44, 0), (3, 45, E.EAGLE_DEV_NONFINITE), (1, 60, E.EAGLE_DEV_NONFINITE)):
        vd = args[4].clone()
        vd[0, 0, block] = 2.0 ** exp
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        E.eagle_tree_attn_kv8(*args[:4], vd, *args[5:], dev_status=st)
        assert int(st.item()) == bit
    big = args[6].clone()
    big[0, 2, 0, 5] = 2.0 ** 60
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    E.eagle_tree_attn_kv8(*args[:6], big, *args[7:], dev_status=st)
    assert int(st.item()) == E.EAGLE_DEV_NONFINITE


def _leave_nan_in_shared_memory():
    """A prompt of nothing but NaN, on every SM: its tiles stay in shared memory and its products in TMEM."""
    E = _E()
    x = torch.full((400, 8, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    cu = _dev(np.arange(0, 401, 400))
    for _ in range(4):
        E.eagle_prompt_attn(x.repeat(16, 4, 1), x.repeat(16, 1, 1), x.repeat(16, 1, 1), _dev(np.arange(0, 6401, 400)))
    E.eagle_prompt_attn(x, x, x, cu)


@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 16, 17, 30, 40, 63, 64])
@pytest.mark.parametrize("L", [0, 5, 130, 1000])
def test_tree_attention_does_not_read_what_an_earlier_kernel_left(n, L):
    B, Hq, Hkv = 40, 8, 4
    _leave_nan_in_shared_memory()
    _tree_check(B, n, Hq, Hkv, [L] * B, 1024, 161 + n)


@pytest.mark.parametrize("n", [1, 5, 64, 130, 300])
def test_prompt_attention_does_not_read_what_an_earlier_kernel_left(n):
    E = _E()
    B, Hq, Hkv = 50, 6, 2
    q, k, v = _bf16((B * n, Hq, D), 171), _bf16((B * n, Hkv, D), 172), _bf16((B * n, Hkv, D), 173)
    cu = [b * n for b in range(B + 1)]
    _leave_nan_in_shared_memory()
    out = E.eagle_prompt_attn(q.cuda(), k.cuda(), v.cuda(), _dev(cu))
    torch.cuda.synchronize()
    o, _, tol = ref.prompt_attn(q, k, v, cu, cu, D ** -0.5)
    assert ((out.double().cpu() - o).abs() <= tol).all()
