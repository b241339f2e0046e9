"""GPU checks of the 8-bit cache's tree attention to the tolerance of its own roundings
(oracle/prompt_kv8.py, tree_attn_kv8_tight), per output element."""
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


def _bf16(shape, seed, gain=0.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * torch.exp(gain * torch.randn(shape[-1], generator=g))).bfloat16()


def _dev(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x)).to(dtype).cuda().contiguous()


def _quantise(x, L):
    """x [B, Hkv, Lmax, D] float64, rows below L[b] written as the calls write them."""
    B, Hkv, Lmax = x.shape[:3]
    codes = np.full(x.shape, 0x7F, np.uint8)
    scales = np.full((B, Hkv, -(-Lmax // ref.KV8_BLOCK)), np.nan)
    for b in range(B):
        for h in range(Hkv):
            ref.write_rows(x[b, h, :L[b]], 0, codes[b, h], scales[b, h])
    return codes, scales


def _cache(B, Hkv, L, Lmax, seed):
    return _quantise(_bf16((B, Hkv, Lmax, D), seed).double().numpy(), L)


def _trees(B, n, seed):
    return np.stack([W.random_tree(n, 12, seed, b) if n > 1 else np.array([-1], np.int32) for b in range(B)])


def _check(q, k, v, kt, vt, L, parent, scale=None):
    """k, v: (codes, scales) of the cache."""
    E = _E()
    put = lambda c: (torch.from_numpy(c[0].copy()).cuda().view(torch.float8_e4m3fn), torch.from_numpy(c[1]).float().cuda())  # noqa: E731
    (k8, ks), (v8, vs) = put(k), put(v)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = E.eagle_tree_attn_kv8(q.cuda(), k8, v8, ks, vs, kt.cuda(), vt.cuda(), _dev(L), _dev(parent), scale=scale, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    o, tol = ref.tree_attn_kv8_tight(q, *k, *v, kt, vt, L, parent, scale or D ** -0.5)
    worst = float(((out.double().cpu() - o).abs() / (tol + 1e-300)).max())
    assert worst <= 1.0, f"output off by {worst:.3g} times the bound"


# ---------------------------------------------------------------- V of very different size
@pytest.mark.parametrize("n,Hq", [(1, 2), (5, 2), (48, 4)])
@pytest.mark.parametrize("at", [0, 500, 998])
@pytest.mark.parametrize("power", [8, 16, 24, 30, 40, 51])
def test_one_large_value_leaves_other_columns_alone(power, at, n, Hq):
    """One element of V is 2^power, all others are around one: in the other 127 columns its block
    holds (nearly) zeros, and the other blocks' weights are the whole output."""
    L = [999]
    x = _bf16((1, 1, 1024, D), 3).double().numpy()
    x[0, 0, at, 17] = 2.0 ** power
    q, kt, vt = _bf16((1, n, Hq, D), 1), _bf16((1, n, 1, D), 4), _bf16((1, n, 1, D), 5)
    _check(q, _cache(1, 1, L, 1024, 2), _quantise(x, L), kt, vt, L, _trees(1, n, 6))


@pytest.mark.parametrize("n,Hq", [(2, 2), (20, 2), (64, 4)])
@pytest.mark.parametrize("power", [12, 30, 50])
def test_one_large_value_of_the_tree_leaves_other_columns_alone(power, n, Hq):
    """The same with the large element in the tree's root, which every node sees."""
    L = [130]
    q, kt, vt = _bf16((1, n, Hq, D), 11), _bf16((1, n, 1, D), 14), _bf16((1, n, 1, D), 15)
    vt[0, 0] = 0
    vt[0, 0, 0, 17] = 2.0 ** power
    _check(q, _cache(1, 1, L, 160, 12), _cache(1, 1, L, 160, 13), kt, vt, L, _trees(1, n, 16))


@pytest.mark.parametrize("n,Hq,Hkv", [(1, 8, 2), (9, 4, 2), (60, 8, 2)])
def test_blocks_of_any_scale(n, Hq, Hkv):
    """V blocks from 2^-60 to 2^44; the ones from 2^-10 on have no value in half of the columns."""
    L, Lmax = [3000, 40], 95 * 32
    codes, _ = _cache(2, Hkv, L, Lmax, 22)
    scales = np.exp2(np.random.default_rng(7).integers(-60, 45, (2, Hkv, 95)).astype(np.float64))
    blocks = codes.reshape(2, Hkv, 95, 32, D)
    blocks[..., :64] = np.where(scales[..., None, None] >= 2.0 ** -10, 0, blocks[..., :64])
    q, kt, vt = _bf16((2, n, Hq, D), 21), _bf16((2, n, Hkv, D), 24), _bf16((2, n, Hkv, D), 25)
    vt[..., :64] = 0
    _check(q, _cache(2, Hkv, L, Lmax, 23), (codes, scales), kt, vt, L, _trees(2, n, 26))


def test_wide_units_beside_ordinary_ones():
    """More units than SMs, heads of a wide spread among others, in every third sequence."""
    B, Hkv, n = 24, 8, 3
    L = [100 + 37 * b for b in range(B)]
    x = _bf16((B, Hkv, 1000, D), 33).double().numpy()
    x[::3, ::2, 70, 5] = 2.0 ** 33
    x[1, 3, 40:70] *= 2.0 ** -30
    q, kt, vt = _bf16((B, n, 16, D), 31), _bf16((B, n, Hkv, D), 34), _bf16((B, n, Hkv, D), 35)
    vt[5, 1] = 0
    vt[6, 2] *= 2.0 ** -40
    _check(q, _cache(B, Hkv, L, 1000, 32), _quantise(x, L), kt, vt, L, _trees(B, n, 36))


@pytest.mark.parametrize("Hq,Hkv,n", [(6, 2, 43), (8, 1, 64), (5, 1, 26), (130, 1, 1), (2, 2, 60), (1, 1, 1)])
def test_wide_units_of_every_shape(Hq, Hkv, n):
    """Rows that end inside a tile, one and two pairs of row tiles, one row."""
    L = [300, 0, 61]
    x = _bf16((3, Hkv, 320, D), 73).double().numpy()
    x[:, :, 50, 9] = 2.0 ** 28
    q, kt, vt = _bf16((3, n, Hq, D), 71), _bf16((3, n, Hkv, D), 74), _bf16((3, n, Hkv, D), 75)
    vt[1, -1] *= 2.0 ** -20
    _check(q, _cache(3, Hkv, L, 320, 72), _quantise(x, L), kt, vt, L, _trees(3, n, 76))


def test_a_replayed_graph_follows_the_spread():
    """The same captured call on a narrow cache, a wide one and the narrow one again equals eager calls."""
    E = _E()
    B, n, Hq, Hkv, L = 3, 7, 8, 2, [500, 300, 64]
    x = _bf16((B, Hkv, 512, D), 83).double().numpy()
    narrow = _quantise(x, L)
    x[1, 0, 100, 3] = 2.0 ** 30
    wide = _quantise(x, L)
    k = _cache(B, Hkv, L, 512, 82)
    put = lambda c: (torch.from_numpy(c[0].copy()).cuda().view(torch.float8_e4m3fn), torch.from_numpy(c[1]).float().cuda())  # noqa: E731
    (k8, ks), (v8, vs) = put(k), put(narrow)
    q, kt, vt = _bf16((B, n, Hq, D), 81).cuda(), _bf16((B, n, Hkv, D), 84).cuda(), _bf16((B, n, Hkv, D), 85).cuda()
    args = (q, k8, v8, ks, vs, kt, vt, _dev(L), _dev(_trees(B, n, 86)))
    ws = [torch.empty(max(1, E.tree_attn_kv8_workspace_size(B, n, Hq, Hkv, D, 512)), dtype=torch.uint8, device="cuda") for _ in range(2)]
    out = torch.empty_like(q)
    E.eagle_tree_attn_kv8(*args, out=out, workspace=ws[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        E.eagle_tree_attn_kv8(*args, out=out, workspace=ws[0])
    got = []
    for c in (narrow, wide, narrow):
        new = put(c)
        v8.view(torch.uint8).copy_(new[0].view(torch.uint8))
        vs.copy_(new[1])
        graph.replay()
        want = E.eagle_tree_attn_kv8(*args, workspace=ws[1])
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        got.append(out.clone())
    assert torch.equal(got[0], got[2]) and not torch.equal(got[0], got[1])


# ---------------------------------------------------------------- ordinary rows
def _plain_check(B, n, Hq, Hkv, L, Lmax, seed, scale=None):
    q, kt, vt = _bf16((B, n, Hq, D), seed), _bf16((B, n, Hkv, D), seed + 1), _bf16((B, n, Hkv, D), seed + 2)
    _check(q, _cache(B, Hkv, L, Lmax, seed + 3), _cache(B, Hkv, L, Lmax, seed + 4), kt, vt, L, _trees(B, n, seed), scale)


@pytest.mark.parametrize("L", [0, 1, 33, 128, 129, 300, 1000])
@pytest.mark.parametrize("n,Hq,Hkv", [(1, 4, 2), (17, 6, 2), (64, 8, 1)])
def test_every_length(L, n, Hq, Hkv):
    _plain_check(1, n, Hq, Hkv, [L], max(L, 1) + L % 5, 100 + L + n)


def test_ragged_batch():
    L = [0, 1, 700, 64, 129, 31, 2000, 513]
    _plain_check(8, 11, 8, 2, L, 2048, 141)


@pytest.mark.parametrize("scale", [1.0, 1e-3])
def test_sharp_and_flat_softmax(scale):
    _plain_check(1, 20, 4, 1, [900], 1000, 147, scale)


@pytest.mark.parametrize("n,Hq", [(1, 1), (1, 8), (30, 4)])
def test_one_long_sequence_of_one_head(n, Hq):
    """30 000 rows of one kv head: more parts of a unit than a warp has lanes to merge."""
    _plain_check(1, n, Hq, 1, [30000], 30016, 151)


def cancelling_rows(seed):
    """Two cache rows whose values cancel but for the weights' difference, for 64 nodes whose own
    values are zero: what is left of an output is the weights' rounding errors."""
    n, Hq = 64, 4
    q, kt = _bf16((1, n, Hq, D), seed) * 0.02, _bf16((1, n, 1, D), seed + 1) * 0.02
    k = _cache(1, 1, [2], 32, seed + 2)
    a = torch.randint(8, 16, (D,), generator=torch.Generator().manual_seed(seed + 3)).double().numpy() / 8
    x = np.zeros((1, 1, 32, D))
    x[0, 0, 0], x[0, 0, 1] = a, -a
    return q, k, _quantise(x, [2]), kt, torch.zeros(1, n, 1, D).bfloat16(), [2], W.random_tree(n, 12, seed, 0)[None]


@pytest.mark.parametrize("seed", [161, 171, 181])
def test_weights_keep_eleven_bits(seed):
    _check(*cancelling_rows(seed))


@pytest.mark.parametrize("B,n,Hq,Hkv,L", [(3, 1, 2, 1, 20), (4, 5, 8, 2, 300), (40, 9, 8, 8, 200), (400, 1, 8, 8, 40)])
def test_a_wide_spread_leaves_the_other_sequences_and_heads_alone(B, n, Hq, Hkv, L):
    """Bit-equal outputs of every other (sequence, head), whether or not one has a wide spread."""
    E = _E()
    g = torch.Generator(device="cuda").manual_seed(91)
    mk = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    k8, v8, ks, vs = (t[0] for t in E.kv8_cache(1, B, Hkv, L))
    rows = mk(B * L, 2 * Hkv, D)
    E.eagle_kv8_append(rows[:, :Hkv], rows[:, Hkv:], _dev(np.arange(B + 1) * L), _dev(np.zeros(B)), k8, v8, ks, vs)
    args = lambda scales, tree: (q, k8, v8, ks, scales, kt, tree, _dev([L] * B), _dev(_trees(B, n, 96)))  # noqa: E731
    q, kt, vt = mk(B, n, Hq, D), mk(B, n, Hkv, D), mk(B, n, Hkv, D)
    want = E.eagle_tree_attn_kv8(*args(vs, vt))
    wide, tree = vs.clone(), vt.clone()
    wide[B // 2, Hkv - 1, 0] *= 2.0 ** 12
    tree[0, 0, 0] *= 2.0 ** 12
    got = E.eagle_tree_attn_kv8(*args(wide, tree))
    torch.cuda.synchronize()
    G = Hq // Hkv
    same = torch.ones(B, Hkv, dtype=torch.bool)
    same[B // 2, Hkv - 1] = same[0, 0] = False
    equal = (got == want).view(B, n, Hkv, G * D).all(-1).all(1).cpu()
    assert equal[same].all() and not equal[~same].any()
