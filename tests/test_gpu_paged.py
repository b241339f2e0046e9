"""GPU parity of the paged cache's calls with the 64-bit forms of oracle/paged.py.

What is moved or counted is compared bit for bit, every page that must not be touched included; the
rotation and the attention to the bounds derived there, per output element.
"""
import numpy as np
import pytest
import torch

from oracle import paged as ref

pytestmark = pytest.mark.gpu
D = 128
BAD_TREE, CAPACITY = 0x01, 0x10


def _E():
    import eagle_tree_speculative_gb300 as E
    return E


def _bf16(shape, seed, gain=0.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * torch.exp(gain * torch.randn(shape[-1], generator=g))).bfloat16()


def _dev(x):
    return torch.as_tensor(np.asarray(x)).to(torch.int32).cuda().contiguous()


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _tree(rng, n):
    return [-1] + [int(rng.integers(max(0, i - 6), i)) for i in range(1, n)]


def _table(rng, rows, page, extra=2, width=None):
    """Shuffled pages for each sequence's rows; entries behind them hold page numbers that do not exist."""
    need = [-(-r // page) for r in rows]
    N = sum(need) + extra
    ids = list(rng.permutation(N))
    width = max(max(need), 1) if width is None else width
    t = rng.integers(-(2 ** 31), 2 ** 31, (len(rows), width))
    t[np.abs(t) <= N] = -1
    for b, m in enumerate(need):
        t[b, :m] = [ids.pop() for _ in range(m)]
    return t.astype(np.int64), N


def _bits(x):
    return x.view(torch.int16).cpu()


def _times_bound(got, want, tol):
    """How many times its bound the result is off, at worst (NaN where NaN is due counts as right)."""
    g = got.double().cpu()
    same = (g == want) | (torch.isnan(g) & torch.isnan(want))
    off = torch.where(same, 0.0, (g - want).abs() / (tol + 1e-300))
    return float(torch.nan_to_num(off, nan=1e9).max())


# ---------------------------------------------------------------- norms and rotation
def _rope(lens, pos, Hq, Hkv, seed, page=16, tree=False, interleaved=False, rot=128, norm=True, dest="both", base=10000.0,
          cu=None, T=None, change=None, status=0, stride=0, inplace=False, table=None, N=None):
    E, rng = _E(), np.random.default_rng(seed)
    B = len(lens)
    cu = [0] + list(np.cumsum(lens)) if cu is None else cu
    T = cu[-1] if T is None else T
    parent = [_tree(rng, lens[0]) for _ in lens] if tree else None
    if change == "tree":
        parent[1][2] = 2
    qkv = _bf16((T, (Hq + 2 * Hkv) * D + stride), seed)
    q, k, v = (x.unflatten(1, (-1, D)) for x in qkv[:, :(Hq + 2 * Hkv) * D].split([Hq * D, Hkv * D, Hkv * D], 1))
    if callable(change):
        change(q, k, v)
    qw, kw = (_bf16((D,), seed + 1) + 1, _bf16((D,), seed + 2) + 1) if norm else (None, None)
    f = (base ** -(torch.arange(0, rot, 2).double() / rot)).float()
    if table is None and dest != "packed":
        ends = [max(p, 0) + m for p, m in zip(pos, lens)]
        table, N = _table(rng, [m for m in ends], page) if max(ends) < 4000 else _far_table(rng, pos, lens, page)
        if change == "page":
            table[1, pos[1] // page] = N
    kp = vp = None
    if dest != "packed":
        kp, vp = _bf16((N, Hkv, page, D), seed + 3), _bf16((N, Hkv, page, D), seed + 4)
    want = ref.qkv_rope(q, k, v, qw, kw, f, pos, cu, parent, 1e-6, interleaved, page, N, None if dest == "packed" else table)
    gq, gk, gv = (x.unflatten(1, (-1, D)) for x in qkv.cuda()[:, :(Hq + 2 * Hkv) * D].split([Hq * D, Hkv * D, Hkv * D], 1))
    if inplace:
        gq, gk = gq.contiguous(), gk.contiguous()
    fill = lambda H: torch.full((T, H, D), 7.0, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    q_out, k_out = (gq, gk) if inplace else (fill(Hq), fill(Hkv) if dest != "pages" else None)
    st = _status()
    gp = [None if x is None else x.cuda() for x in (kp, vp)]
    E.eagle_qkv_rope(gq, gk, gv, f.cuda(), _dev(pos), cu=None if tree else _dev(cu), parent=_dev(parent) if tree else None,
                     q_weight=None if qw is None else qw.cuda(), k_weight=None if kw is None else kw.cuda(), eps=1e-6,
                     interleaved=interleaved, k_pages=gp[0], v_pages=gp[1], page_table=None if dest == "packed" else _dev(table),
                     q_out=q_out, k_out=k_out, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == status
    for t, w in enumerate(want):
        for got, name, was in ((q_out, "q", q), (k_out, "k", k)):
            if got is None:
                continue
            if w is None:
                assert torch.equal(got[t].cpu(), was[t] if inplace else torch.full_like(was[t], 7.0)), (t, name)
                continue
            assert _times_bound(got[t], *w[name]) <= 1.0, (t, name)
        if w is not None and w["place"] is not None:
            id_, r = w["place"]
            kp[id_, :, r] = torch.nan                      # compared here, the rest below
            assert _times_bound(gp[0][id_, :, r], *w["k"]) <= 1.0, (t, "page")
            if k_out is not None:
                assert torch.equal(_bits(gp[0][id_, :, r]), _bits(k_out[t])), "the same rounding in both places"
            vp[id_, :, r] = w["v"]
    if dest != "packed":
        keys = torch.isnan(kp)
        assert torch.equal(_bits(gp[1]), _bits(vp)), "V pages"
        assert torch.equal(_bits(gp[0])[~keys], _bits(kp)[~keys]), "K pages that are nobody's new rows"


def _far_table(rng, pos, lens, page):
    """A table of far positions: pages for the new rows alone."""
    width = -(-max(p + m for p, m in zip(pos, lens)) // page)
    t = np.full((len(pos), width), -1, np.int64)
    N = sum(-(-(p + m) // page) - p // page for p, m in zip(pos, lens)) + 2
    ids = list(rng.permutation(N))
    for b, (p, m) in enumerate(zip(pos, lens)):
        for x in range(p // page, -(-(p + m) // page)):
            t[b, x] = ids.pop()
    return t, N


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [16, 32, 48, 64, 96, 112, 128])
def test_rope_dims(rot, interleaved):
    _rope([5, 17, 1], [3, 14, 100], 4, 2, rot, rot=rot, interleaved=interleaved)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 1), (3, 1), (5, 5), (6, 2), (7, 1), (28, 4), (32, 8), (40, 40)])
@pytest.mark.parametrize("dest", ["pages", "packed", "both"])
def test_rope_heads(Hq, Hkv, dest):
    _rope([4, 9], [7, 0], Hq, Hkv, Hq, dest=dest, norm=Hq % 2 == 0)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("pos", [0, 1, 15, 16, 63, 64, 127])
def test_rope_rows_into_pages(page, pos):
    _rope([1, 130, 33], [pos, pos, 2 * pos], 2, 1, 10 * page + pos, page=page)


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 64])
def test_rope_trees(n):
    """Position is the depth, the row is the node."""
    _rope([n] * 3, [0, 5, 130], 4, 2, n, tree=True, page=32)


def test_rope_chain_of_64_nodes():
    E = _E()
    q, k = _bf16((64, 2, D), 1), _bf16((64, 1, D), 2)
    f = (10000.0 ** -(torch.arange(0, D, 2).double() / D)).float()
    chain = [[-1] + list(range(63))]
    out = E.eagle_qkv_rope(q.cuda(), k.cuda(), None, f.cuda(), _dev([40]), parent=_dev(chain))
    packed = E.eagle_qkv_rope(q.cuda(), k.cuda(), None, f.cuda(), _dev([40]), cu=_dev([0, 64]))
    assert all(torch.equal(a, b) for a, b in zip(out, packed))


@pytest.mark.parametrize("pos", [1 << 16, 131071, (1 << 20) + 3, (1 << 24) + 1])
def test_rope_far_positions(pos):
    """Angles of far positions, where a product in 32 bits has lost them."""
    _rope([3, 2], [pos, pos // 3], 2, 1, 5, dest="packed", base=500000.0)
    if pos < 1 << 20:
        _rope([3, 2], [pos, pos // 3], 2, 1, 5, base=500000.0, page=128)


def test_rope_many_tokens_and_sequences():
    """More sequences than lanes, empty ones among them; enough tokens that a warp has a whole one."""
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(0, 60, 90)]
    lens[0] = lens[31] = lens[32] = lens[89] = 0
    _rope(lens, [int(x) for x in rng.integers(0, 50, 90)], 2, 1, 9, page=16)


@pytest.mark.parametrize("B", [33, 34, 63, 64, 65, 100, 1025, 1057])
def test_rope_finds_a_token_s_sequence(B):
    """Sequences behind the first 32, most of them empty; rows of nobody before the first and behind the last."""
    rng = np.random.default_rng(B)
    lens = [int(x) for x in rng.integers(1, 4, B) * (rng.random(B) < (0.9 if B < 100 else 0.2))]
    cu = [3] + list(3 + np.cumsum(lens))
    _rope(lens, [int(x) for x in rng.integers(0, 900, B)], 1, 1, B, dest="packed", cu=cu, T=int(cu[-1]) + 5)


def test_rope_large_call():
    """Several thousand tokens: on a sample of them."""
    E = _E()
    T, Hq, Hkv = 6000, 3, 1
    q, k = _bf16((T, Hq, D), 5), _bf16((T, Hkv, D), 6)
    w = _bf16((D,), 7)
    f = (10000.0 ** -(torch.arange(0, D, 2).double() / D)).float()
    a, b = E.eagle_qkv_rope(q.cuda(), k.cuda(), None, f.cuda(), _dev([11]), cu=_dev([0, T]), q_weight=w.cuda())
    for t in list(range(0, T, 397)) + [T - 1]:
        for got, x, y in ((a, q, w), (b, k, None)):
            o, tol = ref.turned(x[t], y, f, 11 + t, 1e-6, False)
            assert _times_bound(got[t], o, tol) <= 1.0, t


def test_rope_strided_rows_in_place_and_tokens_of_nobody():
    _rope([4, 7], [1, 2], 3, 1, 3, stride=24)
    _rope([4, 7], [1, 2], 3, 1, 4, inplace=True)
    _rope([3, 4], [1, 2], 3, 1, 5, cu=[2, 5, 9], T=12)


def test_rope_magnitudes():
    """Squares that leave fp32, rows of zeros, and infinities where nothing is turned."""
    def change(q, k, v):
        q[0] *= 2.0 ** 100
        q[1, 0] = 3e38
        q[2] *= 2.0 ** -100
        q[3] = 0.0
        q[4, 0, 5] = torch.inf
        q[5, 0, 7] = torch.nan
        k[1] *= 2.0 ** 70
        v[2] = torch.inf
    _rope([7], [3], 2, 1, 8, change=change)
    _rope([7], [3], 2, 1, 8, change=change, rot=64, norm=False, interleaved=True)

    def behind(q, k, v):
        q[:, :, 64] = torch.inf
        k[:, :, 100] = -torch.inf
    _rope([7], [3], 2, 1, 8, change=behind, rot=64, norm=False)


def test_rope_refused_sequences():
    """What is refused is left out, the others are done."""
    _rope([4, 4, 4], [3, -1, 9], 2, 1, 1, status=CAPACITY)
    _rope([5, 5, 5], [3, 4, 9], 2, 1, 2, tree=True, change="tree", status=BAD_TREE)
    rng = np.random.default_rng(1)
    t, N = _table(rng, [32, 32], 16, width=2)
    _rope([4, 4], [29, 20], 2, 1, 3, table=t, N=N, status=CAPACITY)     # 33 rows
    _rope([4, 4], [29, 20], 2, 1, 4, change="page", status=CAPACITY)    # a page that does not exist


@pytest.mark.parametrize("cu", [[0, 5, 3], [-1, 2, 6], [0, 3, 7]])
def test_rope_bad_starts_write_nothing(cu):
    E = _E()
    q, k = _bf16((6, 2, D), 1).cuda(), _bf16((6, 1, D), 2).cuda()
    qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    st = _status()
    E.eagle_qkv_rope(q, k, None, torch.ones(64, device="cuda"), _dev([0, 0]), cu=_dev(cu), q_out=qo, k_out=ko, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == CAPACITY and bool((qo == 7).all()) and bool((ko == 7).all())


# ---------------------------------------------------------------- attention
def _attn(L, n, Hq, Hkv, page, seed, status=0, scale=None, change=None, dirty=True, gain=0.5):
    E, rng = _E(), np.random.default_rng(seed)
    B = len(L)
    table, N = _table(rng, [max(x, 0) + n for x in L], page, extra=3)
    parent = [_tree(rng, n) for _ in L]
    q = _bf16((B, n, Hq, D), seed, gain)
    kp, vp = _bf16((N, Hkv, page, D), seed + 1, gain), _bf16((N, Hkv, page, D), seed + 2, gain)
    if change:
        change(table, parent, L, q, kp, vp, N)
    want, tol = ref.tree_attn_paged(q, kp, vp, table, L, parent, scale or D ** -0.5)
    if dirty:
        # whatever is not a row of a sequence is NaN or infinite
        used = torch.zeros(N, page, dtype=torch.bool)
        for b, x in enumerate(L):
            for p, r in ref.places(table[b], page, range(min(max(x, 0) + n, table.shape[1] * page))):
                if 0 <= p < N:
                    used[p, r] = True
        for x, y in ((kp, torch.nan), (vp, torch.inf)):
            x.masked_fill_(~used[:, None, :, None], y)
        vp[:, :, 1::3] = torch.where(used[:, None, 1::3, None], vp[:, :, 1::3], torch.nan)
    st = _status()
    args = (q.cuda(), kp.cuda(), vp.cuda(), _dev(table), _dev(L), _dev(parent))
    out = E.eagle_tree_attn_paged(*args, scale=scale, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == status
    assert _times_bound(out, want, tol) <= 1.0
    return args, out


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("L", [0, 1, 15, 16, 63, 64, 126, 127, 128, 129, 255, 256, 300])
def test_decoding_of_every_length(L, page):
    _attn([L], 1, 4, 2, page, L + page)


@pytest.mark.parametrize("n", [2, 3, 31, 32, 33, 60, 63, 64])
@pytest.mark.parametrize("L", [0, 5, 64, 100, 127, 128, 200, 511])
def test_trees(n, L):
    _attn([L, L + 1], n, 4, 1, 32, n + L)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 1), (3, 1), (4, 4), (5, 1), (6, 2), (7, 1), (14, 2), (8, 1), (16, 1), (12, 1),
                                    (33, 1), (64, 2), (128, 1), (100, 1)])
@pytest.mark.parametrize("n", [1, 7, 40])
def test_group_sizes(Hq, Hkv, n):
    _attn([150, 0, 301], n, Hq, Hkv, 64, Hq + n)


def test_ragged_batch():
    """More sequences than lanes, pieces that hold many units and units that are cut."""
    rng = np.random.default_rng(6)
    L = [int(x) for x in rng.integers(0, 200, 70)]
    L[3], L[40] = 3000, 0
    _attn(L, 1, 4, 2, 16, 1)
    _attn(L[:40], 5, 4, 2, 64, 2)


@pytest.mark.parametrize("n,Hq,Hkv", [(1, 8, 1), (60, 4, 1), (50, 8, 1)])
def test_one_long_sequence_over_all_ctas(n, Hq, Hkv):
    """Few units: cut over the device and merged."""
    _attn([20011], n, Hq, Hkv, 16, n)


def test_three_row_tiles():
    """A pair of row tiles and a single one of the same sequence."""
    _attn([700, 20, 5000], 40, 8, 1, 32, 4)
    _attn([700, 20], 64, 5, 1, 128, 5)


@pytest.mark.parametrize("size", [2.0 ** -30, 1.0, 2.0 ** 20])
def test_magnitudes(size):
    """Scores far from each other, V far from one; the largest key last, so that the maximum rises late."""
    def change(table, parent, L, q, kp, vp, N):
        q *= 4.0
        vp *= size
        for b, x in enumerate(L):
            p, r = ref.places(table[b], 16, [x - 1])[0]
            kp[p, :, r] *= 8.0
    _attn([400, 131], 3, 4, 2, 16, 7, change=change)


def test_scale_argument():
    _attn([77], 4, 4, 2, 16, 8, scale=1.0, gain=0.1)
    _attn([77], 4, 4, 2, 16, 8, scale=1e-3)


def test_refused_sequences_are_zeros_and_the_others_are_not():
    def tree(table, parent, L, q, kp, vp, N):
        parent[1][3] = 3
    args, out = _attn([50, 60, 70], 5, 4, 2, 16, 9, status=BAD_TREE, change=tree)
    assert not out[1].any() and out[0].any() and out[2].any()

    def length(table, parent, L, q, kp, vp, N):
        L[0], L[2] = -1, table.shape[1] * 16 - 4
    args, out = _attn([50, 60, 70], 5, 4, 2, 16, 10, status=CAPACITY, change=length)
    assert not out[0].any() and not out[2].any() and out[1].any()

    def page(table, parent, L, q, kp, vp, N):
        table[1, 2], table[1, 1] = N, -5
    _attn([50, 60, 300], 5, 4, 2, 16, 11, status=CAPACITY, change=page)       # its rows count as zeros


@pytest.mark.parametrize("n,Hq,Hkv,page", [(1, 16, 16, 16), (1, 40, 20, 128), (16, 20, 20, 32), (20, 64, 8, 64), (33, 16, 8, 16)])
def test_many_short_units_of_a_cta(n, Hq, Hkv, page):
    """Units of one tile, of two and of three next to one another, and refused sequences between them: more than a few a CTA."""
    rng = np.random.default_rng(n + Hq)
    B = 150 if n < 20 else 80
    L = [int(x) for x in rng.choice([0, 1, 60, 90, 127 - n, 128 - n, 129 - n, 200, 300], B, p=[.1, .2, .1, .2, .1, .1, .1, .05, .05])]

    def change(table, parent, L, q, kp, vp, N):
        for b in rng.choice(B, 12, replace=False):
            L[b] = -1 if b % 2 else table.shape[1] * page
        for b in (7, 8, 9, 10):
            L[b] = -5
    _attn(L, n, Hq, Hkv, page, n, status=CAPACITY, change=change)
    _attn([min(max(x, 0), 128 - n) for x in L], n, Hq, Hkv, page, n + 1)


def test_replayed_graph_and_two_streams():
    E = _E()
    args, out = _attn([900, 30, 4000], 9, 8, 2, 16, 12)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = E.eagle_tree_attn_paged(*args)
    again.fill_(3)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(again, out)
    args2, out2 = _attn([2000, 7], 20, 4, 1, 64, 13)
    s = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        got.append((E.eagle_tree_attn_paged(*args, stream=s[0]), E.eagle_tree_attn_paged(*args2, stream=s[1])))
    torch.cuda.synchronize()
    assert all(torch.equal(a, out) and torch.equal(b, out2) for a, b in got)


# ---------------------------------------------------------------- pages
class _Slots:
    """The cache's numbers on the host, by the 64-bit form, beside the device's."""

    def __init__(self, B, N, P, page, layers, Hkv, seed):
        E = _E()
        self.page, self.B, self.N = page, B, N
        self.table, self.held, self.refs, self.len = [[-1] * P for _ in range(B)], [0] * B, [0] * N, [0] * B
        self.k, self.v = _bf16((layers, N, Hkv, page, D), seed), _bf16((layers, N, Hkv, page, D), seed + 1)
        _, _, self.d_table, self.d_held, self.d_refs = E.paged_cache(0, N, Hkv, page, B, P)
        self.d_k, self.d_v, self.d_len = self.k.cuda(), self.v.cuda(), _dev(self.len)

    def assign(self, grow, src=None, refused=False):
        E, st = _E(), _status()
        E.eagle_pages_assign(self.d_k, self.d_v, self.d_table, self.d_held, self.d_refs, self.d_len, _dev(grow),
                             src=None if src is None else _dev(src), dev_status=st)
        got = ref.pages_assign(self.table, self.held, self.refs, self.len, grow, src, self.page)
        assert (got is None) == refused
        if got is not None:
            self.table, self.held, self.refs, self.len, copies = got
            for frm, to, rows in copies:
                for x in (self.k, self.v):
                    x[:, to, :, :rows] = x[:, frm, :, :rows]
        self.same()
        assert int(st.item()) == (CAPACITY if refused else 0)
        return 0 if got is None else len(copies)

    def same(self):
        torch.cuda.synchronize()
        assert self.d_len.tolist() == self.len and self.d_held.tolist() == self.held
        assert self.d_table.tolist() == self.table and self.d_refs.tolist() == self.refs
        for x, y in ((self.d_k, self.k), (self.d_v, self.v)):
            assert torch.equal(_bits(x), _bits(y))

    def set_len(self, lens):
        self.len = list(lens)
        self.d_len.copy_(_dev(lens))


@pytest.mark.parametrize("B,N,P,page,layers,Hkv", [(1, 8, 6, 16, 1, 1), (5, 60, 12, 16, 2, 3), (40, 700, 40, 32, 1, 1),
                                                   (150, 5000, 9, 64, 1, 1), (7, 200, 70, 128, 1, 2)])
def test_assign_random_steps(B, N, P, page, layers, Hkv):
    """Growth, forks, reorders and ends in turn, lengths cut back into shared pages among them."""
    rng = np.random.default_rng(B)
    c = _Slots(B, N, P, page, layers, Hkv, B)
    per = max(1, N // (3 * B))                            # pages a slot may come to hold
    copied = 0
    for step in range(14):
        src = None
        if step % 3 == 1:
            src = [int(x) for x in rng.integers(-1, B, B)]
        elif step % 3 == 2:
            src = [int(rng.integers(-1, B)) if rng.random() < 0.3 else b for b in range(B)]
        now = [c.len[b] if src is None else (c.len[src[b]] if src[b] >= 0 else 0) for b in range(B)]
        grow = [int(rng.integers(0, max(1, min(P, per) * page - x) + 1)) for x in now]
        grow = [min(g, P * page - x) for g, x in zip(grow, now)]
        if sum(r == 0 for r in c.refs) < B * (min(P, per) + 1):
            c.assign([0] * B, [b if rng.random() < 0.5 else -1 for b in range(B)])
            c.assign([0] * B)                             # what was given back is free now
            continue
        copied += c.assign(grow, src)
        # some of the new rows are written; some sequences go back
        c.set_len([int(rng.integers(max(0, x - 20), x + g + 1)) for x, g in zip(now, grow)])
    assert copied > 0 or B == 1


def test_assign_one_prompt_into_every_slot():
    c = _Slots(9, 60, 8, 16, 3, 2, 1)
    c.assign([75] + [0] * 8)
    c.set_len([75] + [0] * 8)
    assert c.assign([1] * 9, [0] * 9) == 8                 # the last page, eight times
    assert c.refs.count(9) == 4
    assert c.assign([0] * 9, [3] * 9) == 8                 # slot 3 keeps its page, the others take theirs afresh
    assert c.assign([5] * 9, [-1] * 9) == 0                # all end, and begin again
    assert c.assign([0] * 9, [-1] * 9) == 0
    assert c.refs == [0] * 60


def test_assign_a_full_page_is_shared_without_copies():
    c = _Slots(4, 30, 6, 32, 2, 1, 2)
    c.assign([64, 0, 0, 0])
    c.set_len([64, 0, 0, 0])
    assert c.assign([0] * 4, [0] * 4) == 0
    assert sorted(c.refs)[-2:] == [4, 4]
    assert c.assign([1] * 4) == 0
    # a slot that went back into a shared page gets one of its own before it writes there
    c.set_len([50, 64, 64, 64])
    assert c.assign([10, 1, 1, 1]) == 1


def test_assign_too_few_pages_changes_nothing():
    c = _Slots(3, 7, 6, 16, 1, 1, 3)
    c.assign([32, 20, 16])
    c.set_len([32, 20, 16])
    c.assign([40, 20, 0], refused=True)
    c.assign([16, 0, 16])
    c.assign([0, 0, 0], [1, 1, 1], refused=True)           # what is given back is free in the next call only
    c.assign([0, 0, 0], [-1, 1, -1])
    c.assign([0, 0, 0], [1, 1, 1])


@pytest.mark.parametrize("what", ["src", "src2", "grow", "len", "beyond", "wide", "held", "page", "page2"])
def test_assign_refuses_numbers_out_of_range(what):
    c = _Slots(3, 20, 4, 16, 1, 1, 4)
    c.assign([40, 20, 16])
    c.set_len([40, 20, 16])
    keep = [x.clone() for x in (c.d_table, c.d_held, c.d_refs, c.d_len, c.d_k, c.d_v)]
    grow, src = [1, 1, 1], [0, 1, 1]
    if what == "src":
        src[1] = 3
    if what == "src2":
        src[2] = -2
    if what == "grow":
        grow[0] = -1
    if what == "wide":
        grow[0] = 2 ** 31 - 1
    if what == "len":
        c.d_len[1] = -1
    if what == "beyond":
        c.d_len[1] = 33                                   # two pages are held
    if what == "held":
        c.d_held[0] = 5
    if what == "page":
        c.d_table[1, 1] = 20
    if what == "page2":
        c.d_table[2, 0] = -7                              # given back by slot 2
    now = [x.clone() for x in (c.d_table, c.d_held, c.d_refs, c.d_len)]
    st = _status()
    _E().eagle_pages_assign(c.d_k, c.d_v, c.d_table, c.d_held, c.d_refs, c.d_len, _dev(grow), src=_dev(src), dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == CAPACITY
    assert all(torch.equal(x, y) for x, y in zip((c.d_table, c.d_held, c.d_refs, c.d_len), now))
    assert torch.equal(c.d_k, keep[4]) and torch.equal(c.d_v, keep[5])


def _commit(L, n, path, acc, depth, page, layers, Hkv, seed, status=0, table=None, N=None, separate=False):
    E, rng = _E(), np.random.default_rng(seed)
    if table is None:
        table, N = _table(rng, [max(x, 0) + n for x in L], page)
    k, v = _bf16((layers, N, Hkv, page, D), seed), _bf16((layers, N, Hkv, page, D), seed + 1)
    dk, dv, dl, st = k.cuda(), v.cuda(), _dev(L), _status()
    out = torch.full_like(dl, -9) if separate else dl
    got = E.eagle_pages_commit(dk, dv, _dev(table), dl, _dev(path), _dev(acc), depth, kv_len_out=out if separate else None, dev_status=st)
    torch.cuda.synchronize()
    want = ref.pages_commit([k, v], table, L, path, acc, depth, page, N)
    assert got is out and got.tolist() == want and int(st.item()) == status
    assert not separate or dl.tolist() == L
    assert torch.equal(_bits(dk), _bits(k)) and torch.equal(_bits(dv), _bits(v))


def _paths(rng, B, n, depth):
    acc = [int(rng.integers(-1, min(depth, n - 1) + 1)) for _ in range(B)]
    return acc, [([0] + sorted(int(x) for x in rng.choice(np.arange(1, n), max(a, 0), replace=False)) + [-1] * depth)[:depth + 1]
                 for a in acc]


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("B,n,depth,layers,Hkv", [(1, 60, 6, 32, 8), (3, 64, 63, 2, 1), (70, 12, 5, 1, 3), (9, 2, 1, 3, 2), (4, 1, 0, 2, 2)])
def test_commit(B, n, depth, layers, Hkv, page):
    rng = np.random.default_rng(B + n)
    acc, path = _paths(rng, B, n, depth)
    if depth == 63:
        acc[0], path[0] = 63, list(range(64))              # every node
        acc[1], path[1] = 62, [0] + list(range(2, 64)) + [-1]        # a chain of overlapping moves
    _commit([int(x) for x in rng.integers(0, 200, B)], n, path, acc, depth, page, layers, Hkv, page + B, separate=B == 3)


def test_commit_refused_sequences():
    path = [[0, 2, 3]] * 3
    _commit([5, 6, 7], 4, [[0, 2, 3], [1, 2, 3], [0, 3, 3]], [2, 2, 2], 2, 16, 2, 1, 1, status=BAD_TREE)
    _commit([5, -1, 7], 4, path, [2, 2, 3], 2, 16, 2, 1, 2, status=CAPACITY)
    rng = np.random.default_rng(5)
    t, N = _table(rng, [32, 32, 32], 16, width=2)
    _commit([30, 29, 28], 4, path, [2, 2, 2], 2, 16, 2, 1, 3, status=CAPACITY, table=t, N=N)
    t[1, 1] = N
    _commit([14, 14, 28], 4, path, [2, 2, 2], 2, 16, 2, 1, 4, status=CAPACITY, table=t, N=N)


# ---------------------------------------------------------------- together, as a server runs them
def test_a_server_s_steps():
    """Prompts, a fork, two tree steps and a decoding step in two layers: every attention against keys and
    values kept per sequence on the host, in the order in which they were accepted."""
    E, rng = _E(), np.random.default_rng(2)
    layers, Hq, Hkv, page, B, n, depth = 2, 8, 2, 16, 4, 7, 3
    kp, vp, table, held, refs = E.paged_cache(layers, 64, Hkv, page, B, 12)
    st, kv_len = _status(), _dev([0] * B)
    f = (10000.0 ** -(torch.arange(0, D, 2).double() / D)).float().cuda()
    w = (_bf16((D,), 1) + 1).cuda()
    rows = [[([], []) for _ in range(B)] for _ in range(layers)]          # K, V of each sequence, on the host

    def project(T, seed):
        return [x.unflatten(1, (-1, D)) for x in _bf16((T, (Hq + 2 * Hkv) * D), seed).cuda().split([Hq * D, Hkv * D, Hkv * D], 1)]

    # prompts of two sequences
    lens = [37, 16, 0, 0]
    cu = _dev([0] + list(np.cumsum(lens)))
    E.eagle_pages_assign(kp, vp, table, held, refs, kv_len, _dev(lens), src=_dev([-1] * B), dev_status=st)
    for l in range(layers):
        q, k, v = project(sum(lens), 10 + l)
        k_out = torch.empty(sum(lens), Hkv, D, dtype=torch.bfloat16, device="cuda")
        qr, kr = E.eagle_qkv_rope(q, k, v, f, kv_len, cu=cu, q_weight=w, k_weight=w, k_pages=kp[l], v_pages=vp[l], page_table=table,
                                  k_out=k_out, dev_status=st)
        E.eagle_prompt_attn(qr, kr, v, cu, dev_status=st)
        at = 0
        for b, m in enumerate(lens):
            rows[l][b][0].extend(kr[at:at + m].cpu())
            rows[l][b][1].extend(v[at:at + m].cpu())
            at += m
    kv_len += _dev(lens)
    # every slot goes on with the first or the second
    src = [0, 1, 0, 1]
    E.eagle_pages_assign(kp, vp, table, held, refs, kv_len, _dev([n] * B), src=_dev(src), dev_status=st)
    rows = [[([*r[s][0]], [*r[s][1]]) for s in src] for r in rows]
    for step, m in enumerate([n, n, 1]):
        if step:
            E.eagle_pages_assign(kp, vp, table, held, refs, kv_len, _dev([m] * B), dev_status=st)
        parent = [_tree(rng, m) for _ in range(B)]
        acc, path = _paths(rng, B, m, depth)
        acc = [max(a, 0) for a in acc]
        for l in range(layers):
            q, k, v = project(B * m, 100 + 10 * step + l)
            k_tree = torch.empty(B * m, Hkv, D, dtype=torch.bfloat16, device="cuda")
            qr, _ = E.eagle_qkv_rope(q, k, v, f, kv_len, parent=_dev(parent), q_weight=w, k_weight=w, k_pages=kp[l], v_pages=vp[l],
                                     page_table=table, k_out=k_tree, dev_status=st)
            out = E.eagle_tree_attn_paged(qr.view(B, m, Hq, D), kp[l], vp[l], table, kv_len, _dev(parent), dev_status=st)
            for b in range(B):
                K, V = rows[l][b]
                kt, vt = k_tree.view(B, m, Hkv, D)[b].cpu(), v.reshape(B, m, Hkv, D)[b].cpu()
                one = [torch.stack(K + list(kt)).transpose(0, 1), torch.stack(V + list(vt)).transpose(0, 1)]     # one page each
                want, tol = ref.tree_attn_paged(qr.view(B, m, Hq, D)[b:b + 1].cpu(), one[0][None], one[1][None], np.zeros((1, 1), int),
                                                [len(K)], [parent[b]], D ** -0.5)
                assert _times_bound(out[b], want[0], tol[0]) <= 1.0
                K.extend(kt[path[b][t]] for t in range(acc[b] + 1))
                V.extend(vt[path[b][t]] for t in range(acc[b] + 1))
        E.eagle_pages_commit(kp, vp, table, kv_len, _dev(path), _dev(acc), depth, dev_status=st)
    assert kv_len.tolist() == [len(rows[0][b][0]) for b in range(B)]
    assert int(st.item()) == 0
