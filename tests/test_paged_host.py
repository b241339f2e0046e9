"""Host checks of the paged cache's calls (no GPU work is done), and pins of their 64-bit forms."""
import ctypes
import os

import numpy as np
import pytest
import torch

import oracle
from oracle import paged as ref

OK, INVALID, SHAPE, CAPACITY = 0, 1, 2, 3
A = 4096                                     # a 16-byte aligned, never dereferenced address
D = 128


@pytest.fixture(scope="module")
def L():
    from eagle_tree_speculative_gb300 import _lib, build
    import shutil
    if not os.path.exists(build.LIB):
        if shutil.which(build.NVCC) is None:
            pytest.skip("nvcc not available to build the library")
        build.build()
    lib = ctypes.CDLL(build.LIB)
    for name, (res, args) in _lib.SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    return lib


def _call(fn, names, good, **change):
    vals = {**good, **change}
    return fn(*[vals[n] for n in names])


ASSIGN = "k v table held refs kv_len grow src layers B N Hkv page d P ws ws_bytes status stream".split()
ASSIGN_OK = dict(k=A, v=A, table=A, held=A, refs=A, kv_len=A, grow=A, src=None, layers=2, B=3, N=9, Hkv=2, page=16, d=128, P=4,
                 ws=A, ws_bytes=1 << 40, status=None, stream=None)
COMMIT = "k v table kv_len kv_out path acc layers B N Hkv page d P D status stream".split()
COMMIT_OK = dict(k=A, v=A, table=A, kv_len=A, kv_out=A, path=A, acc=A, layers=2, B=1, N=9, Hkv=2, page=16, d=128, P=4, D=3,
                 status=None, stream=None)
ROPE = ("q k v qw kw f cu parent pos q_out k_out kp vp table T B n Hq Hkv d rot inter eps qs ks vs N page P status "
        "stream").split()
ROPE_OK = dict(q=A, k=A, v=A, qw=A, kw=A, f=A, cu=A, parent=None, pos=A, q_out=A, k_out=A, kp=A, vp=A, table=A, T=10, B=2, n=0,
               Hq=8, Hkv=2, d=128, rot=128, inter=0, eps=1e-6, qs=1024, ks=256, vs=256, N=9, page=16, P=4, status=None,
               stream=None)
TREE = "q k v table kv_len parent out B n Hq Hkv d N page P scale ws ws_bytes status stream".split()
TREE_OK = dict(q=A, k=A, v=A, table=A, kv_len=A, parent=A, out=A, B=1, n=4, Hq=8, Hkv=2, d=128, N=9, page=16, P=40, scale=0.1,
               ws=A, ws_bytes=1 << 40, status=None, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(layers=-1), INVALID), (dict(B=-1), INVALID), (dict(N=0), INVALID), (dict(Hkv=0), INVALID), (dict(P=0), INVALID),
    (dict(page=48), SHAPE), (dict(page=8), SHAPE), (dict(page=256), SHAPE), (dict(d=64), SHAPE), (dict(N=1 << 27), SHAPE),
    (dict(P=(1 << 26) + 1), SHAPE), (dict(B=1 << 20, P=1 << 12), SHAPE), (dict(table=None), INVALID), (dict(held=None), INVALID),
    (dict(refs=None), INVALID), (dict(kv_len=None), INVALID), (dict(grow=None), INVALID), (dict(k=None), INVALID),
    (dict(v=None), INVALID), (dict(k=A + 8), INVALID), (dict(ws=A + 4), INVALID), (dict(ws=None), CAPACITY),
    (dict(ws_bytes=10), CAPACITY)])
def test_assign_refusals(L, change, status):
    assert _call(L.eagle_pages_assign, ASSIGN, ASSIGN_OK, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(layers=-1), INVALID), (dict(B=-1), INVALID), (dict(N=0), INVALID), (dict(P=0), INVALID), (dict(D=-1), INVALID),
    (dict(D=65), SHAPE), (dict(page=20), SHAPE), (dict(d=256), SHAPE), (dict(k=None), INVALID), (dict(kv_out=None), INVALID),
    (dict(path=None), INVALID), (dict(table=None), INVALID), (dict(v=A + 2), INVALID)])
def test_commit_refusals(L, change, status):
    assert _call(L.eagle_pages_commit, COMMIT, COMMIT_OK, **change) == status


def test_slots_that_a_call_can_have(L):
    many = dict(B=(1 << 16) + 1, P=1)
    assert _call(L.eagle_pages_assign, ASSIGN, ASSIGN_OK, **many) == SHAPE
    assert _call(L.eagle_pages_commit, COMMIT, COMMIT_OK, **many) == SHAPE
    assert _call(L.eagle_pages_commit, COMMIT, COMMIT_OK, B=(1 << 30) - 1, P=1) == SHAPE
    assert L.eagle_pages_workspace_size(1 << 16, 9, 1) > 0 and L.eagle_pages_workspace_size((1 << 16) + 1, 9, 1) == 0


NO_PAGES = dict(kp=None, vp=None, table=None, v=None, N=0, page=0, P=0, vs=0)


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), INVALID), (dict(B=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hkv=0), INVALID), (dict(eps=0.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID), (dict(d=64), SHAPE), (dict(rot=0), SHAPE),
    (dict(rot=24), SHAPE), (dict(rot=144), SHAPE), (dict(qs=1016), INVALID), (dict(ks=260), INVALID), (dict(vs=128), INVALID),
    (dict(N=0), INVALID), (dict(P=0), INVALID), (dict(page=17), SHAPE), (dict(cu=None), INVALID), (dict(parent=A), INVALID),
    (dict(cu=None, parent=A, n=4), INVALID), (dict(cu=None, parent=A, n=65, T=130), SHAPE), (dict(q=None), INVALID),
    (dict(k=None), INVALID), (dict(f=None), INVALID), (dict(pos=None), INVALID), (dict(q_out=None), INVALID),
    (dict(v=None), INVALID), (dict(kp=None), INVALID), (dict(table=None), INVALID), (dict(**NO_PAGES, k_out=None), INVALID),
    (dict(q=A + 8), INVALID), (dict(qw=A + 2), INVALID), (dict(k_out=A + 4), INVALID), (dict(Hq=70000, qs=70000 * 128), SHAPE)])
def test_rope_refusals(L, change, status):
    assert _call(L.eagle_qkv_rope, ROPE, ROPE_OK, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(B=-1), INVALID), (dict(n=0), INVALID), (dict(Hq=0), INVALID), (dict(Hkv=0), INVALID), (dict(N=0), INVALID),
    (dict(P=0), INVALID), (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(n=65), SHAPE), (dict(d=64), SHAPE), (dict(Hkv=3), SHAPE), (dict(Hq=258), SHAPE), (dict(page=100), SHAPE),
    (dict(P=1 << 27), SHAPE), (dict(N=1 << 30), SHAPE), (dict(B=1 << 25, n=64), SHAPE), (dict(q=None), INVALID),
    (dict(k=None), INVALID), (dict(table=None), INVALID), (dict(kv_len=None), INVALID), (dict(parent=None), INVALID),
    (dict(out=None), INVALID), (dict(q=A + 8), INVALID), (dict(out=A + 2), INVALID), (dict(ws=A + 8), INVALID),
    (dict(ws=None, B=64), CAPACITY), (dict(ws_bytes=64, B=64), CAPACITY)])
def test_tree_attention_refusals(L, change, status):
    assert _call(L.eagle_tree_attn_paged, TREE, TREE_OK, **change) == status


def test_empty_batches_are_no_ops(L):
    none = dict(k=None, v=None, table=None, kv_len=None, B=0)
    assert _call(L.eagle_pages_assign, ASSIGN, ASSIGN_OK, **none, held=None, refs=None, grow=None, ws=None, ws_bytes=0) == OK
    assert _call(L.eagle_pages_commit, COMMIT, COMMIT_OK, **none, kv_out=None, path=None, acc=None) == OK
    assert _call(L.eagle_pages_commit, COMMIT, COMMIT_OK, k=None, layers=0) == OK
    assert _call(L.eagle_tree_attn_paged, TREE, TREE_OK, **none, q=None, parent=None, out=None, ws=None, ws_bytes=0) == OK
    for change in (dict(B=0, T=0), dict(T=0), dict(B=0)):
        assert _call(L.eagle_qkv_rope, ROPE, ROPE_OK, **change, q=None, cu=None, pos=None, q_out=None, f=None) == OK


def test_workspace_sizes(L):
    assert L.eagle_pages_workspace_size(0, 5, 5) == 0 and L.eagle_pages_workspace_size(1 << 20, 5, 1 << 12) == 0
    small, large = L.eagle_pages_workspace_size(4, 100, 10), L.eagle_pages_workspace_size(64, 10000, 500)
    assert 0 < small < large
    size = L.eagle_tree_attn_paged_workspace_size
    assert size(1, 1, 8, 1, 128, 16, 1) == 0               # one piece
    assert size(64, 60, 32, 8, 128, 64, 65) > 0
    assert size(64, 65, 32, 8, 128, 64, 65) == size(64, 60, 32, 8, 64, 64, 65) == size(64, 60, 32, 8, 128, 63, 65) == 0


# ---------------------------------------------------------------- pins of the 64-bit forms
def _bf16(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).bfloat16()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("half", [8, 32, 64])
def test_rotation_is_a_complex_product(half, interleaved):
    x, w = _bf16((3, D), half), _bf16((D,), 1)
    f = torch.rand(half, generator=torch.Generator().manual_seed(2))
    out, _ = ref.turned(x, w, f, 77, 1e-5, interleaved)
    y = torch.nn.functional.rms_norm(x.double(), (D,), w.double(), 1e-5)
    assert torch.allclose(out[:, 2 * half:], y[:, 2 * half:], rtol=1e-12)
    pair = lambda t: t[:, :2 * half].unflatten(1, (half, 2)) if interleaved else t[:, :2 * half].unflatten(1, (2, half)).transpose(1, 2)  # noqa: E731
    z = torch.view_as_complex(pair(y).contiguous()) * torch.polar(torch.ones(half).double(), 77 * f.double())
    assert torch.allclose(pair(out), torch.view_as_real(z), rtol=1e-10, atol=1e-12)


def test_rotation_by_known_angles():
    x = torch.zeros(1, D)
    x[0, 0], x[0, 1] = 1.0, 2.0
    f = torch.tensor([np.pi / 2, np.pi])
    out, _ = ref.turned(x, None, f, 1, 1e-6, False)        # pairs (0, 2) and (1, 3): a quarter and half a turn
    assert torch.allclose(out[0, :4], torch.tensor([0.0, -2.0, 1.0, 0.0]).double(), atol=1e-6)
    out, _ = ref.turned(x, None, f[:1], 1, 1e-6, True)      # the pair (0, 1), a quarter turn
    assert torch.allclose(out[0, :2], torch.tensor([-2.0, 1.0]).double(), atol=1e-6)
    assert ref.depths([-1, 0, 0, 2, 3]) == [0, 1, 1, 2, 3] and ref.depths([-1, 1]) is None and ref.depths([0]) is None


@pytest.mark.parametrize("page", [16, 64])
def test_attention_over_pages_is_attention_over_the_rows_in_order(page):
    rng = np.random.default_rng(page)
    B, n, Hq, Hkv, L = 3, 6, 4, 2, np.array([40, 0, 63], np.int32)
    parent = np.array([[-1, 0, 0, 1, 3, 2]] * B, np.int32)
    P = 5 if page == 16 else 2
    N = B * P
    table = rng.permutation(N).reshape(B, P)
    kp, vp = _bf16((N, Hkv, page, D), 1), _bf16((N, Hkv, page, D), 2)
    q = _bf16((B, n, Hq, D), 3)
    out, tol = ref.tree_attn_paged(q, kp, vp, table, L, parent, D ** -0.5)
    k, v = (torch.stack([torch.cat([x[i] for i in table[b]], 1) for b in range(B)]) for x in (kp, vp))
    want = oracle.tree_attn(q, k, v, L, parent, D ** -0.5)
    assert np.abs(out.numpy() - want).max() < 1e-6 and float(tol.min()) > 0


def test_assignment_by_hand():
    """Two slots of 20 and 32 rows, pages of 16; slot 1 goes on with slot 0, then slot 0 ends."""
    t, held, refs, lens, copies = ref.pages_assign([[-1] * 3] * 2, [0, 0], [0] * 6, [0, 0], [20, 32], None, 16)
    assert t == [[0, 1, -1], [2, 3, -1]] and held == [2, 2] and refs == [1, 1, 1, 1, 0, 0] and lens == [0, 0] and not copies
    t, held, refs, lens, copies = ref.pages_assign(t, held, refs, [20, 32], [0, 13], [0, 0], 16)
    # page 0 is shared, page 1's four rows are copied into page 4, rows 20 .. 32 need page 5
    assert t == [[0, 1, -1], [0, 4, 5]] and held == [2, 3] and refs == [2, 1, 0, 0, 1, 1] and lens == [20, 20] and copies == [(1, 4, 4)]
    t, held, refs, lens, copies = ref.pages_assign(t, held, refs, lens, [0, 0], [-1, 1], 16)
    assert t == [[-1, -1, -1], [0, 4, -1]] and refs == [1, 0, 0, 0, 1, 0] and lens == [0, 20] and not copies
    assert ref.pages_assign(t, held, refs, lens, [48, 28], None, 16) is not None
    assert ref.pages_assign(t, held, refs, lens, [49, 0], None, 16) is None            # wider than the table
    assert ref.pages_assign([[0, 1, 2]], [3], [1, 1, 1], [40], [0], [0], 16) is not None
    assert ref.pages_assign([[0, 1, 2], [-1] * 3], [3, 0], [1, 1, 1], [40, 0], [0, 1], None, 16) is None      # no page is free


def test_assignment_keeps_counts_and_rows():
    """Over random steps: refs are the table's counts, and every slot reads the rows it should."""
    rng = np.random.default_rng(4)
    B, P, page, N = 5, 6, 16, 80
    table, held, refs, lens = [[-1] * P] * B, [0] * B, [0] * N, [0] * B
    store = np.zeros((N, page), np.int64)
    seen = [[] for _ in range(B)]                          # what each slot's rows should hold
    stamp = 1
    for step in range(60):
        src = None if step % 3 == 0 else [int(x) for x in rng.integers(-1, B, B)]
        now = [lens[b] if src is None else (lens[src[b]] if src[b] >= 0 else 0) for b in range(B)]
        grow = [int(rng.integers(0, min(40, P * page - x) + 1)) for x in now]
        got = ref.pages_assign(table, held, refs, lens, grow, src, page)
        if got is None:
            continue
        table, held, refs, lens, copies = got
        for frm, to, rows in copies:
            store[to, :rows] = store[frm, :rows]
        seen = [list(seen[b]) if src is None else (list(seen[src[b]]) if src[b] >= 0 else []) for b in range(B)]
        assert lens == now and [sum(p in row[:m] for row, m in zip(table, held)) for p in range(N)] == refs
        for b in range(B):
            add = int(rng.integers(0, grow[b] + 1))
            for r in range(lens[b], lens[b] + add):
                store[table[b][r // page], r % page] = stamp
                seen[b].append(stamp)
                stamp += 1
            lens[b] += add
            back = int(rng.integers(0, 5))
            lens[b] = max(0, lens[b] - back)
            seen[b] = seen[b][:lens[b]]
        for b in range(B):
            assert [store[p][r] for p, r in ref.places(table[b], page, range(lens[b]))] == seen[b]


def test_commit_over_pages_is_compaction_of_the_rows_in_order():
    rng = np.random.default_rng(9)
    B, P, page, Hkv, layers, n, depth = 3, 3, 16, 2, 2, 9, 4
    N = B * P
    table = rng.permutation(N).reshape(B, P)
    k, v = _bf16((layers, N, Hkv, page, D), 1), _bf16((layers, N, Hkv, page, D), 2)
    dense = [torch.stack([torch.cat([x[:, i] for i in table[b]], 2) for b in range(B)], 1) for x in (k, v)]
    L = np.array([13, 0, 30], np.int32)
    path = np.array([[0, 2, 3, 8, -1], [0, 1, -1, -1, -1], [0, 4, 5, 6, 8]], np.int32)
    acc = np.array([3, 1, 4], np.int32)
    bits = [x.contiguous().view(torch.int16).numpy().view(np.uint16).copy() for x in dense]
    lens = ref.pages_commit([k, v], table, list(L), path, list(acc), depth, page, N)
    oracle.kv_compact(bits[0], bits[1], L, path, acc, depth)
    assert lens == list(L)
    for x, y in zip((k, v), bits):
        got = torch.stack([torch.cat([x[:, i] for i in table[b]], 2) for b in range(B)], 1)
        assert np.array_equal(got.contiguous().view(torch.int16).numpy().view(np.uint16), y)
