"""GPU parity of eagle_prompt_attn with the 64-bit form: packed sequences of different
lengths, chunks behind a prefix, group sizes that do and do not divide a tile, strided
inputs, rows that see nothing, rows of no sequence.

Tolerance per output element: oracle/prompt_kv8.py derives it (bf16 output and weights).
lse: the score's error (2^-17 of the sum of magnitudes) plus 2^-20 relative and absolute.
"""
import numpy as np
import pytest
import torch

from oracle import prompt_kv8 as ref

pytestmark = pytest.mark.gpu
D = 128


def _E():
    import eagle_tree_speculative_gb300 as E
    return E


def _rows(T, H, seed, gain=0.5):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, D, generator=g) * torch.exp(gain * torch.randn(D, generator=g))
    return x.bfloat16()


def _cu(lens, start=0):
    return [start] + list(start + np.cumsum(lens))


def _dev(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _compare(out, lse, want, scale=D ** -0.5):
    o, z, tol = want
    here = ~torch.isnan(z)
    off = (out.double().cpu() - o).abs()
    worst = torch.where(here[..., None], off / (tol + 1e-30), 0.0).max()
    assert worst <= 1.0, f"output off by {float(worst):.3g} times the bound"
    got = lse.double().cpu()
    none = here & torch.isinf(z)
    assert torch.equal(got[none], z[none]), "a row that sees nothing has lse = -inf"
    fin = here & ~torch.isinf(z)
    assert ((got - z).abs()[fin] <= 1e-5 + 1e-5 * z.abs()[fin]).all()


def _check(q_lens, Hq, Hkv, seed, k_lens=None, scale=None):
    E = _E()
    k_lens = q_lens if k_lens is None else k_lens
    q, k, v = _rows(sum(q_lens), Hq, seed), _rows(sum(k_lens), Hkv, seed + 1), _rows(sum(k_lens), Hkv, seed + 2)
    cq, ck = _cu(q_lens), _cu(k_lens)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = E.eagle_prompt_attn(q.cuda(), k.cuda(), v.cuda(), _dev(cq), _dev(ck), scale=scale,
                                   return_lse=True, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    _compare(out, lse, ref.prompt_attn(q, k, v, cq, ck, scale or D ** -0.5))


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 511, 513, 700])
def test_one_prompt_of_every_length(n):
    _check([n], 8, 2, n)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 1), (3, 1), (4, 4), (5, 1), (6, 2), (7, 1), (14, 2), (8, 1), (16, 1),
                                    (12, 1), (33, 1), (64, 2), (128, 1), (100, 1)])
def test_group_sizes(Hq, Hkv):
    _check([150, 3, 301], Hq, Hkv, 50 + Hq)


def test_many_sequences_of_different_lengths():
    """More sequences than a warp has lanes, some empty."""
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(0, 90, size=75)]
    lens[5] = lens[40] = lens[74] = 0
    lens[33] = 400
    _check(lens, 4, 2, 7)


@pytest.mark.parametrize("nq,nk", [(1, 1), (1, 500), (7, 128), (64, 129), (100, 1000), (300, 301)])
def test_chunks_behind_a_prefix(nq, nk):
    _check([nq, 5, nq], 8, 2, 11 + nq, k_lens=[nk, 5, nk + 13])


def test_rows_that_see_nothing():
    """More queries than keys (or no keys at all): the first nq - nk rows are 0, lse -inf."""
    _check([200, 40, 3, 130], 4, 1, 13, k_lens=[60, 0, 3, 1])


def test_sharp_softmax():
    """Scores of tens of units: one key carries a row, and the running maximum jumps."""
    _check([400, 260], 4, 2, 17, scale=2.0)


def test_late_large_keys_move_the_running_maximum():
    """Every tile's keys are larger than the last one's, so the reference maximum moves in
    each tile."""
    E = _E()
    n = 900
    q, k, v = _rows(n, 2, 61), _rows(n, 1, 62), _rows(n, 1, 63)
    k = (k.float() * torch.linspace(0.05, 3.0, n)[:, None, None]).bfloat16()
    out, lse = E.eagle_prompt_attn(q.cuda(), k.cuda(), v.cuda(), _dev([0, n]), return_lse=True)
    _compare(out, lse, ref.prompt_attn(q, k, v, [0, n], [0, n], D ** -0.5))


def test_strided_tokens_of_a_fused_projection():
    """q, k and v as slices of one [T, (Hq + 2 Hkv) d] projection output."""
    E = _E()
    Hq, Hkv, lens = 8, 2, [77, 130, 1]
    T = sum(lens)
    qkv = _rows(T, Hq + 2 * Hkv, 21).cuda()
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    cu = _cu(lens)
    out, lse = E.eagle_prompt_attn(q, k, v, _dev(cu), return_lse=True)
    torch.cuda.synchronize()
    _compare(out, lse, ref.prompt_attn(q.cpu(), k.cpu(), v.cpu(), cu, cu, D ** -0.5))


def test_rows_of_no_sequence_are_left_and_may_hold_anything():
    """cu begins at 9 and ends before the last rows, which hold NaN and infinities; the output
    there keeps its sentinel."""
    E = _E()
    lens, lead, trail = [70, 133], 9, 23
    T = lead + sum(lens) + trail
    q, k, v = _rows(T, 4, 31), _rows(T, 2, 32), _rows(T, 2, 33)
    cu = _cu(lens, lead)
    for t in (q, k, v):
        t[:lead] = float("nan")
        t[cu[-1]:] = float("inf")
        t[-1] = float("nan")
    out = torch.full((T, 4, D), 3.5, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, 4), 7.0, device="cuda")
    E.eagle_prompt_attn(q.cuda(), k.cuda(), v.cuda(), _dev(cu), out=out, lse=lse)
    torch.cuda.synchronize()
    _compare(out, lse, ref.prompt_attn(q, k, v, cu, cu, D ** -0.5))
    edge = torch.cat([out[:lead], out[cu[-1]:]])
    assert (edge == 3.5).all() and (lse[:lead] == 7.0).all() and (lse[cu[-1]:] == 7.0).all()


def test_other_sequences_values_do_not_leak():
    """NaN in one sequence stays in it: its neighbours share tiles with it."""
    E = _E()
    lens = [50, 90, 40]
    q, k, v = _rows(180, 4, 41), _rows(180, 2, 42), _rows(180, 2, 43)
    cu = _cu(lens)
    want = ref.prompt_attn(q, k, v, cu, cu, D ** -0.5)
    k[50:140], v[50:140] = float("nan"), float("nan")
    out, lse = E.eagle_prompt_attn(q.cuda(), k.cuda(), v.cuda(), _dev(cu), return_lse=True)
    torch.cuda.synchronize()
    keep = torch.ones(180, dtype=torch.bool)
    keep[50:140] = False
    _compare(out[keep.cuda()], lse[keep.cuda()], [t[keep] for t in want])
    assert torch.isnan(out[50:140].float()).all()


@pytest.mark.parametrize("cu_q,cu_k", [([0, 5, 3, 8], [0, 3, 5, 8]), ([0, 3, 5, 9], [0, 3, 5, 8]),
                                       ([-1, 3, 5, 8], [0, 3, 5, 8]), ([0, 3, 5, 8], [0, 6, 5, 8]),
                                       ([0, 3, 5, 8], [0, 3, 5, 90])])
def test_bad_offsets_write_nothing(cu_q, cu_k):
    E = _E()
    q, k, v = _rows(8, 4, 51), _rows(8, 2, 52), _rows(8, 2, 53)
    out = torch.full((8, 4, D), 2.0, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    E.eagle_prompt_attn(q.cuda(), k.cuda(), v.cuda(), _dev(cu_q), _dev(cu_k), out=out, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == E.EAGLE_DEV_CAPACITY and (out == 2.0).all()


def test_empty_batches():
    E = _E()
    q, k = torch.empty(0, 4, D, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 2, D, dtype=torch.bfloat16, device="cuda")
    assert E.eagle_prompt_attn(q, k, k, _dev([0])).shape == (0, 4, D)
    out, lse = E.eagle_prompt_attn(q, k, k, _dev([0, 0, 0]), return_lse=True)
    assert out.shape == (0, 4, D) and lse.shape == (0, 4)
    # queries without any keys
    q = _rows(5, 4, 1).cuda()
    out, lse = E.eagle_prompt_attn(q, k, k, _dev([0, 5]), _dev([0, 0]), return_lse=True)
    assert (out == 0).all() and torch.isinf(lse).all()


def test_runs_twice_the_same_and_in_a_captured_graph():
    """Bit-equal results on a side stream, and from a captured graph replayed on new inputs."""
    E = _E()
    lens = [300, 77, 129]
    q, k, v = (_rows(sum(lens), h, s).cuda() for h, s in ((8, 71), (2, 72), (2, 73)))
    cu = _dev(_cu(lens))
    first = E.eagle_prompt_attn(q, k, v, cu)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    second = E.eagle_prompt_attn(q, k, v, cu, stream=side)
    side.synchronize()
    assert torch.equal(first, second)
    out = torch.empty_like(first)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        E.eagle_prompt_attn(q, k, v, cu, out=out)
    q2, cu2 = _rows(sum(lens), 8, 74).cuda(), _dev(_cu([129, 300, 77]))
    want = E.eagle_prompt_attn(q2, k, v, cu2)
    q.copy_(q2)
    cu.copy_(cu2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_full_size_rows_against_the_64_bit_form():
    """A 5000-token prompt beside short ones, 32/8 heads: the last 40 queries and a short
    neighbour, every head."""
    E = _E()
    lens, Hq, Hkv = [5000, 61, 900], 32, 8
    T = sum(lens)
    q, k, v = _rows(T, Hq, 81), _rows(T, Hkv, 82), _rows(T, Hkv, 83)
    out, lse = E.eagle_prompt_attn(q.cuda(), k.cuda(), v.cuda(), _dev(_cu(lens)), return_lse=True)
    torch.cuda.synchronize()
    want = ref.prompt_attn(q[4960:5061], k[:5061], v[:5061], [0, 40, 101], [0, 5000, 5061], D ** -0.5)
    _compare(out[4960:5061], lse[4960:5061], want)
