"""Pins of the tolerance that the 8-bit tree attention is tested to: it passes weights of 11 bits and
fails weights of 8."""
import numpy as np
import pytest
import torch

from oracle import prompt_kv8 as ref
from tests.test_gpu_kv8_bounds import D, cancelling_rows


def _with_rounded_weights(q, k, v, kt, vt, L, parent, dtype):
    """The attention in 64 bits, but for the weights (2^6 for the largest) and the output."""
    q, kt, vt = q.double(), kt.double(), vt.double()
    n, G = q.shape[1], q.shape[2]
    sees = ref._tree_sees(n, L[0], parent[0])
    K, V = ref._key_rows(*k, kt, 0, 0, L[0]), ref._key_rows(*v, vt, 0, 0, L[0])
    out = torch.zeros_like(q)
    for g in range(G):
        s = torch.where(sees, (q[0, :, g] @ K.T) * D ** -0.5, -torch.inf)
        p = 64 * torch.exp(s - s.amax(1, keepdim=True))
        out[0, :, g] = (p.to(dtype).double() @ V) / p.sum(1, keepdim=True)
    return out.bfloat16().double()


@pytest.mark.parametrize("seed", [161, 171, 181])
def test_tolerance_tells_eight_bits_of_a_weight_from_eleven(seed):
    q, k, v, kt, vt, L, parent = cancelling_rows(seed)
    o, tight = ref.tree_attn_kv8_tight(q, *k, *v, kt, vt, L, parent, D ** -0.5)
    o2, loose = ref.tree_attn_kv8(q, *k, *v, kt, vt, L, parent, D ** -0.5)
    assert torch.equal(o, o2) or torch.allclose(o, o2, rtol=1e-9, atol=1e-12)
    half = (_with_rounded_weights(q, k, v, kt, vt, L, parent, torch.float16) - o).abs()
    bf16 = (_with_rounded_weights(q, k, v, kt, vt, L, parent, torch.bfloat16) - o).abs()
    assert (half <= tight).all()
    assert (bf16 <= loose).all() and not (bf16 <= tight).all()


def test_tolerance_of_a_wide_spread_is_that_of_eight_bits():
    q, k, v, kt, vt, L, parent = cancelling_rows(161)
    v[1][:] = 1.0
    vt[0, 3] = 2.0 ** 20
    _, wide = ref.tree_attn_kv8_tight(q, *k, *v, kt, vt, L, parent, D ** -0.5)
    o, _ = ref.tree_attn_kv8(q, *k, *v, kt, vt, L, parent, D ** -0.5)
    assert ((_with_rounded_weights(q, k, v, kt, vt, L, parent, torch.bfloat16) - o).abs() <= wide).all()


def test_row_exponents():
    rows = torch.zeros(4, D).double()
    rows[0, 3], rows[1, 5], rows[2, 0] = -1.0, 255.0, 2.0 ** -130
    e = ref._row_exponents(rows)
    assert e[0] == -7 and e[1] == 0 and torch.isnan(e[2]) and torch.isnan(e[3])
    assert np.isfinite(float(e[0]))
