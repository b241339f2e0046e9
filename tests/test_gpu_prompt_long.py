"""eagle_prompt_attn on the longest sequences: 2^27 keys at most."""
import pytest
import torch

pytestmark = pytest.mark.gpu
D = 128


def test_a_sequence_of_too_many_keys_is_refused():
    """One query behind more keys than a unit can go through before a wait gives up: the status is set
    and nothing is written.  34 GB of keys, which nothing reads."""
    import eagle_tree_speculative_gb300 as E
    T = 2 ** 27 + 1
    if torch.cuda.mem_get_info()[0] < 40 * 2 ** 30:
        pytest.skip("needs 34 GB")
    k = torch.empty(T, 1, D, dtype=torch.bfloat16, device="cuda")
    q = torch.ones(1, 1, D, dtype=torch.bfloat16, device="cuda")
    out, st = torch.full_like(q, 5.0), torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    E.eagle_prompt_attn(q, k, k, cu(0, 1), cu(0, T), out=out, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == E.EAGLE_DEV_CAPACITY and (out == 5.0).all()


def test_one_query_behind_a_million_keys():
    """Equal keys: the output is the mean of the values, whichever part of them a tile holds."""
    import eagle_tree_speculative_gb300 as E
    T = 2 ** 20 + 77
    k = torch.ones(T, 1, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros(T, 1, D, dtype=torch.bfloat16, device="cuda")
    v[:, 0, 3], v[: T // 2, 0, 4], v[-1, 0, 5] = 1.0, 2.0, 2.0 ** 20
    q = torch.ones(1, 1, D, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    out, lse = E.eagle_prompt_attn(q, k, v, cu(0, 1), cu(0, T), return_lse=True, dev_status=st)
    torch.cuda.synchronize()
    want = torch.zeros(D).double()
    want[3], want[4], want[5] = 1.0, 2.0 * (T // 2) / T, 2.0 ** 20 / T
    # equal weights; the products' sum takes T additions at most, the weights' T / 2, each off by 2^-24: 2^-4, 2^-5
    assert int(st.item()) == 0
    assert ((out[0, 0].double().cpu() - want).abs() <= (2.0 ** -8 + 2.0 ** -3) * want).all()
    assert abs(float(lse[0, 0]) - (D * D ** -0.5 + float(torch.log(torch.tensor(float(T)))))) <= 2.0 ** -4
