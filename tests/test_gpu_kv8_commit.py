"""eagle_kv8_commit at the numbers of sequences where its launch changes, bit for bit."""
import numpy as np
import pytest
import torch

from oracle import prompt_kv8 as ref

pytestmark = pytest.mark.gpu
D = 128


def _dev(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("over", [-75, 0, 1, 153])
def test_commit_of_many_sequences(over, in_place):
    """From about half as many sequences as the card has SMs to twice as many, two heads and three
    layers, blocks that hold rows already, one to three blocks a path, skipped sequences."""
    import eagle_tree_speculative_gb300 as E
    B = torch.cuda.get_device_properties(0).multi_processor_count + over
    layers, Hkv, n, depth, Lmax = 3, 2, 45, 40, 130
    rng = np.random.default_rng(B)
    acc = rng.integers(-1, depth + 1, B)
    L = rng.integers(0, 85, B)
    path = np.full((B, depth + 1), -1, np.int32)
    for b, a in enumerate(acc):
        if a >= 0:
            path[b, :a + 1] = [0] + sorted(rng.choice(np.arange(1, n), a, replace=False))
    g = torch.Generator().manual_seed(B)
    x, y = ((torch.randn(layers, B, n, Hkv, D, generator=g) * torch.exp(torch.randn(B, 1, 1, 1, generator=g))).bfloat16() for _ in range(2))
    want, got = [], []
    for t in (x, y):
        codes = torch.randint(0, 0x7F, (layers, B, Hkv, Lmax, D), generator=g, dtype=torch.int32).to(torch.uint8).numpy()
        scales = np.exp2(rng.integers(-12, 2, (layers, B, Hkv, -(-Lmax // 32))).astype(np.float64))
        got += [torch.from_numpy(codes.copy()).cuda().view(torch.float8_e4m3fn), torch.from_numpy(scales).float().cuda()]
        ref.kv8_commit(t.double().numpy(), L, path, acc, codes, scales)
        want += [codes, scales]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv_len = _dev(L)
    out = kv_len if in_place else torch.full_like(kv_len, -3)
    E.eagle_kv8_commit(x.cuda(), y.cuda(), got[0], got[2], got[1], got[3], kv_len, _dev(path), _dev(acc), depth, kv_len_out=out, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and out.tolist() == [int(l + a + 1) for l, a in zip(L, acc)]
    for k in (0, 2):
        assert np.array_equal(got[k].view(torch.uint8).cpu().numpy(), want[k])
        assert np.array_equal(got[k + 1].double().cpu().numpy(), want[k + 1])
