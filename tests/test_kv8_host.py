"""Host checks of the prompt attention and the 8-bit cache's calls (no GPU work is done), and
pins of their 64-bit forms."""
import ctypes
import os

import numpy as np
import pytest
import torch

from oracle import prompt_kv8 as ref

OK, INVALID, SHAPE, CAPACITY = 0, 1, 2, 3
P = 4096                                     # a 16-byte aligned, never dereferenced address


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


PROMPT = "q k v cu_q cu_k out lse Tq Tk B Hq Hkv d qs ks vs scale status stream".split()
PROMPT_OK = dict(q=P, k=P, v=P, cu_q=P, cu_k=P, out=P, lse=P, Tq=10, Tk=10, B=1, Hq=8, Hkv=2, d=128, qs=1024, ks=256,
                 vs=256, scale=0.1, status=None, stream=None)
APPEND = "k v cu pos k8 v8 k_scale v_scale T B Hkv d Lmax ks vs status stream".split()
APPEND_OK = dict(k=P, v=P, cu=P, pos=P, k8=P, v8=P, k_scale=P, v_scale=P, T=10, B=1, Hkv=2, d=128, Lmax=64, ks=256,
                 vs=256, status=None, stream=None)
COMMIT = "k v k8 v8 k_scale v_scale kv_len kv_out path acc layers B n Hkv d Lmax D status stream".split()
COMMIT_OK = dict(k=P, v=P, k8=P, v8=P, k_scale=P, v_scale=P, kv_len=P, kv_out=P, path=P, acc=P, layers=2, B=1, n=4, Hkv=2,
                 d=128, Lmax=64, D=3, status=None, stream=None)
TREE = "q k8 v8 k_scale v_scale kt vt kv_len parent out B n Hq Hkv d Lmax scale ws ws_bytes status stream".split()
TREE_OK = dict(q=P, k8=P, v8=P, k_scale=P, v_scale=P, kt=P, vt=P, kv_len=P, parent=P, out=P, B=1, n=4, Hq=8, Hkv=2,
               d=128, Lmax=64, scale=0.1, ws=P, ws_bytes=1 << 40, status=None, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(Tq=-1), INVALID), (dict(Tk=-1), INVALID), (dict(B=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hkv=0), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(d=64), SHAPE), (dict(Hkv=3), SHAPE), (dict(Hq=258, Hkv=2, qs=258 * 128), SHAPE), (dict(qs=1016), INVALID),
    (dict(qs=1028), INVALID), (dict(ks=248), INVALID), (dict(vs=260), INVALID), (dict(q=None), INVALID),
    (dict(k=None), INVALID), (dict(cu_k=None), INVALID), (dict(out=None), INVALID), (dict(q=P + 8), INVALID),
    (dict(v=P + 2), INVALID)])
def test_prompt_attention_refusals(L, change, status):
    assert _call(L.eagle_prompt_attn, PROMPT, PROMPT_OK, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), INVALID), (dict(B=-1), INVALID), (dict(Hkv=0), INVALID), (dict(Lmax=0), INVALID), (dict(d=64), SHAPE),
    (dict(Hkv=70000, ks=70000 * 128, vs=70000 * 128), SHAPE), (dict(ks=128), INVALID), (dict(vs=257), INVALID),
    (dict(k=None), INVALID), (dict(pos=None), INVALID), (dict(v_scale=None), INVALID), (dict(k8=P + 8), INVALID),
    (dict(v=P + 2), INVALID)])
def test_append_refusals(L, change, status):
    assert _call(L.eagle_kv8_append, APPEND, APPEND_OK, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(layers=-1), INVALID), (dict(B=-1), INVALID), (dict(n=0), INVALID), (dict(Hkv=0), INVALID), (dict(Lmax=0), INVALID),
    (dict(D=-1), INVALID), (dict(d=64), SHAPE), (dict(n=65), SHAPE), (dict(D=65), SHAPE), (dict(k=None), INVALID),
    (dict(kv_out=None), INVALID), (dict(k_scale=None), INVALID), (dict(v8=P + 4), INVALID)])
def test_commit_refusals(L, change, status):
    assert _call(L.eagle_kv8_commit, COMMIT, COMMIT_OK, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(B=-1), INVALID), (dict(n=0), INVALID), (dict(Hq=0), INVALID), (dict(Lmax=0), INVALID), (dict(scale=-1.0), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(n=65), SHAPE), (dict(d=64), SHAPE), (dict(Hkv=3), SHAPE), (dict(q=None), INVALID),
    (dict(kt=None), INVALID), (dict(v_scale=None), INVALID), (dict(out=P + 8), INVALID), (dict(k8=P + 1), INVALID)])
def test_tree_attention_kv8_refusals(L, change, status):
    assert _call(L.eagle_tree_attn_kv8, TREE, TREE_OK, **change) == status


def test_empty_batches_are_no_ops_with_null_pointers(L):
    none = lambda good: {k: None for k, v in good.items() if v == P}  # noqa: E731
    for fn, names, good in ((L.eagle_prompt_attn, PROMPT, PROMPT_OK), (L.eagle_kv8_append, APPEND, APPEND_OK),
                            (L.eagle_kv8_commit, COMMIT, COMMIT_OK), (L.eagle_tree_attn_kv8, TREE, TREE_OK)):
        assert _call(fn, names, good, **none(good), B=0) == OK
        assert _call(fn, names, good, **none(good)) == INVALID
    assert _call(L.eagle_prompt_attn, PROMPT, PROMPT_OK, **none(PROMPT_OK), Tq=0) == OK
    assert _call(L.eagle_kv8_append, APPEND, APPEND_OK, **none(APPEND_OK), T=0) == OK
    assert _call(L.eagle_kv8_commit, COMMIT, COMMIT_OK, **none(COMMIT_OK), layers=0) == OK


def test_binding_refuses_host_tensors_and_wrong_types():
    import eagle_tree_speculative_gb300 as E
    bf = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    i32 = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError):
        E.eagle_prompt_attn(bf, bf, bf, i32)
    with pytest.raises(TypeError):
        E.eagle_kv8_append(bf, bf, i32, i32[:1], *E.kv8_cache(1, 1, 2, 32, device="cpu"))
    with pytest.raises(TypeError):
        E.eagle_kv8_commit(bf[None, None], bf[None, None], *E.kv8_cache(1, 1, 2, 32, device="cpu"), i32[:1], i32, i32[:1], 1)
    with pytest.raises(TypeError):
        E.eagle_tree_attn_kv8(bf[None], *E.kv8_cache(1, 1, 2, 32, device="cpu"), bf[None], bf[None], i32[:1], i32)


# ---------------------------------------------------------------- pins of the 64-bit forms
def test_e4m3_codes_agree_with_torch():
    """The search over all values against torch's own conversion, over every value, every
    midpoint and its neighbours."""
    v = np.sort(ref._VALUES)
    mid = (v[1:] + v[:-1]) / 2
    x = np.concatenate([v, mid, mid * (1 + 2.0 ** -20), mid * (1 - 2.0 ** -20)])
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    got = ref.e4m3(x.astype(np.float32).astype(np.float64))
    zero = (got & 0x7F) == 0
    assert np.array_equal(got[~zero], want[~zero]) and ((want[zero] & 0x7F) == 0).all()
    assert ref.e4m3(np.array([1e9, -1e9, 460.0, np.inf, np.nan])).tolist() == [0x7E, 0xFE, 0x7E, 0x7E, 0x7F]


def test_scale_is_the_least_power_of_two():
    assert ref.scale_of(448.0) == 1.0 and ref.scale_of(448.0001) == 2.0 and ref.scale_of(224.0) == 0.5
    assert ref.scale_of(0.0) == 2.0 ** -64 and ref.scale_of(1e-30) == 2.0 ** -64


def test_rows_written_in_parts_equal_rows_written_at_once_up_to_the_last_rounding():
    """Appending in two parts gives the scale of appending at once; a code differs only where
    the first part was rounded on a finer grid before (at most one step)."""
    g = np.random.default_rng(0)
    x = g.normal(size=(32, 128))
    x[20:] *= 6
    one, two = np.zeros((32, 128), np.uint8), np.zeros((32, 128), np.uint8)
    s1, s2 = np.ones(1), np.ones(1)
    ref.write_rows(x, 0, one, s1)
    ref.write_rows(x[:11], 0, two, s2)
    ref.write_rows(x[11:], 11, two, s2)
    assert s1 == s2
    a, b = ref._value(one) * s1, ref._value(two) * s2
    assert (np.abs(a - x) <= 2.0 ** -4 * np.abs(x) + 2.0 ** -10 * s1).all()
    assert (np.abs(a - b) <= 2.0 ** -9 * s1 + 1e-12).all()


def test_prompt_form_against_a_softmax_written_out():
    g = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn(n, h, 128, generator=g).bfloat16() for n, h in ((5, 4), (7, 2), (7, 2)))
    out, lse, _ = ref.prompt_attn(q, k, v, [0, 2, 5], [0, 4, 7], 0.09)
    s = (q[1, 3].double() @ k[:4, 1].double().T) * 0.09                 # the second query of sequence 0 sees all four
    assert torch.allclose(out[1, 3], torch.softmax(s, 0) @ v[:4, 1].double())
    assert torch.allclose(lse[1, 3], torch.logsumexp(s, 0))
    assert torch.allclose(out[2, 0], v[4, 0].double())                  # the first of sequence 1 sees one key


def test_tree_form_with_an_exact_cache_is_ordinary_attention():
    """Codes with scale 1 are exact values: node 1 (parent 0) sees the cache, 0 and itself."""
    g = np.random.default_rng(1)
    codes = g.integers(0, 120, (1, 1, 40, 128)).astype(np.uint8)
    one = np.ones((1, 1, 2))
    t = torch.Generator().manual_seed(2)
    q, kt, vt = (torch.randn(1, 3, h, 128, generator=t).bfloat16() for h in (2, 1, 1))
    out, _ = ref.tree_attn_kv8(q, codes, one, codes, one, kt, vt, [33], [[-1, 0, 0]], 1e-3)
    rows = torch.from_numpy(ref._value(codes[0, 0, :33]))
    k, v = torch.cat([rows, kt[0, :2, 0].double()]), torch.cat([rows, vt[0, :2, 0].double()])
    assert torch.allclose(out[0, 1, 1], torch.softmax(q[0, 1, 1].double() @ k.T * 1e-3, 0) @ v)
