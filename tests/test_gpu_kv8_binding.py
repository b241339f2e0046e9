"""What the Python binding of the prompt and 8-bit cache calls refuses before anything is launched."""
import pytest
import torch

pytestmark = pytest.mark.gpu
D = 128


def _good():
    import eagle_tree_speculative_gb300 as E
    B, n, Hq, Hkv, Lmax, T, layers, depth = 2, 4, 4, 2, 64, 9, 3, 3
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    k8, v8, ks, vs = E.kv8_cache(layers, B, Hkv, Lmax)
    one = dict(k8=k8[0], v8=v8[0], k_scale=ks[0], v_scale=vs[0])
    return {
        "eagle_prompt_attn": dict(q=bf(T, Hq, D), k=bf(T, Hkv, D), v=bf(T, Hkv, D), cu_q=i32(B + 1), cu_k=i32(B + 1),
                                  out=bf(T, Hq, D), lse=torch.zeros(T, Hq, device="cuda"), dev_status=i32(1)),
        "eagle_kv8_append": dict(k=bf(T, Hkv, D), v=bf(T, Hkv, D), cu=i32(B + 1), pos=i32(B), **one, dev_status=i32(1)),
        "eagle_kv8_commit": dict(k_tree=bf(layers, B, n, Hkv, D), v_tree=bf(layers, B, n, Hkv, D), k8=k8, v8=v8, k_scale=ks,
                                 v_scale=vs, kv_len=i32(B), path=i32(B, depth + 1), accept_len=i32(B) - 1, max_depth=depth,
                                 kv_len_out=i32(B), dev_status=i32(1)),
        "eagle_tree_attn_kv8": dict(q=bf(B, n, Hq, D), **one, k_tree=bf(B, n, Hkv, D), v_tree=bf(B, n, Hkv, D), kv_len=i32(B),
                                    parent=i32(B, n), out=bf(B, n, Hq, D), dev_status=i32(1)),
    }


CALLS = sorted(["eagle_prompt_attn", "eagle_kv8_append", "eagle_kv8_commit", "eagle_tree_attn_kv8"])


@pytest.mark.parametrize("name", CALLS)
def test_every_tensor_is_checked(name):
    """Each tensor in turn on the host, of another type, with another row, and not dense."""
    import eagle_tree_speculative_gb300 as E
    good = _good()[name]
    call = getattr(E, name)
    call(**good)
    for arg, t in good.items():
        if not isinstance(t, torch.Tensor):
            continue
        bits = t.view(torch.uint8) if t.dtype is torch.float8_e4m3fn else t
        wrong = {"host": t.cpu(), "type": torch.zeros(t.shape, dtype=torch.float64, device="cuda")}
        if arg != "dev_status":
            wrong["row"] = torch.cat([bits, bits[:1]]).view(t.dtype)
        if t.dim() > 1 and t.shape[-1] > 1:
            wrong["dense"] = bits.transpose(-1, -2).contiguous().view(t.dtype).transpose(-1, -2)
        for what, x in wrong.items():
            # one more row of the first argument, or of the sequence counts, may only show against the others
            with pytest.raises((TypeError, ValueError, E.EagleError)):
                call(**{**good, arg: x})
                pytest.fail(f"{name}: {arg} ({what}) was taken")
    torch.cuda.synchronize()


def test_strides_that_the_kernels_cannot_take():
    import eagle_tree_speculative_gb300 as E
    good = _good()["eagle_prompt_attn"]
    base = torch.zeros(9, 4 * D + 4, dtype=torch.bfloat16, device="cuda")
    odd = base[:, :4 * D].unflatten(1, (4, D))                     # a token stride that is no multiple of 8
    with pytest.raises(ValueError):
        E.eagle_prompt_attn(**{**good, "q": odd})
    with pytest.raises(ValueError):
        E.eagle_prompt_attn(**{**good, "q": good["q"][:1].expand(9, 4, D)})
    shifted = torch.zeros(9 * 4 * D + 4, dtype=torch.bfloat16, device="cuda")[4:].view(9, 4, D)
    with pytest.raises(E.EagleError):                              # not 16-byte aligned
        E.eagle_prompt_attn(**{**good, "q": shifted})


def test_workspaces_too_small_or_unaligned():
    import eagle_tree_speculative_gb300 as E
    good = _good()["eagle_tree_attn_kv8"]
    need = E.tree_attn_kv8_workspace_size(2, 4, 4, 2, D, 64)
    assert need > 0
    for ws in (torch.empty(need - 1, dtype=torch.uint8, device="cuda"), torch.empty(need + 16, dtype=torch.uint8, device="cuda")[8:]):
        with pytest.raises(E.EagleError):
            E.eagle_tree_attn_kv8(**good, workspace=ws)
    E.eagle_tree_attn_kv8(**good, workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
